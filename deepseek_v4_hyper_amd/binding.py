"""ctypes binding of libds4hc.so (include/ds4hc.h).

Argument marshalling only: each Python function checks tensor shapes/dtypes,
passes device pointers and the current HIP stream to the C function of the
same name, and turns a non-OK status into an exception. Every step of the op
runs in the library's HIP kernels; PyTorch only provides device memory and
the stream. There is no fallback: if the library is missing, calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libds4hc.so")

DS4HC_OK = 0
DS4HC_ERR_INVALID_ARG = 1
DS4HC_ERR_UNSUPPORTED = 2
DS4HC_ERR_HIP = 3
DS4HC_F32 = 0
DS4HC_BF16 = 1
DS4HC_F16 = 2
DS4HC_FLAG_DETERMINISTIC = 1
DS4HC_FLAG_FORCE_ROWRES = 2
DS4HC_FLAG_FORCE_SPLITK = 4
DS4HC_FLAG_FORCE_TILE = 8
DS4HC_ROPE_HALF = 1
DS4HC_ROPE_INVERSE = 2
DS4HC_ATTN_FULL = 1

EXPORTED = ("ds4hc_pre", "ds4hc_sinkhorn", "ds4hc_post", "ds4hc_fused", "ds4hc_workspace_bytes",
            "ds4hc_post_pre", "ds4hc_post_pre_workspace_bytes", "ds4hc_post_pre_noalloc",
            "ds4hc_partials", "ds4hc_partials_workspace_bytes", "ds4hc_combine",
            "ds4hc_rope", "ds4hc_rope_frequencies", "ds4hc_latent_append", "ds4hc_latent_attn",
            "ds4hc_latent_attn_workspace_bytes", "ds4hc_latent_prefill",
            "ds4hc_status_string", "ds4hc_last_hip_error", "ds4hc_abi_version")


class Ds4hcError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where} failed: {status_string(status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class Params(ctypes.Structure):
    _fields_ = [("n_hc", ctypes.c_int32), ("d", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("sinkhorn_iters", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Strides(ctypes.Structure):
    """ds4hc_strides: elements between tokens and between heads."""
    _fields_ = [("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class PagedCache(ctypes.Structure):
    """ds4hc_paged_cache: the cache's layout and the batch of sequences of a call."""
    _fields_ = [("dtype", ctypes.c_int), ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p)]


def make_params(n_hc: int, d: int, rms_eps: float = 1e-6, sinkhorn_iters: int = 20,
                flags: int = 0) -> Params:
    return Params(int(n_hc), int(d), float(rms_eps), int(sinkhorn_iters), int(flags))


_lib = None


def load(path: str = LIB_PATH):
    """Load libds4hc.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libds4hc.so not found at {path}; build it with "
                           "`python -m deepseek_v4_hyper_amd.build_lib`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Params)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    lib.ds4hc_pre.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ds4hc_sinkhorn.argtypes = [i64, i32, i32, vp, vp, vp]
    lib.ds4hc_post.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, vp]
    lib.ds4hc_fused.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ds4hc_post_pre.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ds4hc_post_pre_noalloc.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.ds4hc_partials.argtypes = [P, i64, ctypes.c_int, vp, vp, vp, vp, sz, vp]
    lib.ds4hc_combine.argtypes = [P, i32, i64, ctypes.c_int, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    u32, f32, f64, dt = ctypes.c_uint32, ctypes.c_float, ctypes.c_double, ctypes.c_int
    C, S = ctypes.POINTER(PagedCache), Strides
    lib.ds4hc_rope.argtypes = [i64, i32, i32, dt, vp, S, vp, vp, f32, u32, vp, S, vp]
    lib.ds4hc_rope_frequencies.argtypes = [i32, f64, f64, i64, f64, f64, vp, vp]
    lib.ds4hc_latent_append.argtypes = [C, i64, dt, vp, i64, vp, f32, vp, vp, f32, u32, vp, vp]
    lib.ds4hc_latent_attn.argtypes = [C, i64, i32, f32, vp, S, vp, S, vp, vp, i32, vp, S, vp, vp, sz, vp]
    lib.ds4hc_latent_attn_workspace_bytes.argtypes = [C, i64, i32]
    lib.ds4hc_latent_attn_workspace_bytes.restype = sz
    lib.ds4hc_latent_prefill.argtypes = [i64, i64, i32, i32, dt, f32, u32, vp, vp, vp, i64, vp, vp, vp, vp, vp]
    for f in ("ds4hc_rope", "ds4hc_rope_frequencies", "ds4hc_latent_append", "ds4hc_latent_attn",
              "ds4hc_latent_prefill"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("ds4hc_pre", "ds4hc_sinkhorn", "ds4hc_post", "ds4hc_fused", "ds4hc_post_pre",
              "ds4hc_post_pre_noalloc", "ds4hc_partials", "ds4hc_combine"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("ds4hc_workspace_bytes", "ds4hc_post_pre_workspace_bytes",
              "ds4hc_partials_workspace_bytes"):
        getattr(lib, f).argtypes = [P, i64, ctypes.c_int]
        getattr(lib, f).restype = sz
    lib.ds4hc_status_string.argtypes = [ctypes.c_int]
    lib.ds4hc_status_string.restype = ctypes.c_char_p
    lib.ds4hc_last_hip_error.restype = ctypes.c_char_p
    lib.ds4hc_abi_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().ds4hc_status_string(int(status)).decode()
    except Exception:
        return f"status {status}"


def abi_version() -> int:
    return load().ds4hc_abi_version()


def _check(status: int, where: str):
    if status != DS4HC_OK:
        detail = load().ds4hc_last_hip_error().decode() if status == DS4HC_ERR_HIP else ""
        raise Ds4hcError(status, where, detail)


# ------------------------------------------------------------------ raw pointer calls

def ds4hc_workspace_bytes(params: Params, T: int, dtype: int) -> int:
    return int(load().ds4hc_workspace_bytes(ctypes.byref(params), int(T), int(dtype)))


def ds4hc_post_pre_workspace_bytes(params: Params, T: int, dtype: int) -> int:
    return int(load().ds4hc_post_pre_workspace_bytes(ctypes.byref(params), int(T), int(dtype)))


def ds4hc_post_pre_raw(params, T, dtype, X, coeffs_prev, layer_out, W_next, bias_next, X_out,
                       layer_in, coeffs, logits, ws, ws_bytes, stream):
    return load().ds4hc_post_pre(ctypes.byref(params), int(T), int(dtype), X, coeffs_prev,
                                 layer_out, W_next, bias_next, X_out, layer_in, coeffs, logits, ws,
                                 int(ws_bytes), stream)


NOALLOC_SCRATCH_BYTES = 2 << 20   # DS4HC_NOALLOC_SCRATCH_BYTES


def ds4hc_post_pre_noalloc_raw(params, T, dtype, X, coeffs_prev, layer_out, W_next, bias_next,
                               X_out, layer_in, coeffs, logits, stream):
    return load().ds4hc_post_pre_noalloc(ctypes.byref(params), int(T), int(dtype), X, coeffs_prev,
                                         layer_out, W_next, bias_next, X_out, layer_in, coeffs,
                                         logits, stream)


def ds4hc_pre_raw(params, T, dtype, X, W, bias, layer_in, coeffs, logits, ws, ws_bytes, stream):
    return load().ds4hc_pre(ctypes.byref(params), int(T), int(dtype), X, W, bias, layer_in,
                            coeffs, logits, ws, int(ws_bytes), stream)


def ds4hc_fused_raw(params, T, dtype, X, W, bias, layer_out, layer_in, coeffs, X_out, ws,
                    ws_bytes, stream):
    return load().ds4hc_fused(ctypes.byref(params), int(T), int(dtype), X, W, bias, layer_out,
                              layer_in, coeffs, X_out, ws, int(ws_bytes), stream)


def ds4hc_post_raw(params, T, dtype, X, coeffs, layer_out, X_out, stream):
    return load().ds4hc_post(ctypes.byref(params), int(T), int(dtype), X, coeffs, layer_out,
                             X_out, stream)


def ds4hc_sinkhorn_raw(T, n_hc, iters, logits_res, H, stream):
    return load().ds4hc_sinkhorn(int(T), int(n_hc), int(iters), logits_res, H, stream)


def ds4hc_partials_workspace_bytes(params: Params, T: int, dtype: int) -> int:
    return int(load().ds4hc_partials_workspace_bytes(ctypes.byref(params), int(T), int(dtype)))


def ds4hc_partials_raw(params, T, dtype, X_share, W_share, partials, ws, ws_bytes, stream):
    return load().ds4hc_partials(ctypes.byref(params), int(T), int(dtype), X_share, W_share,
                                 partials, ws, int(ws_bytes), stream)


def ds4hc_combine_raw(params, d_total, T, dtype, G, partials, bias, X_share, layer_out_share,
                      layer_in_share, coeffs, X_out_share, stream):
    return load().ds4hc_combine(ctypes.byref(params), int(d_total), int(T), int(dtype), int(G),
                                partials, bias, X_share, layer_out_share, layer_in_share, coeffs,
                                X_out_share, stream)


# ------------------------------------------------------------------ torch-tensor calls

def _torch():
    import torch
    return torch


def _state_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DS4HC_F32
    if t.dtype == torch.bfloat16:
        return DS4HC_BF16
    raise TypeError(f"state dtype must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Context in which the binding allocates what it passes to a call on `stream`.

    The caching allocator ties a block to the stream that was current when it
    was allocated, and hands it out again once it is freed with no regard for
    work still queued on other streams. Buffers the binding creates (workspace,
    default outputs) are therefore allocated with the kernels' own stream
    current: a workspace dropped on return is then reused only by work ordered
    after the kernels that read it."""
    torch = _torch()
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _need(t, shape, dtype, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def _empty(shape, dtype, device):
    return _torch().empty(shape, dtype=dtype, device=device)


def _scratch(need, workspace, device):
    """The caller's workspace, or a fresh one of `need` bytes (none if 0)."""
    if workspace is None and need:
        workspace = _empty(need, _torch().uint8, device)
    return workspace, (workspace.numel() * workspace.element_size() if workspace is not None else 0)


def ds4hc_pre(X, W, bias, *, rms_eps=1e-6, sinkhorn_iters=20, flags=0, layer_in=None,
              coeffs=None, logits=None, workspace=None, stream=None, want_logits=False):
    """HC-pre. X [T, n, d] (float32|bfloat16), W [m, n*d] float16, bias [m] float32.
    Returns (layer_in [T, d], coeffs [T, m], logits [T, m] or None)."""
    torch = _torch()
    T, n, d = X.shape
    m = 2 * n + n * n
    dt = _state_code(X)
    p = make_params(n, d, rms_eps, sinkhorn_iters, flags)
    _need(X, (T, n, d), X.dtype, "X")
    _need(W, (m, n * d), torch.float16, "W")
    _need(bias, (m,), torch.float32, "bias")
    with _on(stream):
        if layer_in is None:
            layer_in = _empty((T, d), X.dtype, X.device)
        if coeffs is None:
            coeffs = _empty((T, m), torch.float32, X.device)
        if logits is None and want_logits:
            logits = _empty((T, m), torch.float32, X.device)
        workspace, ws_bytes = _scratch(ds4hc_workspace_bytes(p, T, dt), workspace, X.device)
    _check(ds4hc_pre_raw(p, T, dt, _ptr(X), _ptr(W), _ptr(bias), _ptr(layer_in), _ptr(coeffs),
                         _ptr(logits), _ptr(workspace), ws_bytes, _stream(stream)), "ds4hc_pre")
    return layer_in, coeffs, logits


def ds4hc_fused(X, W, bias, layer_out, *, rms_eps=1e-6, sinkhorn_iters=20, flags=0,
                layer_in=None, coeffs=None, X_out=None, workspace=None, stream=None,
                want_coeffs=True):
    """Whole HC op. Returns (layer_in [T, d], coeffs [T, m] or None, X_out [T, n, d])."""
    torch = _torch()
    T, n, d = X.shape
    m = 2 * n + n * n
    dt = _state_code(X)
    p = make_params(n, d, rms_eps, sinkhorn_iters, flags)
    _need(X, (T, n, d), X.dtype, "X")
    _need(W, (m, n * d), torch.float16, "W")
    _need(bias, (m,), torch.float32, "bias")
    _need(layer_out, (T, d), X.dtype, "layer_out")
    with _on(stream):
        if layer_in is None:
            layer_in = _empty((T, d), X.dtype, X.device)
        if coeffs is None and want_coeffs:
            coeffs = _empty((T, m), torch.float32, X.device)
        if X_out is None:
            X_out = _empty(X.shape, X.dtype, X.device)
        workspace, ws_bytes = _scratch(ds4hc_workspace_bytes(p, T, dt), workspace, X.device)
    _check(ds4hc_fused_raw(p, T, dt, _ptr(X), _ptr(W), _ptr(bias), _ptr(layer_out),
                           _ptr(layer_in), _ptr(coeffs), _ptr(X_out), _ptr(workspace), ws_bytes,
                           _stream(stream)), "ds4hc_fused")
    return layer_in, coeffs, X_out


def ds4hc_post(X, coeffs, layer_out, *, X_out=None, stream=None, rms_eps=1e-6,
               sinkhorn_iters=20):
    """hc_post: X' = H.X + post (x) layer_out. X_out may be X itself (in place)."""
    torch = _torch()
    T, n, d = X.shape
    m = 2 * n + n * n
    dt = _state_code(X)
    p = make_params(n, d, rms_eps, sinkhorn_iters, 0)
    _need(X, (T, n, d), X.dtype, "X")
    _need(coeffs, (T, m), torch.float32, "coeffs")
    _need(layer_out, (T, d), X.dtype, "layer_out")
    with _on(stream):
        if X_out is None:
            X_out = _empty(X.shape, X.dtype, X.device)
    _check(ds4hc_post_raw(p, T, dt, _ptr(X), _ptr(coeffs), _ptr(layer_out), _ptr(X_out),
                          _stream(stream)), "ds4hc_post")
    return X_out


def ds4hc_post_pre(X, coeffs_prev, layer_out, W_next, bias_next, *, rms_eps=1e-6,
                   sinkhorn_iters=20, flags=0, X_out=None, layer_in=None, coeffs=None,
                   logits=None, workspace=None, stream=None, want_logits=False):
    """post(l) then pre(l+1): X' = H_l.X + post_l (x) layer_out_l, then HC-pre of
    site l+1 on X'. Returns (X_out [T,n,d], layer_in [T,d], coeffs [T,m], logits or None).
    X_out may be X itself (in place)."""
    torch = _torch()
    T, n, d = X.shape
    m = 2 * n + n * n
    dt = _state_code(X)
    p = make_params(n, d, rms_eps, sinkhorn_iters, flags)
    _need(X, (T, n, d), X.dtype, "X")
    _need(coeffs_prev, (T, m), torch.float32, "coeffs_prev")
    _need(layer_out, (T, d), X.dtype, "layer_out")
    _need(W_next, (m, n * d), torch.float16, "W_next")
    _need(bias_next, (m,), torch.float32, "bias_next")
    with _on(stream):
        if X_out is None:
            X_out = _empty(X.shape, X.dtype, X.device)
        if layer_in is None:
            layer_in = _empty((T, d), X.dtype, X.device)
        if coeffs is None:
            coeffs = _empty((T, m), torch.float32, X.device)
        if logits is None and want_logits:
            logits = _empty((T, m), torch.float32, X.device)
        workspace, ws_bytes = _scratch(ds4hc_post_pre_workspace_bytes(p, T, dt), workspace,
                                       X.device)
    _check(ds4hc_post_pre_raw(p, T, dt, _ptr(X), _ptr(coeffs_prev), _ptr(layer_out), _ptr(W_next),
                              _ptr(bias_next), _ptr(X_out), _ptr(layer_in), _ptr(coeffs),
                              _ptr(logits), _ptr(workspace), ws_bytes, _stream(stream)),
           "ds4hc_post_pre")
    return X_out, layer_in, coeffs, logits


def ds4hc_partials(X_share, W_share, *, flags=0, partials=None, workspace=None, stream=None):
    """One column share: X_share [T, n, d_s], W_share [m, n*d_s] -> partials [T, m+1]
    (unnormalised fn dots, then the sum of squares)."""
    torch = _torch()
    T, n, ds = X_share.shape
    m = 2 * n + n * n
    dt = _state_code(X_share)
    p = make_params(n, ds, 1e-6, 20, flags)
    _need(X_share, (T, n, ds), X_share.dtype, "X_share")
    _need(W_share, (m, n * ds), torch.float16, "W_share")
    with _on(stream):
        if partials is None:
            partials = _empty((T, m + 1), torch.float32, X_share.device)
        workspace, ws_bytes = _scratch(ds4hc_partials_workspace_bytes(p, T, dt), workspace,
                                       X_share.device)
    _check(ds4hc_partials_raw(p, T, dt, _ptr(X_share), _ptr(W_share), _ptr(partials),
                              _ptr(workspace), ws_bytes, _stream(stream)), "ds4hc_partials")
    return partials


def ds4hc_combine(partials, bias, X_share, layer_out_share, d_total, *, rms_eps=1e-6,
                  sinkhorn_iters=20, coeffs=None, want_coeffs=True, layer_in_share=None,
                  X_out_share=None, stream=None):
    """partials [G, T, m+1] of all shares -> (layer_in_share, coeffs or None, X_out_share)."""
    torch = _torch()
    T, n, ds = X_share.shape
    m = 2 * n + n * n
    G = partials.shape[0]
    dt = _state_code(X_share)
    p = make_params(n, ds, rms_eps, sinkhorn_iters, 0)
    _need(partials, (G, T, m + 1), torch.float32, "partials")
    _need(bias, (m,), torch.float32, "bias")
    _need(X_share, (T, n, ds), X_share.dtype, "X_share")
    _need(layer_out_share, (T, ds), X_share.dtype, "layer_out_share")
    with _on(stream):
        if layer_in_share is None:
            layer_in_share = _empty((T, ds), X_share.dtype, X_share.device)
        if coeffs is None and want_coeffs:
            coeffs = _empty((T, m), torch.float32, X_share.device)
        if X_out_share is None:
            X_out_share = _empty(X_share.shape, X_share.dtype, X_share.device)
    _check(ds4hc_combine_raw(p, d_total, T, dt, G, _ptr(partials), _ptr(bias), _ptr(X_share),
                             _ptr(layer_out_share), _ptr(layer_in_share), _ptr(coeffs),
                             _ptr(X_out_share), _stream(stream)), "ds4hc_combine")
    return layer_in_share, coeffs, X_out_share


def ds4hc_sinkhorn(logits_res, *, iters=20, H=None, stream=None):
    """Sinkhorn of residual logits [T, n, n] float32 -> H [T, n, n]."""
    torch = _torch()
    T, n, n2 = logits_res.shape
    _need(logits_res, (T, n, n), torch.float32, "logits_res")
    with _on(stream):
        if H is None:
            H = _empty(logits_res.shape, torch.float32, logits_res.device)
    _check(ds4hc_sinkhorn_raw(T, n, iters, _ptr(logits_res), _ptr(H), _stream(stream)),
           "ds4hc_sinkhorn")
    return H


def ds4hc_post_pre_noalloc(X, coeffs_prev, layer_out, W_next, bias_next, X_out, layer_in, coeffs,
                           *, logits=None, rms_eps=1e-6, sinkhorn_iters=20, flags=0, stream=None):
    """ds4hc_post_pre with the library's device-resident scratch instead of a
    workspace. Every output is the caller's (this function allocates nothing)."""
    torch = _torch()
    T, n, d = X.shape
    m = 2 * n + n * n
    dt = _state_code(X)
    p = make_params(n, d, rms_eps, sinkhorn_iters, flags)
    _need(X, (T, n, d), X.dtype, "X")
    _need(coeffs_prev, (T, m), torch.float32, "coeffs_prev")
    _need(layer_out, (T, d), X.dtype, "layer_out")
    _need(W_next, (m, n * d), torch.float16, "W_next")
    _need(bias_next, (m,), torch.float32, "bias_next")
    _need(X_out, (T, n, d), X.dtype, "X_out")
    _need(layer_in, (T, d), X.dtype, "layer_in")
    _need(coeffs, (T, m), torch.float32, "coeffs")
    if logits is not None:
        _need(logits, (T, m), torch.float32, "logits")
    _check(ds4hc_post_pre_noalloc_raw(p, T, dt, _ptr(X), _ptr(coeffs_prev), _ptr(layer_out),
                                      _ptr(W_next), _ptr(bias_next), _ptr(X_out), _ptr(layer_in),
                                      _ptr(coeffs), _ptr(logits), _stream(stream)),
           "ds4hc_post_pre_noalloc")
    return X_out, layer_in, coeffs, logits


# ------------------------------------------------------------------ operators of an attention site

def ds4hc_rope_raw(N, heads, dim, dtype, x, x_strides, positions, inv_freq, amplitude, flags, y,
                   y_strides, stream):
    return load().ds4hc_rope(int(N), int(heads), int(dim), int(dtype), x, Strides(*x_strides),
                             positions, inv_freq, float(amplitude), int(flags), y,
                             Strides(*y_strides), stream)


def ds4hc_latent_append_raw(c, N, src_dtype, kv, kv_stride, norm_weight, rms_eps, positions,
                            inv_freq, amplitude, flags, cache, stream):
    return load().ds4hc_latent_append(ctypes.byref(c), int(N), int(src_dtype), kv, int(kv_stride),
                                      norm_weight, float(rms_eps), positions, inv_freq,
                                      float(amplitude), int(flags), cache, stream)


def ds4hc_latent_attn_raw(c, N, heads, scale, ql, ql_strides, qr, qr_strides, cache, tree_mask,
                          mask_words, out, out_strides, lse, ws, ws_bytes, stream):
    return load().ds4hc_latent_attn(ctypes.byref(c), int(N), int(heads), float(scale), ql,
                                    Strides(*ql_strides), qr, Strides(*qr_strides), cache,
                                    tree_mask, int(mask_words), out, Strides(*out_strides), lse,
                                    ws, int(ws_bytes), stream)


def ds4hc_latent_attn_workspace_bytes(c: PagedCache, N: int, heads: int) -> int:
    return int(load().ds4hc_latent_attn_workspace_bytes(ctypes.byref(c), int(N), int(heads)))


def ds4hc_latent_prefill_raw(N, S, n_seqs, heads, dtype, scale, flags, q, kv, k_rope, k_rope_stride,
                             cu_q, cu_k, out, lse, stream):
    return load().ds4hc_latent_prefill(int(N), int(S), int(n_seqs), int(heads), int(dtype),
                                       float(scale), int(flags), q, kv, k_rope, int(k_rope_stride),
                                       cu_q, cu_k, out, lse, stream)


# These calls take a few microseconds on the GPU, so their checks are made quick: one
# look at each tensor, and the reason spelt out only for what did not pass. They record no
# gradient: outputs of inputs that require one are detached.

@functools.lru_cache(maxsize=None)
def _codes():
    torch = _torch()
    return {torch.float32: DS4HC_F32, torch.bfloat16: DS4HC_BF16, torch.float16: DS4HC_F16}


@functools.lru_cache(maxsize=4096)
def _strides(token: int, head: int) -> Strides:
    return Strides(token, head)


def _any_code(t, name, halves=False) -> int:
    code = _codes().get(t.dtype)
    if code is None or (halves and code == DS4HC_F32):
        raise TypeError(f"{name}: dtype {t.dtype} is not supported")
    return code


def _device(stream) -> int:
    """The device that the call runs on: the calling thread's current one."""
    here = _torch().cuda.current_device()
    if stream is not None and stream.device.index != here:
        raise ValueError(f"the stream is on {stream.device}, the call on the current device, cuda:{here}")
    return here


def _tensors(**tensors):
    """Device tensors (the rest of a call's checks are made one by one)."""
    torch = _torch()
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")


def _raw_stream(stream, here) -> int:
    return _torch()._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _dense(t, shape, dtype, name, here):
    """A dense array on the call's device."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != here:
        _tensors(**{name: t})
        if t.get_device() != here:
            raise ValueError(f"{name} is on {t.device}, the call runs on the current device, cuda:{here}")
        _need(t, shape, dtype, name)


def _rows(t, shape, dtype, name, here):
    """An array on the call's device whose last dimension is dense."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != here or (shape[-1] > 1 and t.stride(-1) != 1):
        _tensors(**{name: t})
        if t.get_device() != here:
            raise ValueError(f"{name} is on {t.device}, the call runs on the current device, cuda:{here}")
        if t.shape != shape or t.dtype is not dtype:
            raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
        raise ValueError(f"{name}: the last dimension must be dense")


def ds4hc_rope_frequencies(dim, base=10000.0, *, factor=1.0, original_length=0, beta_fast=32.0,
                           beta_slow=1.0, device=None):
    """Angles a position of the dim / 2 pairs (float64 tensor) and the amplitude, for
    ds4hc_rope and ds4hc_latent_append. factor > 1 stretches the positions: all pairs
    alike, or by the ramp in include/ds4hc.h if original_length is given."""
    torch = _torch()
    f = torch.empty(max(int(dim) // 2, 1), dtype=torch.float64)
    amplitude = ctypes.c_float()
    _check(load().ds4hc_rope_frequencies(int(dim), float(base), float(factor), int(original_length),
                                         float(beta_fast), float(beta_slow), _ptr(f),
                                         ctypes.byref(amplitude)), "ds4hc_rope_frequencies")
    return (f if device is None else f.to(device)), amplitude.value


def ds4hc_rope(x, positions, inv_freq, *, interleaved=True, inverse=False, amplitude=1.0, out=None,
               stream=None):
    """Rotary positions. x [N, heads, dim] (float32|bfloat16|float16; a view of part of
    a head is fine, the last dimension dense), positions [N] int64, inv_freq [dim / 2]
    float64. out may be x itself (in place). Returns out [N, heads, dim], detached; the
    gradient of x is that of out rotated with inverse=True."""
    torch = _torch()
    if not getattr(x, "is_cuda", False):
        _tensors(x=x)
    here, shape, dtype = _device(stream), x.shape, x.dtype
    dt = _any_code(x, "x")
    if len(shape) != 3:
        raise ValueError(f"x must be [N, heads, dim], got {tuple(shape)}")
    N, heads, dim = shape
    _rows(x, shape, dtype, "x", here)
    _dense(positions, (N,), torch.int64, "positions", here)
    _dense(inv_freq, (dim // 2,), torch.float64, "inv_freq", here)
    if out is None:
        with _on(stream):
            out = _empty(shape, dtype, x.device)
    else:
        _rows(out, shape, dtype, "out", here)
    xs, os_ = x.stride(), out.stride()
    flags = (0 if interleaved else DS4HC_ROPE_HALF) | (DS4HC_ROPE_INVERSE if inverse else 0)
    st = load().ds4hc_rope(N, heads, dim, dt, x.data_ptr(), _strides(xs[0], xs[1]), positions.data_ptr(),
                           inv_freq.data_ptr(), amplitude, flags, out.data_ptr(), _strides(os_[0], os_[1]),
                           _raw_stream(stream, here))
    if st:
        _check(st, "ds4hc_rope")
    return out


def _paged(cache, cu_q, kv_len, block_table, here=None):
    torch = _torch()
    here = torch.cuda.current_device() if here is None else here
    shape, table = cache.shape, block_table.shape
    if len(shape) != 3 or kv_len.dim() != 1 or len(table) != 2:
        raise ValueError("cache must be [pages, page_size, d_latent + 64], kv_len [B] and block_table [B, max_pages]")
    pages, page_size, D = shape
    B = kv_len.shape[0]
    i32 = torch.int32
    _dense(cache, shape, cache.dtype, "cache", here)
    _dense(cu_q, (B + 1,), i32, "cu_q", here)
    _dense(kv_len, (B,), i32, "kv_len", here)
    _dense(block_table, (B, table[1]), i32, "block_table", here)
    return PagedCache(_any_code(cache, "cache", True), D - 64, 64, page_size, pages, B, table[1], cu_q.data_ptr(),
                      kv_len.data_ptr(), block_table.data_ptr())


def ds4hc_latent_append(kv, positions, inv_freq, cache, cu_q, kv_len, block_table, *,
                        norm_weight=None, rms_eps=1e-6, interleaved=True, amplitude=1.0,
                        stream=None):
    """Norm, rotate and store the call's N tokens into the paged cache.
    kv [N, d_latent + 64] (latent | rope key; rows may be strided), positions [N] int64,
    inv_freq [32] float64, cache [pages, page_size, d_latent + 64] bfloat16|float16,
    cu_q [B + 1], kv_len [B], block_table [B, max_pages] int32, norm_weight [d_latent]
    float32 or None (no norm). Returns cache."""
    torch = _torch()
    if not getattr(kv, "is_cuda", False):
        _tensors(kv=kv)
    here = _device(stream)
    c = _paged(cache, cu_q, kv_len, block_table, here)
    src = _any_code(kv, "kv")
    N, D = kv.shape[0], cache.shape[2]
    _rows(kv, (N, D), kv.dtype, "kv", here)
    _dense(positions, (N,), torch.int64, "positions", here)
    _dense(inv_freq, (32,), torch.float64, "inv_freq", here)
    if norm_weight is not None:
        _dense(norm_weight, (c.d_latent,), torch.float32, "norm_weight", here)
    st = load().ds4hc_latent_append(ctypes.byref(c), N, src, kv.data_ptr(), kv.stride(0) if N > 1 else D,
                                    None if norm_weight is None else norm_weight.data_ptr(), rms_eps,
                                    positions.data_ptr(), inv_freq.data_ptr(), amplitude,
                                    0 if interleaved else DS4HC_ROPE_HALF, cache.data_ptr(), _raw_stream(stream, here))
    if st:
        _check(st, "ds4hc_latent_append")
    return cache


def ds4hc_latent_attn(q_latent, q_rope, cache, cu_q, kv_len, block_table, *, scale, tree_mask=None,
                      out=None, lse=None, workspace=None, stream=None, want_lse=False):
    """Latent attention over the paged cache, absorbed form. q_latent [N, heads, d_latent]
    and q_rope [N, heads, 64] (strided views are fine), cache and batch as in
    ds4hc_latent_append, tree_mask [N, words] int64 or None (causal among the call's own
    tokens). Returns (out [N, heads, d_latent], lse [N, heads] float32 or None), detached.
    Rows behind the last sequence are left as they were."""
    torch = _torch()
    if not getattr(q_latent, "is_cuda", False):
        _tensors(q_latent=q_latent)
    here = _device(stream)
    c = _paged(cache, cu_q, kv_len, block_table, here)
    dtype = cache.dtype
    if q_latent.dim() != 3:
        raise ValueError(f"q_latent must be [N, heads, d_latent], got {tuple(q_latent.shape)}")
    N, heads, _ = q_latent.shape
    shape = (N, heads, c.d_latent)
    _rows(q_latent, shape, dtype, "q_latent", here)
    _rows(q_rope, (N, heads, 64), dtype, "q_rope", here)
    words = 0
    if tree_mask is not None:
        words = tree_mask.shape[-1] if tree_mask.dim() else 0
        _dense(tree_mask, (N, words), torch.int64, "tree_mask", here)
        if words < 1:  # (has no address: would be taken for no mask)
            raise ValueError("tree_mask must be [N, words] of one word a token at least")
    with _on(stream):
        if out is None:
            out = _empty(shape, dtype, cache.device)
        else:
            _rows(out, shape, dtype, "out", here)
        if lse is not None:
            _dense(lse, (N, heads), torch.float32, "lse", here)
        elif want_lse:
            lse = _empty((N, heads), torch.float32, cache.device)
        if workspace is not None:
            _tensors(workspace=workspace)
            if workspace.get_device() != here or not workspace.is_contiguous():
                raise ValueError("workspace must be a dense array on the call's device")
        workspace, ws_bytes = _scratch(load().ds4hc_latent_attn_workspace_bytes(ctypes.byref(c), N, heads), workspace,
                                       cache.device)
    ls, rs, os_ = q_latent.stride(), q_rope.stride(), out.stride()
    st = load().ds4hc_latent_attn(ctypes.byref(c), N, heads, scale, q_latent.data_ptr(), _strides(ls[0], ls[1]),
                                  q_rope.data_ptr(), _strides(rs[0], rs[1]), cache.data_ptr(),
                                  None if tree_mask is None else tree_mask.data_ptr(), words, out.data_ptr(),
                                  _strides(os_[0], os_[1]), None if lse is None else lse.data_ptr(),
                                  None if workspace is None else workspace.data_ptr(), ws_bytes,
                                  _raw_stream(stream, here))
    if st:
        _check(st, "ds4hc_latent_attn")
    return out, lse


def ds4hc_latent_prefill(q, kv, k_rope, cu_q, cu_k, *, scale, causal=True, out=None, lse=None,
                         stream=None, want_lse=False):
    """Latent attention over expanded keys and values of a ragged batch. q [N, heads, 192],
    kv [S, heads, 256] (128 key | 128 value elements a head), k_rope [S, 64] (rows may be
    strided), cu_q and cu_k [B + 1] int32. Returns (out [N, heads, 128], lse [N, heads]
    float32 or None), detached. Rows behind the last sequence are left as they were."""
    torch = _torch()
    if not getattr(q, "is_cuda", False):
        _tensors(q=q)
    here, dtype = _device(stream), q.dtype
    dt = _any_code(q, "q", True)
    if q.dim() != 3 or kv.dim() != 3 or cu_q.dim() != 1:
        raise ValueError("q must be [N, heads, 192], kv [S, heads, 256] and cu_q [B + 1]")
    N, heads, _ = q.shape
    S, B = kv.shape[0], cu_q.shape[0] - 1
    _dense(q, (N, heads, 192), dtype, "q", here)
    _dense(kv, (S, heads, 256), dtype, "kv", here)
    _rows(k_rope, (S, 64), dtype, "k_rope", here)
    _dense(cu_q, (B + 1,), torch.int32, "cu_q", here)
    _dense(cu_k, (B + 1,), torch.int32, "cu_k", here)
    with _on(stream):
        if out is None:
            out = _empty((N, heads, 128), dtype, q.device)
        else:
            _dense(out, (N, heads, 128), dtype, "out", here)
        if lse is not None:
            _dense(lse, (N, heads), torch.float32, "lse", here)
        elif want_lse:
            lse = _empty((N, heads), torch.float32, q.device)
    st = load().ds4hc_latent_prefill(N, S, B, heads, dt, scale, 0 if causal else DS4HC_ATTN_FULL, q.data_ptr(),
                                     kv.data_ptr(), k_rope.data_ptr(), k_rope.stride(0) if S > 1 else 64,
                                     cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(),
                                     None if lse is None else lse.data_ptr(), _raw_stream(stream, here))
    if st:
        _check(st, "ds4hc_latent_prefill")
    return out, lse
