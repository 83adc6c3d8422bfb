"""The attention-site entry points' refusals, and the host function of the rotary
frequencies: everything that needs no GPU. Rejected calls enqueue nothing; the fake
device addresses are never dereferenced, so these run only where no GPU is visible."""
import ctypes
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs without a GPU")
BAD, UNSUP, HIP, OK = B.DS4HC_ERR_INVALID_ARG, B.DS4HC_ERR_UNSUPPORTED, B.DS4HC_ERR_HIP, B.DS4HC_OK
A = 1 << 40


def fake(i, off=0):
    return ctypes.c_void_p(A * (i + 1) + off)


def addr(i, off=0):
    return A * (i + 1) + off


def paged(**over):
    a = dict(dtype=B.DS4HC_BF16, d_latent=512, d_rope=64, page_size=64, n_pages=100, n_seqs=4, max_pages=32,
             cu_q=addr(20), kv_len=addr(21), block_table=addr(22))
    a.update(over)
    return B.PagedCache(*[a[f] for f, _ in B.PagedCache._fields_])


def rope(N=8, heads=4, dim=64, dt=B.DS4HC_BF16, x=fake(0), xs=(256, 64), pos=fake(1), f=fake(2), amp=1.0, flags=0,
         y=fake(3), ys=(256, 64)):
    return B.ds4hc_rope_raw(N, heads, dim, dt, x, xs, pos, f, amp, flags, y, ys, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP),                                                # valid: the launch fails, there is no GPU
    (dict(N=0, x=None, y=None, pos=None, f=None), OK),
    (dict(N=-1), BAD), (dict(heads=0), BAD), (dict(dim=63), BAD), (dict(dim=0), BAD), (dict(dt=3), BAD),
    (dict(flags=4), BAD), (dict(amp=math.inf), BAD), (dict(amp=math.nan), BAD), (dict(xs=(-1, 64)), BAD),
    (dict(ys=(256, -64)), BAD), (dict(heads=1025), UNSUP), (dict(dim=514), UNSUP), (dict(N=(1 << 24) + 1), UNSUP),
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(pos=None), BAD), (dict(f=None), BAD),
    (dict(x=fake(0, 1)), BAD), (dict(y=fake(3, 1)), BAD), (dict(pos=fake(1, 4)), BAD), (dict(f=fake(2, 4)), BAD),
    (dict(x=fake(0, 2), xs=(257, 65)), HIP),                      # any element-aligned address and stride
    (dict(xs=(0, 0)), HIP),                                       # broadcast input
    (dict(ys=(0, 64)), BAD), (dict(ys=(256, 63)), BAD), (dict(ys=(255, 64)), BAD),   # rows of y overlap
    (dict(ys=(64, 512)), HIP),                                    # heads outside tokens
    (dict(y=fake(0)), HIP),                                       # in place
    (dict(y=fake(0), ys=(512, 64)), BAD), (dict(y=fake(0, 128)), BAD),
    (dict(y=fake(1)), BAD), (dict(y=fake(2, -64)), BAD),
])
def test_rope_arguments(kw, want):
    assert rope(**kw) == want


def append(c=None, N=8, src=B.DS4HC_BF16, kv=fake(0), stride=576, w=fake(1), eps=1e-6, pos=fake(2), f=fake(3),
           amp=1.0, flags=0, cache=fake(4)):
    return B.ds4hc_latent_append_raw(c or paged(), N, src, kv, stride, w, eps, pos, f, amp, flags, cache, None)


def attn(c=None, N=8, heads=16, scale=0.1, ql=fake(0), ls=(16 * 512, 512), qr=fake(1), rs=(1024, 64), cache=fake(4),
         tree=None, words=0, out=fake(5), os=(16 * 512, 512), lse=fake(6), ws=fake(7), ws_bytes=1 << 36):
    return B.ds4hc_latent_attn_raw(c or paged(), N, heads, scale, ql, ls, qr, rs, cache, tree, words, out, os, lse,
                                   ws, ws_bytes, None)


CACHE = [
    (dict(dtype=3), BAD), (dict(d_latent=0), BAD), (dict(page_size=0), BAD), (dict(page_size=48), BAD),
    (dict(n_pages=0), BAD), (dict(n_seqs=-1), BAD), (dict(max_pages=0), BAD), (dict(d_rope=-1), BAD),
    (dict(dtype=B.DS4HC_F32), UNSUP), (dict(d_latent=384), UNSUP), (dict(d_rope=32), UNSUP),
    (dict(page_size=1 << 17), UNSUP), (dict(n_seqs=(1 << 20) + 1), UNSUP), (dict(max_pages=1 << 25), UNSUP),
    (dict(n_pages=1 << 31), UNSUP),
    (dict(cu_q=None), BAD), (dict(kv_len=None), BAD), (dict(block_table=None), BAD),
    (dict(cu_q=addr(20, 2)), BAD), (dict(kv_len=addr(21, 2)), BAD), (dict(block_table=addr(22, 1)), BAD),
    (dict(n_seqs=0, cu_q=None, kv_len=None, block_table=None), OK), (dict(), HIP),
]


@no_gpu_only
@pytest.mark.parametrize("kw,want", CACHE)
def test_cache_descriptor(kw, want):
    assert append(paged(**kw)) == want
    assert attn(paged(**kw)) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(src=4), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(flags=2), BAD),
    (dict(amp=math.nan), BAD), (dict(stride=575), BAD), (dict(stride=577), BAD), (dict(stride=584), HIP),
    (dict(kv=None), BAD), (dict(pos=None), BAD), (dict(f=None), BAD), (dict(cache=None), BAD), (dict(w=None), HIP),
    (dict(kv=fake(0, 8)), BAD), (dict(cache=fake(4, 8)), BAD), (dict(w=fake(1, 2)), BAD), (dict(pos=fake(2, 4)), BAD),
    (dict(cache=fake(0)), BAD), (dict(cache=fake(20, -64)), BAD), (dict(N=0, kv=None, pos=None, f=None, cache=None), OK),
    (dict(N=(1 << 24) + 1), UNSUP), (dict(src=B.DS4HC_F32), HIP), (dict(src=B.DS4HC_F16), HIP),
])
def test_append_arguments(kw, want):
    assert append(**kw) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(heads=0), BAD), (dict(heads=1025), UNSUP), (dict(scale=0.0), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(ls=(-8, 512)), BAD),
    (dict(ls=(8192, 516)), BAD), (dict(rs=(1028, 64)), BAD), (dict(os=(8192, 511)), BAD), (dict(os=(8184, 512)), BAD),
    (dict(os=(512, 8 * 512)), HIP), (dict(ls=(512, 8 * 512)), HIP), (dict(ls=(0, 0), rs=(0, 0)), HIP),
    (dict(ql=None), BAD), (dict(qr=None), BAD), (dict(cache=None), BAD), (dict(out=None), BAD), (dict(lse=None), HIP),
    (dict(ql=fake(0, 8)), BAD), (dict(qr=fake(1, 2)), BAD), (dict(out=fake(5, 8)), BAD), (dict(lse=fake(6, 2)), BAD),
    (dict(ws=fake(7, 8)), BAD), (dict(tree=fake(8), words=0), BAD), (dict(tree=fake(8, 4), words=1), BAD),
    (dict(tree=fake(8), words=1), HIP), (dict(tree=fake(8), words=1025), UNSUP),
    (dict(out=fake(0)), BAD), (dict(out=fake(4, 1024)), BAD), (dict(lse=fake(5, 64)), BAD), (dict(ws=fake(5)), None),
    (dict(N=0, ql=None, qr=None, cache=None, out=None, ws=None), OK),
])
def test_attn_arguments(kw, want):
    if want is None:  # only where a workspace is used
        want = BAD if B.ds4hc_latent_attn_workspace_bytes(paged(), 8, 16) else HIP
    assert attn(**kw) == want


@no_gpu_only
def test_attn_workspace():
    c = paged()
    need = B.ds4hc_latent_attn_workspace_bytes(c, 8, 16)
    if need:
        assert attn(ws=None) == BAD and attn(ws_bytes=need - 1) == BAD
    assert attn(ws_bytes=need) == HIP
    # the device arrays are not looked at; invalid arguments give 0
    assert B.ds4hc_latent_attn_workspace_bytes(paged(cu_q=None, kv_len=None, block_table=None), 8, 16) == need
    for kw in (dict(d_latent=100), dict(page_size=3), dict(n_seqs=0)):
        assert B.ds4hc_latent_attn_workspace_bytes(paged(**kw), 8, 16) == 0
    assert B.ds4hc_latent_attn_workspace_bytes(c, 0, 16) == 0
    assert B.ds4hc_latent_attn_workspace_bytes(c, 8, 0) == 0


def prefill(N=8, S=16, seqs=2, heads=4, dt=B.DS4HC_BF16, scale=0.1, flags=0, q=fake(0), kv=fake(1), kr=fake(2),
            stride=64, cu_q=fake(3), cu_k=fake(4), out=fake(5), lse=fake(6)):
    return B.ds4hc_latent_prefill_raw(N, S, seqs, heads, dt, scale, flags, q, kv, kr, stride, cu_q, cu_k, out, lse, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(N=-1), BAD), (dict(S=-1), BAD), (dict(seqs=-1), BAD), (dict(heads=0), BAD), (dict(dt=7), BAD),
    (dict(dt=B.DS4HC_F32), UNSUP), (dict(dt=B.DS4HC_F16), HIP), (dict(scale=0.0), BAD), (dict(scale=math.nan), BAD),
    (dict(flags=2), BAD), (dict(flags=1), HIP), (dict(stride=63), BAD), (dict(stride=68), BAD), (dict(stride=576), HIP),
    (dict(heads=1025), UNSUP), (dict(N=(1 << 24) + 1), UNSUP), (dict(S=(1 << 24) + 1), UNSUP),
    (dict(seqs=(1 << 20) + 1), UNSUP), (dict(q=None), BAD), (dict(kv=None), BAD), (dict(kr=None), BAD),
    (dict(cu_q=None), BAD), (dict(cu_k=None), BAD), (dict(out=None), BAD), (dict(lse=None), HIP),
    (dict(S=0, kv=None, kr=None), HIP), (dict(q=fake(0, 8)), BAD), (dict(kv=fake(1, 8)), BAD), (dict(kr=fake(2, 4)), BAD),
    (dict(out=fake(5, 8)), BAD), (dict(cu_q=fake(3, 2)), BAD), (dict(lse=fake(6, 1)), BAD), (dict(out=fake(0)), BAD),
    (dict(lse=fake(5, 16)), BAD), (dict(out=fake(1, 64)), BAD),
    (dict(N=0, q=None, cu_q=None, cu_k=None, out=None), OK), (dict(seqs=0), OK),
])
def test_prefill_arguments(kw, want):
    assert prefill(**kw) == want


def test_hc_entry_points_refuse_float16():
    """DS4HC_F16 is a type of the attention-site operators alone."""
    p = B.make_params(4, 4096)
    assert B.ds4hc_workspace_bytes(p, 4, B.DS4HC_F16) == 0
    if not torch.cuda.is_available():
        assert B.ds4hc_post_raw(p, 4, B.DS4HC_F16, fake(0), fake(1), fake(2), fake(3), None) == BAD


def test_binding_refuses_host_tensors_and_shapes():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        B.ds4hc_rope(t, torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="device tensor"):
        B.ds4hc_latent_prefill(torch.zeros(4, 2, 192), t, t, t, t, scale=1.0)
    with pytest.raises(ValueError, match="device tensor"):
        B.ds4hc_latent_attn(t, t, t, t, t, t, scale=1.0)
    with pytest.raises(ValueError, match="device tensor"):
        B.ds4hc_latent_append(t, t, t, t, t, t, t)


@pytest.mark.parametrize("dim,base,factor,length", [(64, 10000.0, 1.0, 0), (64, 10000.0, 40.0, 4096),
                                                    (128, 500000.0, 8.0, 8192), (2, 10000.0, 4.0, 100),
                                                    (64, 10000.0, 2.0, 0), (96, 1.5, 3.0, 7)])
def test_rope_frequencies(dim, base, factor, length):
    """Against the formula in Python's float64. pow, log and division differ by a few
    last places at most: 1e-13 relative; the amplitude is float32."""
    f, amp = B.ds4hc_rope_frequencies(dim, base, factor=factor, original_length=length)
    want = []
    ramp = factor > 1 and length > 0
    if ramp:
        turns = lambda b: dim * math.log(length / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), dim // 2 - 1)
    for i in range(dim // 2):
        x = base ** (-2 * i / dim)
        k = 1 - min(max((i - lo) / max(hi - lo, 0.001), 0), 1) if ramp else 0.0
        want.append(x * ((1 - k) / factor + k))
    assert f.dtype == torch.float64 and f.shape == (dim // 2,)
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-13, atol=0)
    assert abs(amp - (0.1 * math.log(factor) + 1 if ramp else 1.0)) <= 2.0 ** -23


@pytest.mark.parametrize("kw", [dict(dim=63), dict(dim=0), dict(dim=64, base=1.0), dict(dim=64, base=math.nan),
                                dict(dim=64, factor=0.5), dict(dim=64, factor=math.inf),
                                dict(dim=64, original_length=-1, factor=2.0), dict(dim=514),
                                dict(dim=64, factor=2.0, original_length=10, beta_slow=0.0),
                                dict(dim=64, factor=2.0, original_length=10, beta_fast=1.0, beta_slow=2.0)])
def test_rope_frequencies_refuses(kw):
    with pytest.raises(B.Ds4hcError):
        B.ds4hc_rope_frequencies(**kw)
