"""Refusals of the entry points over a cache of 8-bit latents and around the attention of drafted tokens:
everything that needs no GPU. Rejected calls enqueue nothing; the fake device addresses are never
dereferenced, so these run only where no GPU is visible."""
import ctypes
import math
import os
import re

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


def append8(c=None, N=8, src=B.DS4HC_BF16, kv=fake(0), stride=576, w=fake(1), eps=1e-6, pos=fake(2), f=fake(3),
            amp=1.0, flags=0, cache=fake(4)):
    return B.ds4hc_latent_append8_raw(c or paged(), N, src, kv, stride, w, eps, pos, f, amp, flags, cache, None)


def attn8(c=None, N=8, heads=16, scale=0.1, ql=fake(0), ls=(16 * 512, 512), qr=fake(1), rs=(1024, 64), cache=fake(4),
          tree=None, words=0, out=fake(5), os=(16 * 512, 512), lse=fake(6), ws=fake(7), ws_bytes=1 << 36):
    return B.ds4hc_latent_attn8_raw(c or paged(), N, heads, scale, ql, ls, qr, rs, cache, tree, words, out, os, lse,
                                    ws, ws_bytes, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), BAD), (dict(d_latent=0), BAD), (dict(page_size=48), BAD), (dict(n_pages=0), BAD), (dict(n_seqs=-1), BAD),
    (dict(dtype=B.DS4HC_F32), UNSUP), (dict(d_latent=384), UNSUP), (dict(d_rope=32), UNSUP), (dict(page_size=1 << 17), UNSUP),
    (dict(n_pages=1 << 31), UNSUP), (dict(cu_q=None), BAD), (dict(block_table=addr(22, 1)), BAD),
    (dict(n_seqs=0, cu_q=None, kv_len=None, block_table=None), OK), (dict(dtype=B.DS4HC_F16), HIP), (dict(), HIP),
])
def test_cache_descriptor(kw, want):
    assert append8(paged(**kw)) == want
    assert attn8(paged(**kw)) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(N=-1), BAD), (dict(src=4), BAD), (dict(eps=-1.0), BAD), (dict(flags=2), BAD), (dict(amp=math.nan), BAD),
    (dict(stride=575), BAD), (dict(stride=577), BAD), (dict(kv=None), BAD), (dict(cache=None), BAD), (dict(w=None), HIP),
    (dict(cache=fake(4, 8)), BAD), (dict(cache=fake(0)), BAD),
    (dict(cache=fake(20, -100 * 64 * 656)), HIP), (dict(cache=fake(20, -100 * 64 * 656 + 16)), BAD),  # up to cu_q, and into it
    (dict(N=0, kv=None, pos=None, f=None, cache=None), OK),
])
def test_append8_arguments(kw, want):
    assert append8(**kw) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(N=-1), BAD), (dict(heads=0), BAD), (dict(heads=1025), UNSUP), (dict(scale=0.0), BAD),
    (dict(scale=math.nan), BAD), (dict(ls=(8192, 516)), BAD), (dict(os=(8192, 511)), BAD), (dict(os=(512, 8 * 512)), HIP),
    (dict(cache=None), BAD), (dict(cache=fake(4, 8)), BAD), (dict(out=fake(4, 100 * 64 * 656 - 16)), BAD),
    (dict(out=fake(4, 100 * 64 * 656)), HIP), (dict(tree=fake(8), words=0), BAD), (dict(ws=None), BAD), (dict(ws_bytes=100), BAD),
    (dict(N=0, ql=None, qr=None, cache=None, out=None, ws=None), OK),
])
def test_attn8_arguments(kw, want):
    assert attn8(**kw) == want


def test_attn8_workspace():
    c = paged()
    need = B.ds4hc_latent_attn8_workspace_bytes(c, 8, 16)
    assert need > 0
    assert B.ds4hc_latent_attn8_workspace_bytes(paged(cu_q=None, kv_len=None, block_table=None), 8, 16) == need
    for kw in (dict(d_latent=100), dict(page_size=3), dict(n_seqs=0)):
        assert B.ds4hc_latent_attn8_workspace_bytes(paged(**kw), 8, 16) == 0
    assert B.ds4hc_latent_attn8_workspace_bytes(c, 0, 16) == 0 and B.ds4hc_latent_attn8_workspace_bytes(c, 8, 0) == 0


# ------------------------------------------------------------------ verification

def verify(N=8, seqs=2, vocab=100, target=fake(0), ts=100, draft=None, ds=0, tokens=fake(2), parents=None, cu=fake(4),
           u=fake(5), path=fake(6), kept=fake(7), nxt=fake(8), ws=fake(9), ws_bytes=1 << 30):
    return B.ds4hc_draft_verify_raw(N, seqs, vocab, target, ts, draft, ds, tokens, parents, cu, u, path, kept, nxt, ws,
                                    ws_bytes, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(draft=fake(1), ds=100), HIP), (dict(parents=fake(3)), HIP),
    (dict(draft=fake(1), ds=100, parents=fake(3)), BAD), (dict(N=-1), BAD), (dict(seqs=-1), BAD), (dict(vocab=0), BAD),
    (dict(ts=99), BAD), (dict(ts=101), HIP), (dict(draft=fake(1), ds=99), BAD), (dict(ts=1 << 40), BAD),
    (dict(N=(1 << 24) + 1), UNSUP), (dict(seqs=65536), UNSUP), (dict(vocab=(1 << 24) + 1, ts=1 << 25), UNSUP),
    (dict(seqs=0), OK), (dict(seqs=0, cu=None, kept=None, nxt=None, ws=None), OK),
    (dict(N=0, target=None, tokens=None, u=None, path=None), HIP),
    (dict(target=None), BAD), (dict(tokens=None), BAD), (dict(cu=None), BAD), (dict(u=None), BAD), (dict(path=None), BAD),
    (dict(kept=None), BAD), (dict(nxt=None), BAD), (dict(ws=None), BAD), (dict(ws_bytes=0), BAD), (dict(ws=fake(9, 8)), BAD),
    (dict(target=fake(0, 2)), BAD), (dict(target=fake(0, 4)), HIP), (dict(tokens=fake(2, 4)), BAD), (dict(nxt=fake(8, 4)), BAD),
    (dict(parents=fake(3, 2)), BAD), (dict(path=fake(6, 1)), BAD), (dict(path=fake(0, 8 * 400 - 4)), BAD),
    (dict(path=fake(0, 8 * 400)), HIP), (dict(kept=fake(6, 28)), BAD), (dict(nxt=fake(2)), BAD), (dict(ws=fake(7)), BAD),
    (dict(path=fake(4, 8)), BAD), (dict(ws=fake(5, 16)), BAD),
])
def test_verify_arguments(kw, want):
    assert verify(**kw) == want


@no_gpu_only
def test_verify_workspace():
    need = B.ds4hc_draft_verify_workspace_bytes(2, 100)
    assert need > 0 and verify(ws_bytes=need) == HIP and verify(ws_bytes=need - 1) == BAD
    for a in ((0, 100), (2, 0), (65536, 100), (2, (1 << 24) + 1), (-1, 5)):
        assert B.ds4hc_draft_verify_workspace_bytes(*a) == 0
    assert B.ds4hc_draft_verify_workspace_bytes(65535, 1 << 24) > 0


# ------------------------------------------------------------------ moves

def store(**over):
    a = dict(layers=3, page_size=16, n_pages=10, row_bytes=656, layer_stride=16 * 10 * 656, data=addr(0))
    a.update(over)
    return B.PageStore(*[a[f] for f, _ in B.PageStore._fields_])


def compact(s=None, N=8, seqs=2, most=4, cu=fake(1), lens=fake(2), table=fake(3), keep=fake(4), n_keep=fake(5)):
    return B.ds4hc_cache_compact_raw(s or store(), N, seqs, most, cu, lens, table, keep, n_keep, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(layers=0), BAD), (dict(page_size=12), BAD), (dict(page_size=0), BAD), (dict(n_pages=0), BAD),
    (dict(row_bytes=0), BAD), (dict(row_bytes=24), BAD), (dict(layer_stride=16 * 10 * 656 - 16), BAD),
    (dict(layer_stride=16 * 10 * 656 + 8), BAD), (dict(layer_stride=16 * 10 * 656 + 16), HIP), (dict(layers=1, layer_stride=-5), HIP),
    (dict(layers=65536), UNSUP), (dict(page_size=1 << 17), UNSUP), (dict(n_pages=1 << 28), UNSUP), (dict(row_bytes=65552), UNSUP),
    (dict(layer_stride=1 << 50), UNSUP), (dict(data=None), BAD), (dict(data=addr(0, 8)), BAD),
])
def test_store_descriptor(kw, want):
    assert compact(store(**kw)) == want
    assert B.ds4hc_pages_copy_raw(store(**kw), 5, fake(1), None) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(seqs=-1), BAD), (dict(most=0), BAD), (dict(N=(1 << 24) + 1), UNSUP), (dict(seqs=65536), UNSUP),
    (dict(most=1 << 27), UNSUP), (dict(N=0), OK), (dict(seqs=0), OK), (dict(cu=None), BAD), (dict(lens=None), BAD),
    (dict(table=None), BAD), (dict(keep=None), BAD), (dict(n_keep=None), BAD), (dict(keep=fake(4, 2)), BAD),
    (dict(cu=fake(0, 64)), BAD), (dict(keep=fake(0, 3 * 16 * 10 * 656 - 4)), BAD), (dict(keep=fake(0, 3 * 16 * 10 * 656)), HIP),
])
def test_compact_arguments(kw, want):
    assert compact(**kw) == want


@no_gpu_only
def test_pages_copy_arguments():
    s = store()
    for n, pairs, want in ((0, None, OK), (-1, fake(1), BAD), ((1 << 20) + 1, fake(1), UNSUP), (3, None, BAD),
                           (3, fake(1, 2), BAD), (3, fake(0, 16), BAD), (1 << 20, fake(1), HIP)):
        assert B.ds4hc_pages_copy_raw(s, n, pairs, None) == want


# ------------------------------------------------------------------ pages

def pool(**over):
    a = dict(page_size=16, n_slots=6, max_pages=4, n_pages=50, block_table=addr(0), kv_len=addr(1), refs=addr(2))
    a.update(over)
    return B.PagePool(*[a[f] for f, _ in B.PagePool._fields_])


def resize(p=None, n=3, slots=fake(3), lens=fake(4), copies=fake(5), status=fake(6), ws=fake(7), ws_bytes=1 << 30):
    return B.ds4hc_pages_resize_raw(p or pool(), n, slots, lens, copies, status, ws, ws_bytes, None)


def fork(p=None, n=3, parents=fake(3), children=fake(4), status=fake(6), ws=fake(7), ws_bytes=1 << 30):
    return B.ds4hc_pages_fork_raw(p or pool(), n, parents, children, status, ws, ws_bytes, None)


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(), HIP), (dict(page_size=0), BAD), (dict(page_size=24), BAD), (dict(n_slots=0), BAD), (dict(max_pages=0), BAD),
    (dict(n_pages=0), BAD), (dict(page_size=1 << 17), UNSUP), (dict(n_slots=(1 << 20) + 1), UNSUP),
    (dict(max_pages=1 << 27), UNSUP), (dict(n_pages=(1 << 28) + 1), UNSUP), (dict(block_table=None), BAD), (dict(kv_len=None), BAD),
    (dict(refs=None), BAD), (dict(refs=addr(2, 2)), BAD), (dict(kv_len=addr(0, 92)), BAD), (dict(kv_len=addr(0, 96)), HIP),
    (dict(refs=addr(4)), BAD),
])
def test_pool_descriptor(kw, want):
    assert resize(pool(**kw)) == want
    assert fork(pool(**kw)) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(n=0, status=None, ws=None), OK), (dict(n=-1), BAD), (dict(n=(1 << 20) + 1), UNSUP), (dict(status=None), BAD),
    (dict(ws=None), BAD), (dict(ws_bytes=8), BAD), (dict(ws=fake(7, 4)), BAD), (dict(status=fake(6, 2)), BAD),
    (dict(status=fake(3)), BAD), (dict(ws=fake(0)), BAD),
])
def test_items(kw, want):
    assert resize(**kw) == want
    assert fork(**kw) == want
    need = B.ds4hc_pages_workspace_bytes(pool(), 3)
    assert need > 0 and resize(ws_bytes=need) == HIP and resize(ws_bytes=need - 1) == BAD and fork(ws_bytes=need - 1) == BAD
    assert resize(slots=None) == BAD and resize(lens=None) == BAD and resize(copies=None) == BAD
    assert resize(copies=fake(4)) == BAD and resize(copies=fake(6, -16)) == BAD and resize(lens=fake(4, 1)) == BAD
    assert fork(parents=None) == BAD and fork(children=None) == BAD and fork(children=fake(1, 4)) == BAD
    for a in ((pool(page_size=3), 3), (pool(), 0), (pool(), -1), (pool(), 1 << 21)):
        assert B.ds4hc_pages_workspace_bytes(*a) == 0
    assert B.ds4hc_pages_workspace_bytes(pool(block_table=None, kv_len=None, refs=None), 3) == need


def test_binding_refuses_host_tensors():
    t, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    calls = [lambda: B.ds4hc_latent_append8(t, t, t, t, t, t, t), lambda: B.ds4hc_latent_attn8(t, t, t, t, t, t, scale=1.0),
             lambda: B.ds4hc_draft_verify(torch.zeros(3, 5), i, i, i), lambda: B.ds4hc_cache_compact(t, i, i, i, i, i),
             lambda: B.ds4hc_pages_copy(t, i), lambda: B.ds4hc_pages_resize(i, i, i, 16, i, i),
             lambda: B.ds4hc_pages_fork(i, i, i, 16, i, i)]
    for call in calls:
        with pytest.raises(ValueError, match="device tensor"):
            call()


@pytest.mark.parametrize("name", ["VERIFY_MAX_TOKENS", "PAGES_DONE", "PAGES_SHORT", "PAGES_INVALID"])
def test_binding_has_the_headers_numbers(name):
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ds4hc.h")
    with open(header) as f:
        said = re.search(rf"#define DS4HC_{name} (\d+)\b", f.read())
    assert int(said.group(1)) == getattr(B, "DS4HC_" + name)
