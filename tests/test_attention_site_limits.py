"""Limits of the attention-site entry points that products of sizes meet; needs no GPU."""
import ctypes

import pytest

from test_attention_site_abi import HIP, UNSUP, append, attn, no_gpu_only, paged, prefill


@no_gpu_only
@pytest.mark.parametrize("call,kw,want", [
    # 2^30 rows are taken: 2^40 bytes of output end where the next fake range starts
    (attn, dict(N=1 << 20, heads=1024, ls=(0, 0), rs=(0, 0), os=(1024 * 512, 512), lse=None), HIP),
    (attn, dict(N=(1 << 20) + 1, heads=1024), UNSUP),
    (prefill, dict(N=(1 << 20) + 1, heads=1024), UNSUP),
    (prefill, dict(N=1 << 24, heads=65), UNSUP),
])
def test_rows_of_a_call(call, kw, want):
    assert call(**kw) == want


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(n_pages=(1 << 25) - 1), HIP), (dict(n_pages=1 << 25), UNSUP), (dict(page_size=1, n_pages=(1 << 31) - 1), HIP),
    (dict(page_size=1, max_pages=1 << 30), HIP), (dict(page_size=2, max_pages=1 << 30), UNSUP),
    (dict(page_size=65536, n_pages=32767, max_pages=16384), HIP), (dict(page_size=65536, n_pages=32768), UNSUP),
])
def test_tokens_of_a_cache(kw, want):
    far = dict(cache=ctypes.c_void_p(1 << 52))  # behind all the other ranges
    c = paged(cu_q=1 << 50, kv_len=(1 << 50) + (1 << 40), block_table=1 << 51, **kw)
    assert append(c, **far) == want and attn(c, **far) == want
