"""The attention-site operators at the edges of what their documentation allows."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from site_testlib import Batch, assert_attention, random_tree

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


# ------------------------------------------------------------------ tiles without a token

def no_sequence_has_page_0(bt, value):
    """Page 0 is nobody's, and all of it holds `value`."""
    spare = (set(range(1, bt.n_pages)) - set(bt.table.flatten().tolist())).pop()
    if (bt.table == 0).any():
        bt.cache[spare] = bt.cache[0]
        bt.table[bt.table == 0] = spare
    bt.cache[0] = value


def check_holes(bt, heads, holes, tree, tokens=None):
    ql, qr = bt.queries(heads)
    table = bt.table.clone()
    for b, p in holes:
        table[b, p] = -1
    out, lse = B.ds4hc_latent_attn(ql.cuda(), qr.cuda(), bt.cache.cuda(), bt.cu.cuda(), bt.lens.cuda(), table.cuda(),
                                   scale=0.07, tree_mask=None if tree is None else tree.cuda(), want_lse=True)
    out, lse = out.cpu(), lse.cpu()
    for t, (ref, n) in enumerate(bt.reference(ql, qr, 0.07, tree, holes)):
        if tokens is None or t in tokens:
            assert_attention(out[t], lse[t], ref, n, bt.dtype, f"token {t}")


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len", [
    (6, 512, 64, [3, 2], [640, 330]), (6, 128, 16, [3, 2], [330, 200]), (16, 256, 128, [2, 2], [640, 300]),  # 32 rows
    (16, 512, 64, [3, 3], [330, 200]), (20, 256, 16, [3, 2], [200, 330]),                                   # 64 rows
    (40, 512, 64, [3, 4], [520, 200]), (64, 128, 16, [4, 4], [330, 140])])                                  # 128 rows
def test_attn_tiles_without_a_token(value, tree, heads, latent, page, q_len, kv_len):
    """Of 64 tokens in a row none is in the cache, at the context's begin, in its middle, at its
    end, where the call's own tokens begin, and all together: they change nothing, whatever the
    cache's first row holds."""
    say(f"[gpu] holes {value} tree={tree} heads={heads} latent={latent} page={page}")
    for dtype in (BF, HF):
        bt = Batch(201 + heads, q_len, kv_len, page, latent, dtype)
        no_sequence_has_page_0(bt, value)
        mask = random_tree(bt.g, q_len, 1) if tree else None
        tile = lambda b, t: [(b, p) for p in range(t * 64 // page, max((t * 64 + 63) // page, t * 64 // page) + 1)  # noqa: E731
                             if p < -(-kv_len[b] // page)]
        border = (kv_len[0] - q_len[0]) // 64
        places = [tile(0, 0), tile(0, 2), tile(0, border - 1), tile(0, border), tile(1, 1)]
        for holes in places + [sum(places, [])]:
            check_holes(bt, heads, sorted(set(holes)), mask)


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_attn_tiles_without_a_token_in_sequences_of_one_workgroup(heads):
    """Many sequences, so that most are not cut, and one whose holes lie in several parts."""
    q_len, kv_len = [1] * 300, [190 + i % 40 for i in range(299)] + [6000]
    bt = Batch(211, q_len, kv_len, 64, 128, BF)
    no_sequence_has_page_0(bt, math.nan)
    check_holes(bt, heads, [(b, b % 3) for b in range(0, 299, 2)] + [(299, p) for p in (0, 7, 8, 50, 93)], None)
