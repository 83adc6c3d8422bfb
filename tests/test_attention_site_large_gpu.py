"""The attention-site operators where their work is split otherwise than for a handful of
rows: many sequences, many heads, batches that several workgroups share."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from site_testlib import Batch, assert_attention, attend64, random_tree

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def say(what):
    print(what, flush=True)


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def sums(v):
    return [0] + torch.tensor(v).cumsum(0).tolist()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,q_len,k_len", [
    (64, [769], [769]),                       # just more than 49152 rows and heads: 128 rows a workgroup
    (64, [768], [768]),                       # and the most of which 64 rows are taken
    (96, [129, 0, 300, 1, 90], [200, 3, 300, 65, 20]),  # rows before the first key, and none
    (8, [40] * 150 + [200], [50] * 150 + [200]),        # more than 64 sequences
    (640, [100], [131]),
])
def test_prefill_of_many_rows(dtype, causal, heads, q_len, k_len):
    say(f"[gpu] prefill {dtype} causal={causal} heads={heads} {len(q_len)} sequences, {sum(q_len)} tokens")
    g = torch.Generator().manual_seed(heads + len(q_len))
    cu_q, cu_k = sums(q_len), sums(k_len)
    N, S = cu_q[-1] + 2, cu_k[-1] + 3
    q, kv = torch.randn(N, heads, 192, generator=g).to(dtype), torch.randn(S, heads, 256, generator=g).to(dtype)
    kr = torch.randn(S, 64, generator=g).to(dtype)
    kv[cu_k[-1]:], kr[cu_k[-1]:] = float("nan"), float("nan")  # behind the last sequence
    out = torch.full((N, heads, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((N, heads), 7.0, device="cuda")
    B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), kr.cuda(), i32(cu_q), i32(cu_k), scale=0.08, causal=causal, out=out, lse=lse)
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()
    out, lse = out.cpu(), lse.cpu()
    last = len(q_len) - 1
    for b in sorted({0, last // 2, last - 1, last} & set(range(last + 1))):
        few, many = q_len[b], k_len[b]
        seen = torch.ones(few, many, dtype=torch.bool)
        if causal:
            seen = seen.tril(many - few)
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in (0, heads // 3, heads - 1):
            ref = attend64(q[qs, h], torch.cat((kv[ks, h, :128], kr[ks]), -1), kv[ks, h, 128:], seen, 0.08)
            assert_attention(out[qs, h], lse[qs, h], ref, seen.sum(-1), dtype, f"sequence {b} head {h}")
    assert torch.isfinite(out[:-2].float()).all()


@pytest.mark.parametrize("heads", [2, 400])  # 64 and 128 rows a workgroup
def test_prefill_values_that_are_not_finite(heads):
    """They reach the rows that see them and no others, wherever in a tile and on whichever
    wave's keys they lie, the last token (which stands in for what lies behind it) among them."""
    g = torch.Generator().manual_seed(79)
    n = 150
    q, kv, kr = (torch.randn(*s, generator=g).to(BF) for s in ((n, heads, 192), (n, heads, 256), (n, 64)))
    cu = i32([0, n])
    clean, clean_lse = B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), kr.cuda(), cu, cu, scale=0.08, want_lse=True)
    for at in (0, 31, 32, 63, 64, 97, 149):
        for value in (math.nan, math.inf):
            bad = kv.clone()
            bad[at, 1, 255] = value
            out, lse = B.ds4hc_latent_prefill(q.cuda(), bad.cuda(), kr.cuda(), cu, cu, scale=0.08, want_lse=True)
            say(f"[gpu] {heads} heads, {value} at {at}")
            assert torch.equal(out[:at], clean[:at]) and torch.equal(lse[:at], clean_lse[:at])
            assert torch.equal(out[:, 0], clean[:, 0])
            assert not torch.isfinite(out[at:, 1, 127].float()).any()
