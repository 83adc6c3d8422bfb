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


def check_tokens(bt, ql, qr, scale, out, lse, tokens, tree=None):
    """Tokens (b, i) of a batch against the 64-bit form."""
    flat, heads = bt.cache.view(-1, bt.latent + 64), ql.shape[1]
    for b, i in tokens:
        q, k, t = bt.q_len[b], bt.kv_len[b], int(bt.cu[b]) + i
        seen = torch.arange(k) <= k - q + i
        if tree is not None:
            seen[max(k - q, 0):] = torch.tensor([(int(tree[t, d // 64]) >> d % 64) & 1 for d in range(max(q - k, 0), q)], dtype=torch.bool)
        keys = flat[bt.rows(b, k)]
        ref = attend64(torch.cat((ql[t], qr[t]), -1), keys, keys[:, :bt.latent], seen.expand(heads, k), scale)
        assert_attention(out[t].cpu(), lse[t].cpu(), ref, [int(seen.sum())] * heads, ql.dtype, f"sequence {b} token {i}")


def run_attn(bt, ql, qr, scale=0.07, tree=None, **kw):
    tree = None if tree is None else tree.cuda()
    return B.ds4hc_latent_attn(ql.cuda(), qr.cuda(), bt.cache.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda(),
                               scale=scale, tree_mask=tree, want_lse=True, **kw)


@pytest.mark.parametrize("n_seqs,heads,latent,page,most", [
    (65, 16, 512, 16, 200), (150, 3, 128, 4, 120), (300, 128, 256, 64, 150), (700, 1, 512, 2, 40), (64, 40, 512, 32, 700)])
def test_attn_of_many_sequences(n_seqs, heads, latent, page, most):
    """No tokens, or no cached ones, among them."""
    say(f"[gpu] attn {n_seqs} sequences, {heads} heads, latent {latent}, page {page}")
    g = torch.Generator().manual_seed(n_seqs)
    q_len = torch.randint(0, 3, (n_seqs,), generator=g).tolist()
    kv_len = [max(int(k), q) if k % 7 else 0 for k, q in zip(torch.randint(0, most, (n_seqs,), generator=g), q_len)]
    bt = Batch(n_seqs, q_len, kv_len, page, latent, BF, extra_tokens=2)
    ql, qr = bt.queries(heads)
    out = torch.full((bt.N, heads, latent), 7.0, dtype=BF, device="cuda")
    lse = torch.full((bt.N, heads), 7.0, device="cuda")
    run_attn(bt, ql, qr, out=out, lse=lse)
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()
    check_tokens(bt, ql, qr, 0.07, out, lse, [(b, i) for b in range(n_seqs) for i in range(q_len[b])])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len,tree", [
    (128, 512, 64, [3, 1, 4], [2900, 700, 3100], False),  # 8 row tiles in groups of four
    (128, 512, 16, [2, 1, 2, 1], [1300, 5000, 64, 2], False),  # in pairs
    (100, 256, 64, [2, 5], [2600, 900], False), (77, 128, 8, [4, 4, 4], [1900, 333, 4], False),
    (16, 512, 16, [40, 33, 2], [4000, 1500, 600], True), (24, 256, 64, [64, 17], [1000, 2100], True),
    (128, 512, 64, [1], [20000], False), (8, 128, 1, [1, 2], [1500, 40], False), (40, 256, 2, [1], [3300], False)])
def test_attn_cut_into_parts(dtype, heads, latent, page, q_len, kv_len, tree):
    say(f"[gpu] attn {dtype} heads={heads} latent={latent} page={page} q={q_len} kv={kv_len} tree={tree}")
    bt = Batch(heads + latent, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    mask = random_tree(bt.g, q_len, 1) if tree else None
    out, lse = run_attn(bt, ql, qr, tree=mask)
    check_tokens(bt, ql, qr, 0.07, out, lse, [(b, i) for b in range(len(q_len)) for i in range(q_len[b])], mask)
    again, lse_again = run_attn(bt, ql, qr, tree=mask)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


def test_attn_on_two_streams_at_once():
    """Two calls that run beside each other, each with a workspace of its own."""
    bts = [Batch(91, [1, 2, 1], [3000, 900, 40], 64, 512), Batch(93, [4], [2500], 16, 512)]
    calls = []
    for bt in bts:
        ql, qr = bt.queries(64)
        args = [t.cuda() for t in (ql, qr, bt.cache, bt.cu, bt.lens, bt.table)]
        want = B.ds4hc_latent_attn(*args, scale=0.07, want_lse=True)
        need = B.ds4hc_latent_attn_workspace_bytes(B._paged(*args[2:]), bt.N, 64)
        calls.append((args, want, torch.empty_like(want[0]), torch.empty_like(want[1]),
                      torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, _, out, lse, ws, stream in calls:
            B.ds4hc_latent_attn(*args, scale=0.07, out=out, lse=lse, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for _, want, out, lse, _, _ in calls:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("n_seqs", [64, 65, 500])
def test_append_to_many_sequences(n_seqs):
    g = torch.Generator().manual_seed(n_seqs)
    q_len = torch.randint(0, 4, (n_seqs,), generator=g).tolist()
    kv_len = [q + int(k) for q, k in zip(q_len, torch.randint(0, 30, (n_seqs,), generator=g))]
    bt = Batch(n_seqs, q_len, kv_len, 4, 128, HF, extra_tokens=3)
    kv = torch.randn(bt.N, 192, generator=g).to(HF)
    positions = torch.zeros(bt.N, dtype=torch.int64)  # no rotation: what is stored is what was given
    before, cache = bt.cache.clone().view(-1, 192), bt.cache.cuda()
    f = B.ds4hc_rope_frequencies(64)[0]
    B.ds4hc_latent_append(kv.cuda(), positions.cuda(), f.cuda(), cache, bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda())
    for b, (q, k) in enumerate(zip(q_len, kv_len)):
        before[bt.rows(b, k)[k - q:]] = kv[bt.cu[b]:bt.cu[b] + q]
    assert torch.equal(cache.cpu().view(-1, 192).view(torch.int16), before.view(torch.int16))


def test_rope_of_the_most_tokens():
    """2^24 tokens: more threads than one dimension of a dispatch takes."""
    n, f = 1 << 24, torch.tensor([0.25], dtype=torch.float64, device="cuda")
    x = torch.ones(n, 1, 2, device="cuda")
    positions = torch.arange(n, device="cuda")
    y = B.ds4hc_rope(x, positions, f)
    a = positions.double() * 0.25
    want = torch.stack((a.cos() - a.sin(), a.sin() + a.cos()), -1)
    # a part of a turn of at most half a turn in float32 (4 e in cos and sin of it), two products and a sum
    assert ((y[:, 0].double() - want).abs() <= 2 * 16 * 2.0 ** -24 + a.abs()[:, None] * 2.0 ** -50).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [3, 600])
def test_weights_sum_to_one_as_they_were_rounded(dtype, heads):
    """A row that sees one token gives its values to the last bit: w v / w in float32 is
    within 2 e of v, which no rounding to 16 bits sees. n equal weights, rounded alike,
    leave the mean of the values: (n + 64) e of their sizes for the sums, u for the store."""
    g = torch.Generator().manual_seed(97)
    n = 90
    q, kv, kr = (torch.randn(*s, generator=g).to(dtype) for s in ((n, heads, 192), (n, heads, 256), (n, 64)))
    out = B.ds4hc_latent_prefill(q[:1].cuda(), kv[:1].cuda(), kr[:1].cuda(), i32([0, 1]), i32([0, 1]), scale=0.0837)[0]
    assert torch.equal(out[0].cpu(), kv[0, :, 128:])
    kv[:, :, :128], kr[:] = kv[:1, :, :128].clone(), kr[:1].clone()
    out = B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), kr.cuda(), i32([0, n]), i32([0, n]), scale=0.0837)[0].cpu()
    for h in (0, 1, heads - 1):
        v = kv[:, h, 128:].double()
        many = torch.arange(1, n + 1).double()[:, None]
        want, size = v.cumsum(0) / many, v.abs().cumsum(0) / many
        assert ((out[:, h].double() - want).abs() <= 3 * (n + 64) * 2.0 ** -24 * size + torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent", [(16, 512), (128, 512), (40, 256), (3, 128)])
def test_attn_of_one_token(dtype, heads, latent):
    bt = Batch(101, [1, 1, 1], [1, 1, 1], 16, latent, dtype)
    ql, qr = bt.queries(heads)
    out, _ = run_attn(bt, ql, qr)
    flat = bt.cache.view(-1, latent + 64)
    for b in range(3):
        assert torch.equal(out[b].cpu(), flat[bt.rows(b, 1)][:, :latent].expand(heads, latent))


def test_attn_tree_of_more_tokens_than_the_cache_has():
    """q_len > kv_len: the call's first tokens have no place; bits d of a mask still count the
    call's tokens."""
    bt = Batch(103, [70, 5, 3], [30, 2, 0], 16, 512)
    ql, qr = bt.queries(16)
    mask = random_tree(bt.g, bt.q_len, 2)
    out, lse = run_attn(bt, ql, qr, tree=mask)
    check_tokens(bt, ql, qr, 0.07, out, lse, [(b, i) for b in range(3) for i in range(bt.q_len[b])], mask)


@pytest.mark.parametrize("heads", [16, 128])
def test_attn_of_sequences_that_share_pages(heads):
    """Two samples of one prompt: their tables name the same pages, up to the last, which is each
    one's own; the second sequence names one page twice."""
    bt = Batch(107, [1, 2, 1], [700, 690, 300], 64, 512)
    bt.table[1, :10] = bt.table[0, :10]
    bt.table[2, 3] = bt.table[2, 1]
    flat = bt.cache.view(-1, 576)
    assert torch.isfinite(flat[bt.rows(1, 690)].float()).all()
    ql, qr = bt.queries(heads)
    out, lse = run_attn(bt, ql, qr)
    check_tokens(bt, ql, qr, 0.07, out, lse, [(0, 0), (1, 0), (1, 1), (2, 0)])
