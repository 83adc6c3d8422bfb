"""The operators over a cache of 8-bit latents on the GPU against 64-bit references (bounds derived in
site_testlib), at the sizes, masks, scales and layouts where they can go wrong."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from serve_testlib import Batch8, to_rows8, values8
from site_testlib import assert_attention, random_tree, rope_bound, turn64, u_of

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ append

def check_rows8(rows, latent, slack):
    """Rows of bytes against the latents [n, d] in 64 bits that float32 arithmetic gives to within `slack`: the scale
    is the smallest that fits the largest magnitude, the values are off by at most half a step of e4m3 (2^-4 of the
    value, 2^-10 scales below the normal numbers) more."""
    d = latent.shape[1]
    got, _ = values8(rows, BF)
    top, loose = latent.abs().amax(-1), slack.amax(-1)
    scale = torch.exp2(rows[:, d + 128].double() - 127)
    assert ((top - loose) <= 448 * scale).all() or (rows[:, d + 128] == 246).any()
    low = (top + loose) > 224 * scale
    assert (low | (rows[:, d + 128] == 10)).all()
    bound = slack * (1 + 2.0 ** -4) + torch.maximum(latent.abs() * 2.0 ** -4, scale[:, None] * 2.0 ** -10)
    assert ((got - latent).abs() <= bound).all()
    assert (rows[:, d + 129:] == 0).all()


@pytest.mark.parametrize("src", [F32, BF, HF])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("latent,page,q_len,kv_len,norm,interleaved",
                         [(512, 64, [1, 1, 1], [1, 64, 65], True, True), (128, 1, [3, 0, 5], [3, 7, 9], True, False),
                          (256, 16, [40, 2], [40, 500], False, True), (512, 128, [1], [300], True, False)])
def test_append8(src, dtype, latent, page, q_len, kv_len, norm, interleaved):
    say(f"[gpu] append8 {src}->{dtype} latent={latent} page={page} q={q_len} kv={kv_len}")
    bt = Batch8(5, q_len, kv_len, page, latent, dtype, extra_tokens=2)
    wide = torch.randn(bt.N, latent + 64 + 40, generator=bt.g).to(src)
    kv = wide[:, 24:24 + latent + 64]
    w = 1 + 0.3 * torch.randn(latent, generator=bt.g) if norm else None
    f, _ = B.ds4hc_rope_frequencies(64)
    positions = torch.randint(0, 200000, (bt.N,), generator=bt.g)
    cache = bt.rows8.cuda()
    got = B.ds4hc_latent_append8(wide.cuda()[:, 24:24 + latent + 64], positions.cuda(), f.cuda(), cache, bt.cu.cuda(),
                                 bt.lens.cuda(), bt.table.cuda(), dtype=dtype, norm_weight=None if w is None else w.cuda(),
                                 rms_eps=1e-5, interleaved=interleaved, amplitude=1.5)
    assert got is cache
    c = kv[:, :latent].double()
    if norm:
        c = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w.double()
    slack = c.abs() * ((latent / 2 + 8) * 2.0 ** -24 if norm else 0)  # as for the append to 16 bits
    r = turn64(kv[:, latent:], positions, f, 1.5, interleaved)
    part, _ = rope_bound(kv[:, latent:], positions, f, 1.5, interleaved, dtype)
    u = u_of(dtype)
    flat, old = cache.cpu().view(-1, latent + 144), bt.rows8.view(-1, latent + 144)
    touched = torch.zeros(len(flat), dtype=torch.bool)
    for b, (q, k) in enumerate(zip(q_len, kv_len)):
        if not q:
            continue
        rows, here = bt.rows(b, k)[k - q:], slice(int(bt.cu[b]), int(bt.cu[b]) + q)
        touched[rows] = True
        check_rows8(flat[rows], c[here], slack[here])
        _, rope = values8(flat[rows], dtype)
        bound = part[here] * (1 + u) + u * r[here].abs() + (6e-8 if dtype == HF else 1e-38)
        assert ((rope - r[here]).abs() <= bound).all()
    assert torch.equal(flat[~touched], old[~touched])


def append_rows(x, **kw):
    """Rows [n, latent + 64] appended without a norm to a cache of one page."""
    n, d = x.shape[0], x.shape[1] - 64
    cache = torch.full((1, 64, d + 144), 77, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B.ds4hc_latent_append8(x.cuda(), torch.zeros(n, dtype=torch.int64, device="cuda"),
                           B.ds4hc_rope_frequencies(64)[0].cuda(), cache, i32([0, n]), i32([n]), i32([[0]]), **kw)
    return cache.cpu()[0, :n]


def test_append8_scales_and_ties():
    """Largest magnitudes at and around the borders of the scale, every tie of e4m3, zero, the smallest and the largest
    rows, values that are not finite: the same bytes as from the definition. (No norm: nothing is computed.)"""
    d = 128
    x = torch.zeros(40, d + 64)
    tops = [448.0, 448.00003, 224.0, 224.00002, 1.0, 1.75, 1.7500001, 1.7499999, 0.0, 3e38, 3.4e38, 1e-30, 2.0 ** -109,
            2.0 ** -126, 1e-44, 2.0 ** 127, -448.0, -3.5, 2.0 ** -110, 1.9921875]
    for i, t in enumerate(tops):
        x[i, 5] = t
        x[i, 6:40] = torch.linspace(-1, 1, 34) * abs(t)
    ties = torch.arange(0, 255).float() / 256  # between neighbours 1/8 apart in [1, 2), and finer below
    x[20, 0], x[20, 1:101] = 448.0, 1 + ties[:100] * 0.99609375
    x[21, 0], x[21, 1:128] = 448.0, torch.arange(127) * 2.0 ** -11       # multiples of a quarter of the smallest number
    x[22, 0], x[22, 1:60] = 256.0, 16 + torch.arange(59) * 0.5
    x[23, 3], x[24, 3], x[25, 3] = math.nan, math.inf, -math.inf
    x[23:26, 10:20] = 2.0
    got, want = append_rows(x), to_rows8(x[:, :d].double(), x[:, d:].to(BF))
    same = (got == want) | ((got[:, :] & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
    zero = ((got & 0x7F) == 0) & ((want & 0x7F) == 0)  # -0 and 0
    assert (same | zero).all(), ((~(same | zero)).nonzero()[:10], got[~(same | zero)][:10], want[~(same | zero)][:10])
    assert got[8, d + 128] == 10 and (got[8, :d] & 0x7F == 0).all()
    assert (got[23:26, d + 128] == 255).all() and (got[23:26, :d] & 0x7F == 0x7F).all()


def test_append8_passes_over_what_has_no_place():
    """As the append to 16 bits: only the tokens' own places are written."""
    cache = torch.full((6, 4, 656), 9, dtype=torch.uint8, device="cuda")
    kv = torch.ones(12, 576, dtype=BF, device="cuda")
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    pos = torch.zeros(12, dtype=torch.int64, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B.ds4hc_latent_append8(kv, pos, f, cache, i32([0, 3, 6, 9]), i32([1, 7, 1000]), i32([[0, -1], [1, 99], [2, 3]]))
    rows = set((cache.view(-1, 656) != 9).any(-1).nonzero()[:, 0].tolist())
    assert rows == {0, 13, 14, 15}


# ------------------------------------------------------------------ attention

def run_attn8(bt, ql, qr, scale, tree=None, lens=None, table=None, **kw):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    return B.ds4hc_latent_attn8(d(ql), d(qr), d(bt.rows8), d(bt.cu), d(bt.lens if lens is None else lens),
                                d(bt.table if table is None else table), scale=scale, tree_mask=d(tree), want_lse=True, **kw)


def check_attn8(bt, ql, qr, scale, out, lse, tree=None, holes=()):
    heads = ql.shape[1]
    out, lse = out.cpu(), lse.cpu()
    for t, (ref, n) in enumerate(bt.reference(ql, qr, scale, tree, holes)):
        assert_attention(out[t], lse[t], ref, n, bt.dtype, f"token {t} of {bt.N}, heads {heads}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len", [
    (1, 512, 64, [1], [1]), (16, 512, 64, [1], [0]), (16, 512, 64, [1, 1], [500, 0]), (128, 512, 64, [1], [129]),
    (128, 512, 64, [1, 1, 1], [64, 63, 65]), (5, 256, 16, [2, 1], [33, 16]), (17, 128, 1, [1, 3], [40, 5]),
    (128, 512, 64, [1], [5000]), (16, 512, 128, [4, 4], [2000, 777]), (7, 256, 32, [1, 0, 2], [31, 50, 1000]),
    (40, 128, 64, [130], [200]), (130, 512, 16, [2], [300]), (33, 512, 64, [3], [2]), (1, 512, 64, [70], [70]),
    (64, 512, 64, [2, 1, 1, 5], [70, 1, 260, 5]), (8, 512, 2, [1], [37]), (50, 256, 64, [1], [900]),
    (100, 128, 64, [1, 2], [700, 65])])
def test_attn8_causal(dtype, heads, latent, page, q_len, kv_len):
    say(f"[gpu] attn8 {dtype} heads={heads} latent={latent} page={page} q={q_len} kv={kv_len}")
    bt = Batch8(11 + heads, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    out, lse = run_attn8(bt, ql, qr, 0.07)
    check_attn8(bt, ql, qr, 0.07, out, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len,words", [
    (16, 512, 16, [9, 33], [300, 33], 1), (128, 512, 64, [6], [70], 1), (3, 256, 64, [100, 2], [400, 2], 2),
    (16, 128, 32, [64, 65], [64, 200], 2)])
def test_attn8_tree(dtype, heads, latent, page, q_len, kv_len, words):
    say(f"[gpu] attn8 tree {dtype} heads={heads} latent={latent} q={q_len} kv={kv_len}")
    bt = Batch8(23, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    tree = random_tree(bt.g, q_len, words)
    tree[0] = 0  # sees the context alone
    out, lse = run_attn8(bt, ql, qr, 0.07, tree)
    check_attn8(bt, ql, qr, 0.07, out, lse, tree)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_attn8_tokens_of_unlike_sizes(dtype, heads):
    """Scales that differ by up to 2^12 from token to token: each token's weight and values count as they are. Queries are
    small, so that logits stay moderate."""
    bt = Batch8(61, [2, 1], [150, 333], 16, 512, dtype, spread=6)
    ql, qr = bt.queries(heads)
    ql = (ql.float() / 16).to(dtype)
    out, lse = run_attn8(bt, ql, qr, 0.07)
    check_attn8(bt, ql, qr, 0.07, out, lse)


def test_attn8_large_logits_and_one_weight():
    """Logits of +-400: one weight takes all, sums neither overflow nor vanish."""
    for dtype in (BF, HF):
        bt = Batch8(31, [1, 2], [700, 90], 64, 512, dtype)
        ql, qr = bt.queries(16, 4.0)
        out, lse = run_attn8(bt, ql, qr, 1.0)
        check_attn8(bt, ql, qr, 1.0, out, lse)


def test_attn8_small_weights_of_a_long_context():
    """One token holds most of the weight, 20000 others, each far below what a 16-bit number next to 1 can tell from 0, the
    rest: they count."""
    for dtype in (BF, HF):
        bt = Batch8(67, [1], [20000], 64, 128, dtype)
        d = bt.latent
        flat = bt.rows8.view(-1, d + 144)
        at = bt.rows(0, 20000)
        values = torch.zeros(20000, d, dtype=torch.float64)
        values[:, 1] = 1.0            # the others' value
        values[7777, 0], values[7777, 1] = 4.0, 0.0
        flat[at] = to_rows8(values, torch.zeros(20000, 64, dtype=dtype))
        bt.refresh()
        ql, qr = torch.zeros(1, 16, d, dtype=dtype), torch.zeros(1, 16, 64, dtype=dtype)
        ql[..., 0] = 3.0              # a logit of 12 for the one, 0 for the others: weights of 0.89 and 5.5e-6
        out, lse = run_attn8(bt, ql, qr, 1.0)
        check_attn8(bt, ql, qr, 1.0, out, lse)
        assert out[0, 0, 1].item() > 0.1


def test_attn8_holes_and_lengths_beyond_the_table():
    """Pages that are not in the cache are not seen; a length behind the table is cut; a negative one is 0."""
    bt = Batch8(37, [1, 2, 1, 1], [256, 256, 256, 100], 64, 512, max_pages=4)
    ql, qr = bt.queries(16)
    table, lens = bt.table.clone(), bt.lens.clone()
    table[0, 1], table[1, 0], table[1, 3], table[2] = -1, bt.n_pages, -5, 1 << 30
    lens[0], lens[3] = 1 << 30, -7
    out, lse = run_attn8(bt, ql, qr, 0.07, lens=lens, table=table)
    bt.kv_len[3] = 0
    check_attn8(bt, ql, qr, 0.07, out, lse, holes=[(0, 1), (1, 0), (1, 3)] + [(2, p) for p in range(4)])
    assert (out[3] == 0).all() and (lse[4] == -math.inf).all()


def test_attn8_tree_rows_that_see_nothing():
    bt = Batch8(29, [70, 2], [70, 2], 16, 512)
    ql, qr = bt.queries(4)
    tree = torch.zeros(72, 1, dtype=torch.int64)
    tree[1] = -1
    tree[70] = -2
    out, lse = run_attn8(bt, ql, qr, 0.07, tree)
    check_attn8(bt, ql, qr, 0.07, out, lse, tree)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and (out[71] == 0).all()


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [-5, 2, 3, 4], [0, 1, 2, 900], [4, 4, 4, 4], [0, 0, 0, 0], [3, 2, 1, 0]])
def test_attn8_survives_bad_offsets(cu):
    """cu_q that falls, is negative or passes the tokens: rows of no sequence stay as they were."""
    bt = Batch8(41, [1, 1, 1], [40, 50, 60], 16, 512)
    bt.N, bt.cu = 4, torch.tensor(cu, dtype=torch.int32)
    ql, qr = bt.queries(8)
    out = torch.full((4, 8, 512), 7.0, dtype=BF, device="cuda")
    run_attn8(bt, ql, qr, 0.07, out=out)
    torch.cuda.synchronize()
    inside = set()
    for a, b in zip(cu, cu[1:]):
        inside |= set(range(max(a, 0), min(b, 4)))
    for t in set(range(4)) - inside:
        assert (out[t] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("how", ["latent", "scale", "rope"])
def test_attn8_values_that_are_not_finite(dtype, heads, how):
    """A drafted token with a NaN (in its latent, as its scale, in its rotated key) makes the rows that see it not finite and
    leaves the others as exact as ever; so does a NaN query."""
    bt = Batch8(43, [5, 3], [69, 200], 64, 512, dtype)
    ql, qr = bt.queries(heads)
    row = bt.rows8.view(-1, 656)[bt.rows(0, 69)[66]]  # token 2 of the first sequence's five
    if how == "latent":
        row[100:103] = torch.tensor([0x7F, 0xFF, 0x7F], dtype=torch.uint8)
    elif how == "scale":
        row[640] = 255
    else:
        row[512:640] = torch.full((64,), math.nan, dtype=dtype).view(torch.uint8)
    bt.refresh()
    for tree in (None, torch.tensor([[1], [2], [4], [8], [28], [1], [3], [7]])):
        out, lse = run_attn8(bt, ql, qr, 0.07, tree)
        sees = [2, 3, 4] if tree is None else [2, 4]
        refs = bt.reference(ql, qr, 0.07, tree)
        for t in range(8):
            if t in sees:
                assert not torch.isfinite(out[t].float()).all(-1).any()
            else:
                assert_attention(out[t].cpu(), lse[t].cpu(), refs[t][0], refs[t][1], dtype, f"token {t}")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_attn8_a_query_that_is_not_finite(dtype):
    bt = Batch8(43, [5, 3], [69, 200], 64, 512, dtype)
    ql, qr = bt.queries(16)
    clean, _ = run_attn8(bt, ql, qr, 0.07)
    ql[1, 3, 7] = math.nan
    out, _ = run_attn8(bt, ql, qr, 0.07)
    assert torch.isnan(out[1, 3].float()).all()
    keep = torch.ones(8, 16, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(out[keep.cuda()], clean[keep.cuda()])


def test_attn8_strides_rows_behind_the_last_and_streams():
    bt = Batch8(47, [2, 1], [100, 300], 64, 512, extra_tokens=3)
    ql, qr = bt.queries(24)
    want, want_lse = run_attn8(bt, ql, qr, 0.07)
    wide = torch.zeros(bt.N, 24, 192, dtype=BF)
    wide[..., 128:] = qr
    out = torch.full((24, bt.N, 512), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    lse = torch.full((bt.N, 24), 7.0, device="cuda")
    side = torch.cuda.Stream()
    args = [t.cuda() for t in (bt.rows8, bt.cu, bt.lens, bt.table)]
    a, b = ql.transpose(0, 1).contiguous().cuda().transpose(0, 1), wide.cuda()[..., 128:]
    torch.cuda.synchronize()
    B.ds4hc_latent_attn8(a, b, *args, scale=0.07, out=out, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out[:3], want[:3]) and torch.equal(lse[:3], want_lse[:3])
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()


def test_attn8_repeats_bit_for_bit():
    bt = Batch8(53, [1, 1, 4], [3000, 10, 1500], 64, 512)
    ql, qr = bt.queries(128)
    first = run_attn8(bt, ql, qr, 0.07)
    for _ in range(5):
        again = run_attn8(bt, ql, qr, 0.07)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])


def test_attn8_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, the sequence's pages at its far end; the append writes there too."""
    n_pages, page = 110000, 64
    cache = torch.zeros(n_pages, page, 656, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    bt = Batch8(59, [2], [300], page, 512)
    table = bt.table.clone()
    for p in range(5):
        table[0, p] = n_pages - 1 - 3 * p
        cache[n_pages - 1 - 3 * p] = bt.rows8[bt.table[0, p].long()].cuda()
    ql, qr = bt.queries(16)
    rows = torch.randn(2, 576, generator=bt.g).to(BF)
    B.ds4hc_latent_append8(rows.cuda(), torch.tensor([298, 299]).cuda(), B.ds4hc_rope_frequencies(64)[0].cuda(), cache,
                           bt.cu.cuda(), bt.lens.cuda(), table.cuda())
    bt.rows8.view(-1, 656)[bt.rows(0, 300)[298:]] = cache[n_pages - 1 - 12, 42:44].cpu()
    bt.refresh()
    assert (bt.cache.view(-1, 576)[bt.rows(0, 300)[298:], :512].std() - 1).abs() < 0.1
    out, lse = B.ds4hc_latent_attn8(ql.cuda(), qr.cuda(), cache, bt.cu.cuda(), bt.lens.cuda(), table.cuda(), scale=0.07,
                                    want_lse=True)
    check_attn8(bt, ql, qr, 0.07, out, lse)


def test_attn8_in_a_graph_follows_the_lengths():
    """A captured append and attention, replayed with other lengths and with eager work between the replays: each replay has
    the eager result's bits."""
    bt = Batch8(71, [1, 1, 1], [400, 300, 200], 16, 512)
    ql, qr = (t.cuda() for t in bt.queries(32))
    rows = torch.randn(3, 576, generator=bt.g).to(BF).cuda()
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    cache, cu, lens, table = bt.rows8.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda()
    pos = (lens - 1).long()
    out, lse = torch.empty(3, 32, 512, dtype=BF, device="cuda"), torch.empty(3, 32, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def step():
        B.ds4hc_latent_append8(rows, pos, f, cache, cu, lens, table)
        B.ds4hc_latent_attn8(ql, qr, cache, cu, lens, table, scale=0.07, out=out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([400, 300, 200], [17, 300, 1], [399, 0, 64], [400, 300, 200]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        pos.copy_((lens - 1).long())
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        out.fill_(0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), out.view(torch.int16)) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len", [
    (16, 512, 4, [2, 1], [333, 150]), (128, 512, 8, [1], [1000]), (64, 256, 8, [1, 3], [64, 129]), (16, 128, 2, [5], [400]),
    (128, 512, 1, [2], [200])])
def test_attn8_small_pages(dtype, heads, latent, page, q_len, kv_len):
    """Pages of fewer than 16 tokens over several tiles, one of them missing."""
    bt = Batch8(73, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    table = bt.table.clone()
    table[0, 70 // page] = -1
    tree = random_tree(bt.g, q_len, 1)
    for mask in (None, tree):
        out, lse = run_attn8(bt, ql, qr, 0.07, mask, table=table)
        check_attn8(bt, ql, qr, 0.07, out, lse, mask, holes=[(0, 70 // page)])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page,q_len,kv_len,words", [(64, [200, 60, 1, 9], [260, 700, 65, 9], 0), (4, [256], [300], 4),
                                                     (16, [64, 64, 64, 64, 2], [64, 1000, 129, 2000, 3000], 1)])
def test_attn8_many_rows(dtype, page, q_len, kv_len, words):
    """Calls of 32768 rows and more, which are run by tiles of 128 rows: written whole, and cut between workgroups; then with
    a token that is NaN, which rows behind it see and others do not."""
    bt = Batch8(109, q_len, kv_len, page, 512, dtype)
    ql, qr = bt.queries(128)
    assert bt.N * 128 >= 32768
    tree = random_tree(bt.g, q_len, words) if words else None
    out, lse = run_attn8(bt, ql, qr, 0.07, tree)
    refs = bt.reference(ql, qr, 0.07, tree)
    for t, (ref, n) in enumerate(refs):
        assert_attention(out[t].cpu(), lse[t].cpu(), ref, n, dtype, f"token {t}")
    bad = q_len[0] // 2
    bt.rows8.view(-1, 656)[bt.rows(0, kv_len[0])[kv_len[0] - q_len[0] + bad], 77] = 0x7F
    out, lse = run_attn8(bt, ql, qr, 0.07, tree)
    for t, (ref, n) in enumerate(refs):
        sees = t < q_len[0] and (t >= bad if tree is None else bool((int(tree[t, bad // 64]) >> (bad % 64)) & 1))
        if sees:
            assert not torch.isfinite(out[t].float()).all(-1).any()
        else:
            assert_attention(out[t].cpu(), lse[t].cpu(), ref, n, dtype, f"token {t}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [1, 40, 128])
def test_attn8_one_token_seen_gives_its_values(dtype, heads):
    """A row that sees one token alone has its values, whatever its logit and power of 2 are: the rounded weight's product with
    a value of 4 bits is exact, and the quotient by the same weight off by roundings of float32, which the rounding to 16 bits
    takes back to the value."""
    bt = Batch8(79, [1] * 9, [1] * 9, 16, 512, dtype, spread=3)
    ql, qr = bt.queries(heads, 3.0)
    out, lse = run_attn8(bt, ql, qr, 0.3)
    for b in range(9):
        want = bt.cache.view(-1, 576)[bt.rows(b, 1)[0], :512].to(dtype)
        assert torch.equal(out[b].cpu(), want.expand(heads, 512))
    check_attn8(bt, ql, qr, 0.3, out, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,kv_len", [(16, 300), (128, 300), (64, 6000)])
def test_attn8_logits_of_minus_infinity(dtype, heads, kv_len):
    """Tokens whose rotated key is infinite against the queries' sign weigh nothing, whole tiles and parts of them, too: as if
    their pages were missing."""
    bt = Batch8(83, [1], [kv_len], 64, 512, dtype)
    ql, qr = bt.queries(heads)
    qr[..., 5] = 1 + qr[..., 5].abs()
    pages = [0, 1, 2, 4] if kv_len < 1000 else list(range(40)) + list(range(50, 60)) + [93]
    for p in pages:
        keys = bt.rows8[bt.table[0, p].long(), :, 512:640].view(dtype).clone()
        keys[:, 5] = -math.inf
        bt.rows8[bt.table[0, p].long(), :, 512:640] = keys.view(torch.uint8)
    out, lse = run_attn8(bt, ql, qr, 0.07)
    check_attn8(bt, ql, qr, 0.07, out, lse, holes=[(0, p) for p in pages])


def test_attn8_results_of_more_than_2_to_the_31_elements():
    """40000 sequences of one token, 128 heads: queries and results behind 2^31 elements, and 2^32 bytes."""
    n, page = 40000, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = torch.zeros(n, page, 656, dtype=torch.uint8, device="cuda")
    cache[:, 0, :512] = torch.randint(0, 120, (n, 512), generator=g, dtype=torch.uint8, device="cuda")
    cache[:, 0, 640] = 127
    q = torch.randn(n, 128, 512, generator=g, dtype=BF, device="cuda")
    r = torch.randn(n, 128, 64, generator=g, dtype=BF, device="cuda")
    assert q.numel() > 2 ** 31
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    out, _ = B.ds4hc_latent_attn8(q, r, cache, torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                                  torch.ones(n, dtype=torch.int32, device="cuda"), table, scale=0.05)
    for t in (0, 1, 20000, 32767, 32768, 39998, 39999):
        want = cache[table[t, 0].item(), 0, :512].view(torch.float8_e4m3fn).to(BF)
        assert torch.equal(out[t], want.expand(128, 512)), t


def test_attn8_two_at_once():
    """Calls side by side on two streams, each with the workspace that it was given: as one after another."""
    both = []
    for seed, heads in ((89, 16), (97, 128)):
        bt = Batch8(seed, [1, 2], [3000, 900], 64, 512)
        ql, qr = bt.queries(heads)
        both.append([t.cuda() for t in (ql, qr, bt.rows8, bt.cu, bt.lens, bt.table)])
    want = [B.ds4hc_latent_attn8(*a, scale=0.07, want_lse=True) for a in both]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [B.ds4hc_latent_attn8(*a, scale=0.07, want_lse=True, stream=s) for a, s in zip(both, streams)]
        torch.cuda.synchronize()
        for (o, l), (o2, l2) in zip(got, want):
            assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)


def test_attn8_two_graphs_share_a_workspace():
    """Two captured calls of unlike sizes with one workspace, replayed in turn on one stream with eager work between."""
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    graphs = []
    for seed, heads, kv in ((101, 16, 2000), (103, 128, 700)):
        bt = Batch8(seed, [1, 2], [kv, 900], 64, 512)
        ql, qr = bt.queries(heads)
        a = [t.cuda() for t in (ql, qr, bt.rows8, bt.cu, bt.lens, bt.table)]
        want = B.ds4hc_latent_attn8(*a, scale=0.07)[0]
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.ds4hc_latent_attn8(*a, scale=0.07, out=out, workspace=ws)
        graphs.append((graph, out, want, a))
    for _ in range(3):
        for graph, out, want, a in graphs:
            graph.replay()
        for graph, out, want, a in graphs:
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
            out.zero_()
            B.ds4hc_latent_attn8(*a, scale=0.07, workspace=ws)


def test_refusals_of_the_binding():
    bt = Batch8(107, [1, 1], [5, 9], 16, 512)
    ql, qr = (t.cuda() for t in bt.queries(4))
    cache, cu, lens, table = (t.cuda() for t in (bt.rows8, bt.cu, bt.lens, bt.table))
    ok = dict(scale=0.1)
    kv, pos, f = torch.zeros(2, 576, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), B.ds4hc_rope_frequencies(64)[0].cuda()
    for call in (lambda: B.ds4hc_latent_attn8(ql.float(), qr.float(), cache, cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr.half(), cache, cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache.view(torch.int8), cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache, cu.long(), lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache, cu, lens, table, lse=torch.zeros(2, 4, device="cuda", dtype=BF), **ok),
                 lambda: B.ds4hc_latent_append8(kv, pos, f, cache, cu, lens, table, dtype=F32),
                 lambda: B.ds4hc_latent_append8(kv, pos.int(), f, cache, cu, lens, table)):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: B.ds4hc_latent_attn8(ql[..., :256], qr, cache, cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache[:, :, :640], cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache, cu, lens.cpu(), table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql.cpu(), qr, cache, cu, lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache, cu[:2], lens, table, **ok),
                 lambda: B.ds4hc_latent_attn8(ql, qr, cache, cu, lens, table, tree_mask=torch.zeros(1, 1, dtype=torch.int64, device="cuda"), **ok),
                 lambda: B.ds4hc_latent_append8(kv[:, :500], pos, f, cache, cu, lens, table),
                 lambda: B.ds4hc_latent_append8(kv, pos, f, cache, cu, lens, table.t())):
        with pytest.raises(ValueError):
            call()
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(B.Ds4hcError):
            B.ds4hc_latent_attn8(ql, qr, cache, cu, lens, table, scale=scale)
