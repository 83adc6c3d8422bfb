"""The attention-site operators at the edges of what their documentation allows."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from site_testlib import Batch, assert_attention, attend64, random_tree

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

# ------------------------------------------------------------------ float16 weights

def one_over_many(n, d, seed):
    """n keys of d elements whose logits under the query are normal, and a first one 17.5 above
    them that has 99.5 % of the weight. Element 5, which the query does not look at, is 1 in all
    keys but the first, where it is 0: its output is what the others weigh."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(d, generator=g)
    q[5] = 0
    q = q.to(HF)
    k = torch.randn(n, d, generator=g)
    scale = 1 / q.double().norm().item()
    k[0] = q.float() * (17.5 * scale)
    k[:, 5] = 1
    k[0, 5] = 0
    return q, k.to(HF), scale


def assert_tail(got, q, k, v, scale, where):
    """Every weight is rounded once, by u of it or half a step of the subnormals, 2^-25; the
    largest is above 2^6. With n of them numerator and denominator are each off by at most
    u + n 2^-31 of the weights' sum; logits and sums as in site_testlib."""
    n, u, e = len(k), 2.0 ** -11, 2.0 ** -24
    q, k, v = q.double(), k.double(), v.double()
    s = k @ q * scale
    w = torch.softmax(s, 0)
    out, size = w @ v, w @ v.abs()
    ds = (len(q) + 8) * e * scale * (k.abs() @ q.abs()).max()
    bound = (2 * u + 4 * ds + 2 * (n + 64) * e) * size + u * out.abs() + 2 * n * 2.0 ** -31 * v.abs().amax(0)
    over = ((got.double() - out).abs() / bound).max().item()
    assert over <= 1.0, f"{where}: {over:.3g} times the bound; element 5 {got[5].item():.5f} for {out[5].item():.5f}"


@pytest.mark.parametrize("heads", [1, 64, 128])  # 32, 64 and 128 rows a tile
def test_attn_float16_keeps_the_weights_of_many_small_ones(heads):
    """As many sequences as workgroups, all of the same pages, so that each is summed in one run."""
    n, page = 131072, 4096
    q, k, scale = one_over_many(n, 192, 221)
    cache = k.view(n // page, page, 192).contiguous().cuda()
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(256, -1).contiguous()
    queries = q.cuda().expand(256, heads, 192)
    cu = torch.arange(257, dtype=torch.int32, device="cuda")
    lens = torch.full((256,), n, dtype=torch.int32, device="cuda")
    out, lse = B.ds4hc_latent_attn(queries[..., :128], queries[..., 128:], cache, cu, lens, table, scale=scale, want_lse=True)
    want = torch.logsumexp(k.double() @ q.double() * scale, 0).item()
    for b, h in ((0, 0), (100, heads // 2), (255, heads - 1)):
        assert_tail(out[b, h].cpu(), q, k, k[:, :128], scale, f"sequence {b} head {h}")
        assert abs(lse[b, h].item() - want) < 1e-3


@pytest.mark.parametrize("rows", [1, 49153])  # 64 and 128 rows a workgroup
def test_prefill_float16_keeps_the_weights_of_many_small_ones(rows):
    n = 131072
    q, k, scale = one_over_many(n, 192, 223)
    kv = torch.cat((k[:, :128], k[:, :128]), -1).view(n, 1, 256).contiguous()
    cu = lambda v: torch.tensor([0, v], dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = B.ds4hc_latent_prefill(q.cuda().expand(rows, 1, 192).contiguous(), kv.cuda(), k[:, 128:].contiguous().cuda(),
                                      cu(rows), cu(n), scale=scale, causal=False, want_lse=True)
    for r in {0, rows // 2, rows - 1}:
        assert_tail(out[r, 0].cpu(), q, k, k[:, :128], scale, f"row {r}")


@pytest.mark.parametrize("dtype,far", [(BF, 2.0 ** 30), (HF, 2.0 ** 27)])
def test_far_logits_stay_finite(dtype, far):
    """Up to the documented end of the logits' range, on both sides of 0 and of every step of the
    running maximum: keys along the query, so that logit j is `far` times a number of [-1, 1]."""
    g = torch.Generator().manual_seed(227)
    n, heads = 500, 64
    q = (torch.randn(192, generator=g) * 64).to(dtype)
    for size in (far, far / 7, far / 64, 2.0 ** 14):
        k = (q.float() * (2 * torch.rand(n, 1, generator=g) - 1)).to(dtype)
        s = k.double() @ q.double()
        scale = 0.999 * size / s.abs().max().item()
        cu = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        table = torch.arange(32, dtype=torch.int32, device="cuda")[None]
        cache = torch.zeros(512, 192, dtype=dtype)
        cache[:n] = k
        many = q.cuda().expand(2, heads, 192)
        out, lse = B.ds4hc_latent_attn(many[..., :128], many[..., 128:], cache.view(32, 16, 192).cuda(), cu(0, 2), cu(n), table,
                                       scale=scale, want_lse=True)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all(), size
        kv = torch.cat((k[:, :128], k[:, :128]), -1).view(n, 1, 256).expand(n, heads, 256).contiguous().cuda()
        out, lse = B.ds4hc_latent_prefill(q.cuda().expand(n, heads, 192).contiguous(), kv, k[:, 128:].contiguous().cuda(), cu(0, n),
                                          cu(0, n), scale=scale, want_lse=True)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all(), size

# ------------------------------------------------------------------ infinite logits

@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("heads", [8, 64, 128])
def test_attn_a_logit_of_minus_infinity_is_a_weight_of_0(heads, tree):
    """An infinity in a cached token's rotated part: the rows that see it and whose product with
    it is negative pass over the token; where it is positive they are not finite."""
    bt = Batch(231, [4, 1], [300, 130], 64, 512)
    ql, qr = bt.queries(heads)
    qr[:, ::2, 9], qr[:, 1::2, 9] = -1.0, 1.0
    mask = random_tree(bt.g, bt.q_len, 1) if tree else None
    ref = bt.reference(ql, qr, 0.07, mask, [])
    flat = bt.cache.view(-1, 576)
    for j in (5, 200, 296, 297):  # context, and the call's own first two tokens
        kept = flat[bt.rows(0, 300)[j]].clone()
        flat[bt.rows(0, 300)[j], 512 + 9] = math.inf
        out, lse = B.ds4hc_latent_attn(ql.cuda(), qr.cuda(), bt.cache.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda(),
                                       scale=0.07, tree_mask=None if mask is None else mask.cuda(), want_lse=True)
        out, lse = out.cpu(), lse.cpu()
        with_it = bt.reference(ql[:, ::2], qr[:, ::2], 0.07, mask, [])
        for t in range(5):
            sees = t < 4 and (j < 296 or (j - 296 <= t if mask is None else bool(int(mask[t, 0]) >> (j - 296) & 1)))
            r, n = with_it[t]
            r = r[:3] + (ref[t][0][3][::2],)  # (the logits' error bound of the finite ones)
            assert_attention(out[t, ::2], lse[t, ::2], r, n, BF, f"token {t}, infinity at {j}")
            if sees:
                assert not torch.isfinite(out[t, 1::2].float()).any()
            else:
                assert_attention(out[t, 1::2], lse[t, 1::2], tuple(x[1::2] for x in ref[t][0]), n, BF, f"token {t}, infinity at {j}")
        flat[bt.rows(0, 300)[j]] = kept


def test_attn_rows_whose_every_logit_is_minus_infinity():
    """They are as rows that see nothing, in a tile that all rows see whole, in a masked one and
    over several parts."""
    for kv in (64, 130, 2000):
        bt = Batch(233, [1], [kv], 64, 512)
        ql, qr = bt.queries(64)
        qr[:, ::2, 9], qr[:, 1::2, 9] = -1.0, 1.0
        bt.cache[..., 512 + 9] = math.inf
        bt.cache.view(-1, 576)[bt.rows(0, kv)[kv - 1], 512 + 9] = math.inf
        out, lse = B.ds4hc_latent_attn(ql.cuda(), qr.cuda(), bt.cache.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda(),
                                       scale=0.07, want_lse=True)
        assert (out[0, ::2] == 0).all() and (lse[0, ::2] == -math.inf).all()
        assert not torch.isfinite(out[0, 1::2].float()).any()


@pytest.mark.parametrize("heads", [2, 400])  # 64 and 128 rows a workgroup
@pytest.mark.parametrize("part", ["head", "shared"])
def test_prefill_a_logit_of_minus_infinity_is_a_weight_of_0(heads, part):
    """An infinite key: rows that see it with a negative product pass over it, those with a positive
    one are not finite, those that do not see it are as ever. (To the bound, not to the bit: 32 rows
    share the decision to raise a running maximum, which scales each by a power of 2 of its own and
    moves the rounding of x - maximum, as the bound's share for the logits counts.)"""
    g = torch.Generator().manual_seed(239)
    n = 150
    q, kv, kr = (torch.randn(*s, generator=g).to(BF) for s in ((n, heads, 192), (n, heads, 256), (n, 64)))
    e = 7 if part == "head" else 128 + 9
    q[:, :, e] = torch.where(torch.arange(n) % 2 == 0, -1.0, 1.0).to(BF)[:, None]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for at in (0, 40, 64, 149):
        was = kv[at, :, 7].clone(), kr[at, 9].clone()
        if part == "head":
            kv[at, :, 7] = math.inf
        else:
            kr[at, 9] = math.inf
        out, lse = [t.cpu() for t in B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), kr.cuda(), cu, cu, scale=0.08, want_lse=True)]
        odd = at + (at + 1) % 2
        assert not torch.isfinite(out[odd::2].float()).any()
        even = at + at % 2
        for h in (0, heads - 1):
            seen = torch.ones(n, n, dtype=torch.bool).tril()
            seen[:, at] = False
            keys = torch.cat((kv[:, h, :128], kr), -1)
            for rows in (slice(0, at), slice(even, n, 2)):
                ref = attend64(q[rows, h], keys, kv[:, h, 128:], seen[rows], 0.08)
                assert_attention(out[rows, h], lse[rows, h], ref, seen[rows].sum(-1), BF, f"infinity at {at}, head {h}")
        kv[at, :, 7], kr[at, 9] = was


# ------------------------------------------------------------------ angles

@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_angles_are_not_rounded_to_float32(interleaved):
    """x = (1, 0) gives cos and sin themselves. The float32 functions are documented to a unit in the
    last place, at most 2^-24 below 1; one sum brings in what rounding the reduced angle left, 2^-25
    at most; its parts' roundings and the angle's 64-bit product are far below (rounded to float32,
    the angle of up to half a turn alone would be off by pi 2^-25)."""
    n = 1 << 19
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    g = torch.Generator().manual_seed(241)
    positions = torch.randint(0, 1000000, (n,), generator=g).cuda()
    x = torch.zeros(n, 1, 64, device="cuda")
    first = x[..., 0::2] if interleaved else x[..., :32]
    first.fill_(1)
    y = B.ds4hc_rope(x, positions, f, interleaved=interleaved)[:, 0].double()
    c, s = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :32], y[:, 32:])
    a = positions.double()[:, None] * f
    bound = 1.5 * 2.0 ** -24 + a * 2.0 ** -50 + 2.0 ** -40
    worst = max(((c - a.cos()).abs() / bound).max().item(), ((s - a.sin()).abs() / bound).max().item())
    assert worst <= 1, worst


# ------------------------------------------------------------------ refusals

def test_a_tree_mask_without_words_is_refused():
    """An array of no elements has no address, and a call without a mask is another one: causal."""
    bt = Batch(251, [2], [10], 16, 128)
    ql, qr = bt.queries(2)
    args = [t.cuda() for t in (ql, qr, bt.cache, bt.cu, bt.lens, bt.table)]
    with pytest.raises(ValueError, match="tree_mask"):
        B.ds4hc_latent_attn(*args, scale=0.07, tree_mask=torch.zeros(2, 0, dtype=torch.int64, device="cuda"))
