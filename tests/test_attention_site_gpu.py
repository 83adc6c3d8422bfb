"""The attention-site operators on the GPU against 64-bit references (bounds derived
in site_testlib), at the sizes, masks and layouts where they can go wrong."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from site_testlib import (Batch, assert_attention, attend64, random_tree, rope_bound, turn64, u_of)

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ rotary positions

def check_rope(x, positions, f, amp, interleaved, inverse, out):
    ref = turn64(x, positions, f, amp, interleaved, inverse)
    part, u = rope_bound(x, positions, f, amp, interleaved, x.dtype)
    bound = part * (1 + u) + u * ref.abs() + (6e-8 if x.dtype == HF else 1e-38)  # half a step of float16's subnormals
    over = (out.double() - ref).abs() / bound
    assert over.max().item() <= 1.0, over.max().item()


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("N,heads,head_dim,dim,start", [(1, 1, 2, 2, 0), (3, 5, 70, 6, 17), (4, 128, 192, 64, 1000),
                                                        (257, 3, 64, 64, -90), (2, 7, 512, 512, 1 << 20),
                                                        (33, 1, 128, 128, 3000000), (5, 16, 100, 50, 7)])
def test_rope(dtype, interleaved, N, heads, head_dim, dim, start):
    say(f"[gpu] rope {dtype} N={N} heads={heads} dim={dim} of {head_dim} interleaved={interleaved}")
    g = torch.Generator().manual_seed(N * 1000 + dim)
    full = torch.randn(N, heads, head_dim, generator=g).to(dtype)
    x = full[..., head_dim - dim:]
    positions = torch.randint(0, 5000, (N,), generator=g) + start
    f, amp = B.ds4hc_rope_frequencies(dim, factor=8.0, original_length=4096)
    dev = full.cuda()
    for inverse in (False, True):
        out = B.ds4hc_rope(dev[..., head_dim - dim:], positions.cuda(), f.cuda(), interleaved=interleaved,
                           inverse=inverse, amplitude=amp)
        assert out.is_contiguous() and out.dtype == dtype
        check_rope(x, positions, f, amp, interleaved, inverse, out.cpu())
    # in place: the same bits, and the rest of each head as it was
    y = dev.clone()
    res = B.ds4hc_rope(y[..., head_dim - dim:], positions.cuda(), f.cuda(), interleaved=interleaved, inverse=True,
                       amplitude=amp, out=y[..., head_dim - dim:])
    assert res.data_ptr() == y[..., head_dim - dim:].data_ptr()
    assert torch.equal(y[..., head_dim - dim:], out) and torch.equal(y[..., :head_dim - dim], dev[..., :head_dim - dim])


def test_rope_strides_and_alignment():
    """Heads outside tokens, a broadcast head, rows off every 16-byte boundary: the
    same bits as from dense arrays."""
    g = torch.Generator().manual_seed(1)
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    pos = torch.randint(0, 100000, (9,), generator=g).cuda()
    for dtype in (F32, BF, HF):
        x = torch.randn(9, 5, 64, generator=g).to(dtype).cuda()
        for inter in (True, False):
            want = B.ds4hc_rope(x, pos, f, interleaved=inter)
            turned = x.transpose(0, 1).contiguous().transpose(0, 1)
            out = torch.empty(5, 9, 64, dtype=dtype, device="cuda").transpose(0, 1)
            assert torch.equal(B.ds4hc_rope(turned, pos, f, interleaved=inter, out=out), want)
            odd = torch.full((9, 5, 67), 7.0, dtype=dtype, device="cuda")
            odd[..., 1:65] = x
            place = torch.full((9, 5, 67), 5.0, dtype=dtype, device="cuda")
            assert torch.equal(B.ds4hc_rope(odd[..., 1:65], pos, f, interleaved=inter, out=place[..., 3:]), want)
            assert (place[..., :3] == 5).all()
            one = x[:, :1].expand(9, 5, 64)
            assert torch.equal(B.ds4hc_rope(one, pos, f, interleaved=inter),
                               B.ds4hc_rope(one.contiguous(), pos, f, interleaved=inter))
    assert B.ds4hc_rope(x[:0], pos[:0], f).shape == (0, 5, 64)


def test_rope_gradient_is_the_inverse():
    """With L = sum g . rope(x), dL/dx is the inverse rotation of g: against central
    differences of the operator itself. L is linear in x, so a difference over a step of
    1 has no truncation error: what is left is float32 rounding of 2 x 64 terms of size
    |g||y| <= 4 * 6 (64 * 2 * 24 * 2^-24 < 2e-4)."""
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(2, 1, 8, generator=g), torch.randn(2, 1, 8, generator=g)
    f, _ = B.ds4hc_rope_frequencies(8)
    pos = torch.tensor([3, 77]).cuda()
    for inter in (True, False):
        grad = B.ds4hc_rope(w.cuda(), pos, f.cuda(), interleaved=inter, inverse=True, amplitude=1.25).cpu()
        for t in range(2):
            for e in range(8):
                d = torch.zeros_like(x)
                d[t, 0, e] = 0.5
                up, down = (B.ds4hc_rope((x + s * d).cuda(), pos, f.cuda(), interleaved=inter, amplitude=1.25).cpu()
                            for s in (1, -1))
                assert abs(((up - down) * w).double().sum().item() - grad[t, 0, e].item()) < 2e-4


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("src", [F32, BF, HF])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("latent,page,q_len,kv_len,norm,interleaved",
                         [(512, 64, [1, 1, 1], [1, 64, 65], True, True), (128, 1, [3, 0, 5], [3, 7, 9], True, False),
                          (256, 16, [40, 2], [40, 500], False, True), (512, 128, [1], [300], True, False)])
def test_append(src, dtype, latent, page, q_len, kv_len, norm, interleaved):
    say(f"[gpu] append {src}->{dtype} latent={latent} page={page} q={q_len} kv={kv_len}")
    bt = Batch(5, q_len, kv_len, page, latent, dtype, extra_tokens=2)
    wide = torch.randn(bt.N, latent + 64 + 40, generator=bt.g).to(src)
    kv = wide[:, 24:24 + latent + 64]  # 24 elements: a 16-byte boundary for every type
    w = 1 + 0.3 * torch.randn(latent, generator=bt.g) if norm else None
    f, _ = B.ds4hc_rope_frequencies(64)
    positions = torch.randint(0, 200000, (bt.N,), generator=bt.g)
    before = bt.cache.clone()
    cache = bt.cache.cuda()
    args = (positions.cuda(), f.cuda(), cache, bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda())
    got = B.ds4hc_latent_append(wide.cuda()[:, 24:24 + latent + 64], *args, norm_weight=None if w is None else w.cuda(),
                                rms_eps=1e-5, interleaved=interleaved, amplitude=1.5)
    assert got is cache
    c = kv[:, :latent].double()
    if norm:
        c = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w.double()
    r = turn64(kv[:, latent:], positions, f, 1.5, interleaved)
    part, _ = rope_bound(kv[:, latent:], positions, f, 1.5, interleaved, dtype)
    # the norm: a float32 sum of `latent` squares (latent / 2 e in its root), root, reciprocal and two products
    slack = torch.cat((c.abs() * (latent / 2 + 8) * 2.0 ** -24, part), -1)
    want, u = torch.cat((c, r), -1), u_of(dtype)
    flat, old = cache.cpu().view(-1, latent + 64), before.view(-1, latent + 64)
    touched = torch.zeros(len(flat), dtype=torch.bool)
    for b, (q, k) in enumerate(zip(q_len, kv_len)):
        rows = bt.rows(b, k)[k - q:]
        touched[rows] = True
        ref = want[bt.cu[b]:bt.cu[b] + q]
        bound = slack[bt.cu[b]:bt.cu[b] + q] * (1 + u) + u * ref.abs() + (6e-8 if dtype == HF else 1e-38)
        assert ((flat[rows].double() - ref).abs() <= bound).all()
    assert torch.equal(flat[~touched].view(torch.int16), old[~touched].view(torch.int16))


def test_append_passes_over_what_has_no_place():
    """More tokens than the cache's length, pages not in the cache (-1 and beyond), a
    length behind the table, sequences behind the last: nothing else is written."""
    g = torch.Generator().manual_seed(3)
    cache = torch.zeros(6, 4, 576, dtype=BF, device="cuda")
    kv = torch.ones(12, 576, dtype=BF, device="cuda")
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    pos = torch.zeros(12, dtype=torch.int64, device="cuda")
    cu = torch.tensor([0, 3, 6, 9], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 7, 1000], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, -1], [1, 99], [2, 3]], dtype=torch.int32, device="cuda")
    B.ds4hc_latent_append(kv, pos, f, cache, cu, lens, table)
    rows = set(cache.view(-1, 576).abs().sum(-1).nonzero()[:, 0].tolist())
    # 0: one place (token 2); 1: tokens 4, 5, 6 lie in a page that is not there; 2: length 1000 is taken as 8
    assert rows == {0, 13, 14, 15}


# ------------------------------------------------------------------ latent attention

def run_attn(bt, ql, qr, scale, tree=None, lens=None, table=None, **kw):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    return B.ds4hc_latent_attn(d(ql), d(qr), d(bt.cache), d(bt.cu), d(bt.lens if lens is None else lens),
                               d(bt.table if table is None else table), scale=scale, tree_mask=d(tree), want_lse=True,
                               **kw)


def check_attn(bt, ql, qr, scale, out, lse, tree=None, holes=()):
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
    (64, 512, 64, [2, 1, 1, 5], [70, 1, 260, 5]), (8, 512, 2, [1], [37])])
def test_attn_causal(dtype, heads, latent, page, q_len, kv_len):
    say(f"[gpu] attn {dtype} heads={heads} latent={latent} page={page} q={q_len} kv={kv_len}")
    bt = Batch(11 + heads, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    out, lse = run_attn(bt, ql, qr, 0.07)
    check_attn(bt, ql, qr, 0.07, out, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,latent,page,q_len,kv_len,words", [
    (16, 512, 16, [9, 33], [300, 33], 1), (128, 512, 64, [6], [70], 1), (3, 256, 64, [100, 2], [400, 2], 2),
    (16, 128, 32, [64, 65], [64, 200], 2)])
def test_attn_tree(dtype, heads, latent, page, q_len, kv_len, words):
    say(f"[gpu] attn tree {dtype} heads={heads} latent={latent} q={q_len} kv={kv_len}")
    bt = Batch(23, q_len, kv_len, page, latent, dtype)
    ql, qr = bt.queries(heads)
    tree = random_tree(bt.g, q_len, words)
    tree[0] = 0  # sees the context alone
    out, lse = run_attn(bt, ql, qr, 0.07, tree)
    check_attn(bt, ql, qr, 0.07, out, lse, tree)


def test_attn_tree_rows_that_see_nothing():
    """No context and an empty mask: 0 and -infinity; bits beyond the tokens there are
    and tokens beyond the words given are seen by none."""
    bt = Batch(29, [70, 2], [70, 2], 16, 512)
    ql, qr = bt.queries(4)
    tree = torch.zeros(72, 1, dtype=torch.int64)
    tree[1] = -1
    tree[70] = -2  # of the second sequence: token 1, and 62 tokens that are not there
    out, lse = run_attn(bt, ql, qr, 0.07, tree)
    check_attn(bt, ql, qr, 0.07, out, lse, tree)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and (out[71] == 0).all()


def test_attn_large_logits_and_one_weight():
    """Logits of +-400: one weight takes all, sums neither overflow nor vanish."""
    bt = Batch(31, [1, 2], [700, 90], 64, 512)
    ql, qr = bt.queries(16, 4.0)
    out, lse = run_attn(bt, ql, qr, 1.0)
    check_attn(bt, ql, qr, 1.0, out, lse)


def test_attn_holes_and_lengths_beyond_the_table():
    """Pages that are not in the cache are not seen; a length behind the table is cut; a
    negative one is 0."""
    bt = Batch(37, [1, 2, 1, 1], [256, 256, 256, 100], 64, 512, max_pages=4)
    ql, qr = bt.queries(16)
    table, lens = bt.table.clone(), bt.lens.clone()
    table[0, 1], table[1, 0], table[1, 3], table[2] = -1, bt.n_pages, -5, 1 << 30
    lens[0], lens[3] = 1 << 30, -7
    out, lse = run_attn(bt, ql, qr, 0.07, lens=lens, table=table)
    bt.kv_len[3] = 0
    check_attn(bt, ql, qr, 0.07, out, lse, holes=[(0, 1), (1, 0), (1, 3)] + [(2, p) for p in range(4)])
    assert (out[3] == 0).all() and (lse[4] == -math.inf).all()


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [-5, 2, 3, 4], [0, 1, 2, 900], [4, 4, 4, 4], [0, 0, 0, 0], [3, 2, 1, 0]])
def test_attn_and_append_survive_bad_offsets(cu):
    """cu_q that falls, is negative or passes the tokens: every access stays inside, rows
    of no sequence stay as they were."""
    bt = Batch(41, [1, 1, 1], [40, 50, 60], 16, 512)
    bt.N, bt.cu = 4, torch.tensor(cu, dtype=torch.int32)
    ql, qr = bt.queries(8)
    out = torch.full((4, 8, 512), 7.0, dtype=BF, device="cuda")
    run_attn(bt, ql, qr, 0.07, out=out)
    torch.cuda.synchronize()
    inside = set()
    for a, b in zip(cu, cu[1:]):
        inside |= set(range(max(a, 0), min(b, 4)))
    for t in set(range(4)) - inside:
        assert (out[t] == 7).all()
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    B.ds4hc_latent_append(torch.ones(4, 576, dtype=BF, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), f,
                          bt.cache.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.table.cuda())
    torch.cuda.synchronize()


def test_attn_values_that_are_not_finite():
    """A drafted token with NaN or infinities makes the rows that see it not finite and
    leaves the others as exact as ever; so does a NaN query."""
    for bad in (float("nan"), float("inf")):
        bt = Batch(43, [5, 3], [69, 200], 64, 512)
        ql, qr = bt.queries(16)
        flat = bt.cache.view(-1, 576)
        flat[bt.rows(0, 69)[66], 100:103] = bad   # token 2 of the first sequence's five
        for tree in (None, torch.tensor([[1], [2], [4], [8], [28], [1], [3], [7]])):
            out, lse = run_attn(bt, ql, qr, 0.07, tree)
            sees = [2, 3, 4] if tree is None else [2, 4]
            refs = bt.reference(ql, qr, 0.07, tree)
            for t in range(8):
                if t in sees:
                    assert not torch.isfinite(out[t].float()).all(-1).any()
                else:
                    assert_attention(out[t].cpu(), lse[t].cpu(), refs[t][0], refs[t][1], BF, f"token {t}")
    bt = Batch(43, [5, 3], [69, 200], 64, 512)
    ql, qr = bt.queries(16)
    clean, _ = run_attn(bt, ql, qr, 0.07)
    ql[1, 3, 7] = float("nan")
    out, _ = run_attn(bt, ql, qr, 0.07)
    assert torch.isnan(out[1, 3].float()).all()
    keep = torch.ones(8, 16, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(out[keep.cuda()], clean[keep.cuda()])


def test_attn_strides_rows_behind_the_last_and_streams():
    bt = Batch(47, [2, 1], [100, 300], 64, 512, extra_tokens=3)
    ql, qr = bt.queries(24)
    want, want_lse = run_attn(bt, ql, qr, 0.07)
    head_major = ql.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(bt.N, 24, 192, dtype=BF)
    wide[..., 128:] = qr
    out = torch.full((24, bt.N, 512), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    lse = torch.full((bt.N, 24), 7.0, device="cuda")
    side = torch.cuda.Stream()
    args = [t.cuda() for t in (bt.cache, bt.cu, bt.lens, bt.table)]
    a, b = head_major.cuda().transpose(0, 1).contiguous().transpose(0, 1), wide.cuda()[..., 128:]
    torch.cuda.synchronize()
    B.ds4hc_latent_attn(a, b, *args, scale=0.07, out=out, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out[:3], want[:3]) and torch.equal(lse[:3], want_lse[:3])
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()


def test_attn_repeats_bit_for_bit():
    bt = Batch(53, [1, 1, 4], [3000, 10, 1500], 64, 512)
    ql, qr = bt.queries(128)
    first = run_attn(bt, ql, qr, 0.07)
    for _ in range(5):
        again = run_attn(bt, ql, qr, 0.07)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])


def test_attn_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, the sequence's pages at its far end."""
    n_pages, page = 65000, 64
    cache = torch.zeros(n_pages, page, 576, dtype=BF, device="cuda")
    assert cache.numel() * 2 > 2 ** 32
    bt = Batch(59, [2], [300], page, 512)
    table = bt.table.clone()
    for p in range(5):
        table[0, p] = n_pages - 1 - 3 * p
        cache[n_pages - 1 - 3 * p] = bt.cache[bt.table[0, p].long()].cuda()
    ql, qr = bt.queries(16)
    f = B.ds4hc_rope_frequencies(64)[0]
    rows = torch.randn(2, 576, generator=bt.g).to(BF)
    pos = torch.tensor([298, 299])
    B.ds4hc_latent_append(rows.cuda(), pos.cuda(), f.cuda(), cache, bt.cu.cuda(), bt.lens.cuda(), table.cuda())
    bt.cache.view(-1, 576)[bt.rows(0, 300)[298:]] = cache[n_pages - 1 - 12, 42:44].cpu()
    assert (bt.cache.view(-1, 576)[bt.rows(0, 300)[298:], :512].float().std() - 1).abs() < 0.1
    out, lse = B.ds4hc_latent_attn(ql.cuda(), qr.cuda(), cache, bt.cu.cuda(), bt.lens.cuda(), table.cuda(), scale=0.07,
                                   want_lse=True)
    check_attn(bt, ql, qr, 0.07, out, lse)


def test_attn_in_captured_graphs():
    """Two captured graphs that share a workspace, replayed with lengths that changed in
    between and eager work beside them: every replay equals the eager result."""
    bt = Batch(61, [1, 1, 2], [2000, 300, 50], 64, 512)
    ql, qr = bt.queries(128)
    ql2, qr2 = bt.queries(128)
    dev = [t.cuda() for t in (bt.cache, bt.cu, bt.lens, bt.table)]
    q = [t.cuda() for t in (ql, qr, ql2, qr2)]
    c = B._paged(*dev)
    ws = torch.empty(max(B.ds4hc_latent_attn_workspace_bytes(c, 4, 128), 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(4, 128, 512, dtype=BF, device="cuda") for _ in range(2)]
    lses = [torch.empty(4, 128, device="cuda") for _ in range(2)]
    call = lambda k: B.ds4hc_latent_attn(q[2 * k], q[2 * k + 1], *dev, scale=0.07, out=outs[k], lse=lses[k], workspace=ws)  # noqa: E731
    call(0), call(1)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(k)
        graphs.append(g)
    for lens in ([2000, 300, 50], [1, 300, 2], [0, 0, 0], [64, 7, 1999], [2000, 300, 50]):
        lens = [min(n, k) for n, k in zip(lens, [2048, 320, 64])]
        dev[2].copy_(torch.tensor(lens, dtype=torch.int32))
        want = [B.ds4hc_latent_attn(q[2 * k], q[2 * k + 1], *dev, scale=0.07, want_lse=True) for k in range(2)]
        torch.cuda.synchronize()
        for k in range(2):
            outs[k].fill_(7), lses[k].fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k].view(torch.int16), want[k][0].view(torch.int16))
            assert torch.equal(lses[k].view(torch.int32), want[k][1].view(torch.int32))  # places never filled: NaN


# ------------------------------------------------------------------ expanded form

def check_prefill(q, kv, kr, cu_q, cu_k, scale, causal, out, lse, where=""):
    for b in range(len(cu_q) - 1):
        few, many = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        seen = torch.ones(few, many, dtype=torch.bool)
        if causal:
            seen = seen.tril(many - few)
        for h in range(q.shape[1]):
            ks, qs = slice(cu_k[b], cu_k[b + 1]), slice(cu_q[b], cu_q[b + 1])
            keys = torch.cat((kv[ks, h, :128], kr[ks]), -1)
            ref = attend64(q[qs, h], keys, kv[ks, h, 128:], seen, scale)
            assert_attention(out[qs, h], lse[qs, h], ref, seen.sum(-1), q.dtype, f"{where} sequence {b} head {h}")


def sums(v):
    return [0] + torch.tensor(v).cumsum(0).tolist()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,q_len,k_len", [(1, [1], [1]), (3, [5, 1, 70], [5, 9, 70]), (2, [129], [129]),
                                               (2, [64, 0, 1], [200, 7, 64]), (1, [300], [300]), (5, [33], [500]),
                                               (2, [8, 3], [3, 0]), (1, [257, 31], [257, 32])])
def test_prefill(dtype, causal, heads, q_len, k_len):
    say(f"[gpu] prefill {dtype} causal={causal} heads={heads} q={q_len} k={k_len}")
    g = torch.Generator().manual_seed(sum(q_len))
    cu_q, cu_k = sums(q_len), sums(k_len)
    N, S = cu_q[-1] + 2, cu_k[-1] + 3
    q, kv = torch.randn(N, heads, 192, generator=g).to(dtype), torch.randn(S, heads, 256, generator=g).to(dtype)
    wide = torch.randn(S, 576, generator=g).to(dtype)
    kv[cu_k[-1]:], wide[cu_k[-1]:] = float("nan"), float("nan")  # behind the last sequence
    out = torch.full((N, heads, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((N, heads), 7.0, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), wide.cuda()[:, 512:], i32(cu_q), i32(cu_k), scale=0.08, causal=causal,
                           out=out, lse=lse)
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()
    check_prefill(q, kv, wide[:, 512:], cu_q, cu_k, 0.08, causal, out.cpu(), lse.cpu())


def test_prefill_without_keys_and_bad_offsets():
    q = torch.randn(4, 2, 192).to(BF).cuda()
    kv, kr = torch.zeros(0, 2, 256, dtype=BF, device="cuda"), torch.zeros(0, 64, dtype=BF, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = B.ds4hc_latent_prefill(q, kv, kr, i32([0, 4]), i32([0, 0]), scale=1.0, want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    kv, kr = torch.zeros(9, 2, 256, dtype=BF, device="cuda"), torch.zeros(9, 64, dtype=BF, device="cuda")
    for cu_q, cu_k in (([0, 2, 1, 4], [0, 3, 6, 9]), ([-5, 2, 3, 4], [5, 2, 99, -1]), ([0, 1, 2, 900], [9, 9, 0, 9])):
        out = torch.full((4, 2, 128), 7.0, dtype=BF, device="cuda")
        B.ds4hc_latent_prefill(q, kv, kr, i32(cu_q), i32(cu_k), scale=1.0, out=out)
        torch.cuda.synchronize()


def test_prefill_values_that_are_not_finite_stay_with_the_rows_that_see_them():
    g = torch.Generator().manual_seed(71)
    q, kv, kr = (torch.randn(*s, generator=g).to(BF) for s in ((150, 2, 192), (150, 2, 256), (150, 64)))
    cu = [0, 70, 150]
    i32 = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for where in ("value", "key"):
        bad = kv.clone()
        bad[100, 1, 140 if where == "value" else 3] = float("nan")  # token 30 of the second sequence, head 1
        out, lse = B.ds4hc_latent_prefill(q.cuda(), bad.cuda(), kr.cuda(), i32, i32, scale=0.08, want_lse=True)
        out, lse = out.cpu(), lse.cpu()
        assert not torch.isfinite(out[100:, 1].float()).all(-1).any()
        out[100:, 1], lse[100:, 1] = 0, 0
        clean, clean_lse = B.ds4hc_latent_prefill(q.cuda(), kv.cuda(), kr.cuda(), i32, i32, scale=0.08, want_lse=True)
        clean, clean_lse = clean.cpu(), clean_lse.cpu()
        clean[100:, 1], clean_lse[100:, 1] = 0, 0
        check_prefill(q[:100], kv[:100], kr[:100], [0, 70], [0, 70], 0.08, True, out[:100], lse[:100])
        assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


def test_prefill_in_a_captured_graph():
    g = torch.Generator().manual_seed(73)
    q, kv, kr = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((300, 2, 192), (300, 2, 256), (300, 64)))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    out, lse = torch.empty(300, 2, 128, dtype=BF, device="cuda"), torch.empty(300, 2, device="cuda")
    call = lambda: B.ds4hc_latent_prefill(q, kv, kr, cu, cu, scale=0.08, out=out, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for middle in (100, 1, 299, 150):
        cu.copy_(torch.tensor([0, middle, 300], dtype=torch.int32))
        want = B.ds4hc_latent_prefill(q, kv, kr, cu, cu, scale=0.08, want_lse=True)
        out.fill_(7), lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ together

def test_an_attention_site_prompt_then_decode_and_a_drafted_tree():
    """One attention site as it is used: HC-pre, projections, rotation, append, attention,
    post update; a prompt through the expanded form, then tokens through the absorbed one
    over the cache the prompt filled. The decoded rows are held against the expanded form
    in 64 bits on the same cached vectors."""
    g = torch.Generator().manual_seed(83)
    H, d, page, T = 8, 256, 16, 45
    r = lambda *s, size=1.0: torch.randn(*s, generator=g) * size  # noqa: E731
    W = (r(24, 4 * d, size=0.02)).to(HF).cuda()
    bias = torch.zeros(24).cuda()
    Wq, Wkv = r(d, H * 192, size=d ** -0.5).cuda(), r(d, 576, size=d ** -0.5).cuda()
    Wk, Wv = r(H, 512, 128, size=512 ** -0.5).cuda(), r(H, 512, 128, size=512 ** -0.5).cuda()
    Wo = r(H * 128, d, size=(H * 128) ** -0.5).cuda()
    f, amp = B.ds4hc_rope_frequencies(64, factor=4.0, original_length=4096, device="cuda")
    weight, scale = torch.ones(512).cuda(), 192 ** -0.5
    cache = torch.full((8, page, 576), float("nan"), dtype=BF, device="cuda")
    table = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def site(X, positions, length, attention):
        layer_in, coeffs, _ = B.ds4hc_pre(X, W, bias)
        N = X.shape[0]
        q = (layer_in @ Wq).to(BF).view(N, H, 192)
        B.ds4hc_latent_append(layer_in @ Wkv, positions, f, cache, i32([0, N]), i32([length]), table, norm_weight=weight,
                              amplitude=amp)
        B.ds4hc_rope(q[..., 128:], positions, f, amplitude=amp, out=q[..., 128:])
        o = attention(q)  # [N, H, 128]
        return q, o, B.ds4hc_post(X, coeffs, (o.reshape(N, H * 128).float() @ Wo).contiguous())

    def cached(n):
        j = torch.arange(n, device="cuda")
        return cache[table[0, j // page].long(), j % page]

    def expand(n):
        rows = cached(n)
        c = rows[:, :512].float()
        kv = torch.cat([torch.stack([c @ w[h] for h in range(H)], 1) for w in (Wk, Wv)], -1).to(BF).contiguous()
        return kv, rows[:, 512:]

    def prompt(q):
        kv, kr = expand(T)
        return B.ds4hc_latent_prefill(q, kv, kr, i32([0, T]), i32([0, T]), scale=scale)[0]

    def absorbed(length, tree=None):
        def attention(q):
            N = q.shape[0]
            ql = torch.stack([q[:, h, :128].float() @ Wk[h].T for h in range(H)], 1).to(BF)
            o = B.ds4hc_latent_attn(ql, q[..., 128:], cache, i32([0, N]), i32([length]), table, scale=scale,
                                    tree_mask=tree)[0]
            return torch.stack([o[:, h].float() @ Wv[h] for h in range(H)], 1)
        return attention

    def reference(q, n, seen):
        rows = cached(n).double().cpu()
        res = []
        for h in range(H):
            k = torch.cat((rows[:, :512] @ Wk[h].double().cpu(), rows[:, 512:]), -1)
            res.append(attend64(q[:, h].cpu(), k, rows[:, :512] @ Wv[h].double().cpu(), seen, scale)[0])
        return torch.stack(res, 1)

    X = r(T, 4, d).cuda()
    q, o, X1 = site(X, torch.arange(T, device="cuda"), T, prompt)
    assert torch.isfinite(X1).all()
    # bfloat16 keys (512-term products rounded once), weights and values: a few roundings of 2^-8 a term
    tol = 6 * 2.0 ** -8
    ref = reference(q, T, torch.ones(T, T, dtype=torch.bool).tril())
    assert ((o.double().cpu() - ref).norm(dim=-1) <= tol * ref.norm(dim=-1)).all()
    X = r(1, 4, d).cuda()
    q, o, X1 = site(X, torch.tensor([T], device="cuda"), T + 1, absorbed(T + 1))
    ref = reference(q, T + 1, torch.ones(1, T + 1, dtype=torch.bool))
    assert ((o.double().cpu() - ref).norm(dim=-1) <= tol * ref.norm(dim=-1)).all()
    # a tree of four drafts: 0 - 1 - 3 and 0 - 2; siblings share a position
    tree = torch.tensor([[1], [3], [5], [11]], device="cuda")
    X = r(4, 4, d).cuda()
    q, o, X1 = site(X, torch.tensor([0, 1, 1, 2], device="cuda") + T + 1, T + 5, absorbed(T + 5, tree))
    seen = torch.ones(4, T + 5, dtype=torch.bool)
    seen[:, T + 1:] = torch.tensor([[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]).bool()
    ref = reference(q, T + 5, seen)
    assert ((o.double().cpu() - ref).norm(dim=-1) <= tol * ref.norm(dim=-1)).all()
    assert torch.isfinite(X1).all()
