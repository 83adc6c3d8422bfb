"""The operators around the attention of drafted tokens on the GPU: verification, moves of rows, pages, and a serving step
of all of them, against plain references."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from serve_testlib import Pool, compact_rows, distributions, random_trees, sums_of, verify64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ verification

def check_verify(target, tokens, cu, uniform, draft=None, parents=None, **kw):
    """Whole numbers have to be equal. (A number that chooses the next token may lie so near a border that sums of 64 bits
    in another order fall on its other side: 2^-53 a term and 2^17 terms make 2e-11 of the total at most.)"""
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = B.ds4hc_draft_verify(d(target), d(tokens), i32(cu), d(uniform), draft=d(draft), parents=d(parents), **kw)
    path, kept, following, margin = verify64(target, tokens, cu, uniform, draft, parents)
    for t, p in enumerate(path):
        if p is not None:
            assert got[0][t].item() == p, (t, p, got[0].tolist()[:20])
    assert got[1].tolist() == kept
    for b, (x, m) in enumerate(zip(following, margin)):
        assert got[2][b].item() == x or m < 2e-11, (b, x, got[2][b].item(), m)
    return got


@pytest.mark.parametrize("q_len,vocab", [([1], 1), ([2], 2), ([5, 1, 0, 3], 7), ([9] * 7, 1000), ([5, 2, 8, 1], 32768),
                                         ([3, 6], 100003), ([2] * 130, 257), ([70, 200], 50), ([65, 64, 129], 33),
                                         ([4] * 33, 40001)])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_chains(q_len, vocab, with_draft):
    say(f"[gpu] verify chains {q_len[:8]} vocab={vocab} draft={with_draft}")
    g = torch.Generator().manual_seed(len(q_len) * 1000 + vocab)
    n, cu = sum(q_len), sums_of(q_len)
    for near in (0.2, 1.5):  # most are kept, few are kept
        target, draft = distributions(g, n, vocab, near=near)
        tokens = torch.multinomial(draft, 1, generator=g)[:, 0].roll(1)
        uniform = torch.rand(n, generator=g)
        check_verify(target, tokens, cu, uniform, draft if with_draft else None)


@pytest.mark.parametrize("q_len,vocab", [([2], 5), ([40, 1, 0, 17], 300), ([64] * 5, 32000), ([65, 130], 100), ([9] * 40, 5000),
                                         ([1000, 1024], 64)])
def test_verify_trees(q_len, vocab):
    say(f"[gpu] verify trees {q_len[:8]} vocab={vocab}")
    g = torch.Generator().manual_seed(len(q_len) + vocab)
    n, cu = sum(q_len), sums_of(q_len)
    target, _ = distributions(g, n, vocab)
    trees = random_trees(g, q_len)
    parents = torch.tensor([p for t in trees for p in t], dtype=torch.int32)
    for likely in (True, False):  # a token's children: its most likely followers, then any, some of them twice
        tokens = torch.randint(0, vocab, (n,), generator=g)
        if likely:
            best = target.topk(min(vocab, 32), -1).indices
            for b, t in enumerate(trees):
                for i, p in enumerate(t):
                    if p >= 0:
                        tokens[cu[b] + i] = best[cu[b] + p, t[:i].count(p) % best.shape[1]]
        check_verify(target, tokens, cu, torch.rand(n, generator=g), None, parents)


def test_verify_takes_rows_with_strides_and_leaves_the_rest():
    """Rows inside wider ones, off 16-byte boundaries; entries behind the last sequence stay as they were."""
    g = torch.Generator().manual_seed(5)
    target, draft = distributions(g, 9, 1001)
    tokens = torch.multinomial(draft, 1, generator=g)[:, 0].roll(1).cuda()
    uniform = torch.rand(9, generator=g).cuda()
    cu = i32([0, 4, 7])
    want = B.ds4hc_draft_verify(target.cuda(), tokens, cu, uniform, draft=draft.cuda())
    wide = torch.full((9, 2100), math.nan, device="cuda")
    wide[:, 3:1004], wide[:, 1050:2051] = target.cuda(), draft.cuda()
    path = torch.full((9,), 55, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = B.ds4hc_draft_verify(wide[:, 3:1004], tokens, cu, uniform, draft=wide[:, 1050:2051], path=path, stream=side)
    side.synchronize()
    assert torch.equal(got[0][:7], want[0][:7]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert (path[7:] == 55).all()


def test_verify_where_weights_end():
    """Equal distributions (nothing is left when one is rejected), rows with one weight, without any, with values that are
    not finite or negative; tokens and parents that are none; numbers at the ends of their range."""
    inf, nan = math.inf, math.nan
    v = 8
    p = torch.full((6, v), 1 / v)
    chain = lambda **kw: check_verify(**{**dict(target=p, tokens=torch.tensor([0, 1, 2, 3, 4, 5]), cu=[0, 3, 6],  # noqa: E731
                                                uniform=torch.full((6,), 0.5)), **kw})
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, nan):
        for draft in (None, p, p * 2, p / 2):
            chain(uniform=torch.full((6,), u), draft=draft)
    # p = q and a number that rejects: q * u < p fails only at u = 1, which is taken as the number before it
    one = torch.zeros(6, v)
    one[:, 3] = 1.0
    for draft in (None, p, one):
        chain(target=one, draft=draft)
        chain(target=one, draft=draft, tokens=torch.full((6,), 3))
    got = chain(target=torch.zeros(6, v))
    assert got[2].tolist() == [-1, -1] and got[1].tolist() == [1, 1]
    odd = torch.tensor([[0.1, nan, inf, -0.5, 0.2, 0.0, 0.3, -inf]]).repeat(6, 1)
    for x in range(v):
        chain(target=odd, tokens=torch.full((6,), x), draft=None if x % 2 else p)
    chain(tokens=torch.tensor([0, -1, 2, 0, v, 1 << 40]), draft=p)
    chain(tokens=torch.tensor([0, -(1 << 62), 2, 0, v, 1 << 40]))
    for parents in ([-1, 5, 0, -1, -7, 0], [3, 1, 2, 9, 0, 1], [0, 0, 0, 0, 0, 0], [-1, 0, 1 << 30, 0, 1, 1]):
        chain(parents=torch.tensor(parents, dtype=torch.int32))


@pytest.mark.parametrize("cu", [[0, 4, 2, 6], [-3, 2, 4, 6], [0, 2, 4, 99], [6, 6, 6, 6], [5, 3, 1, 0]])
def test_verify_survives_bad_offsets(cu):
    """Offsets that fall, are negative or pass the tokens: inside the arrays, and nothing for what is empty."""
    g = torch.Generator().manual_seed(3)
    target, draft = distributions(g, 6, 100)
    path = torch.full((6,), 55, dtype=torch.int32, device="cuda")
    got = B.ds4hc_draft_verify(target.cuda(), torch.randint(0, 100, (6,), generator=g).cuda(), i32(cu),
                               torch.rand(6, generator=g).cuda(), draft=draft.cuda(), path=path)
    clamped = [min(max(c, 0), 6) for c in cu]
    for b in range(3):
        few = max(clamped[b + 1] - clamped[b], 0)
        assert (got[1][b].item() == 0 and got[2][b].item() == -1) if few == 0 else 1 <= got[1][b].item() <= few
    inside = set()
    for a, b in zip(clamped, clamped[1:]):
        inside |= set(range(a, b))
    assert all(path[t].item() == 55 for t in set(range(6)) - inside)


def test_verify_more_tokens_than_are_looked_at():
    """Tokens at and behind 1024 are not accepted, of a chain (all before them are) and of a tree."""
    n, v = 1030, 4
    target = torch.zeros(n, v)
    target[:, 2] = 1.0
    tokens, uniform = torch.full((n,), 2), torch.full((n,), 0.5)
    for kw in (dict(), dict(draft=target), dict(parents=torch.arange(-1, n - 1, dtype=torch.int32))):
        got = check_verify(target, tokens, [0, n], uniform, **kw)
        assert got[1].item() == 1024 and got[2].item() == 2
        assert got[0][1023].item() == 1023 and (got[0][1024:] == -1).all()


def test_verify_keeps_the_targets_distribution():
    """The first token that a sequence gains (its drafted one if that is kept, else the next) is distributed as the target,
    whatever the draft: counts of 40000 sequences within 5 standard deviations, sqrt(n p (1 - p)), for each of 6 tokens."""
    g = torch.Generator().manual_seed(9)
    n, v = 40000, 6
    p = torch.tensor([0.4, 0.25, 0.2, 0.1, 0.04, 0.01])
    q = torch.tensor([0.05, 0.5, 0.1, 0.1, 0.05, 0.2])
    cu = i32(list(range(0, 2 * n + 1, 2)))
    uniform = torch.rand(2 * n, generator=g).cuda()
    drawn = torch.multinomial(q, n, replacement=True, generator=g)
    tokens = torch.stack((torch.zeros_like(drawn), drawn), 1).flatten().cuda()
    target, draft = p.repeat(2 * n, 1).cuda(), q.repeat(2 * n, 1).cuda()
    for kw in (dict(draft=draft), dict()):
        _, kept, following = B.ds4hc_draft_verify(target, tokens, cu, uniform, **kw)
        first = torch.where(kept == 2, tokens[1::2], following).cpu()
        count = torch.bincount(first, minlength=v).double()
        assert ((count - n * p).abs() <= 5 * (n * p * (1 - p)).sqrt()).all(), count
    # trees of two children
    cu3 = i32(list(range(0, 3 * n + 1, 3)))
    two = torch.tensor([0, 4, 1]).repeat(n).cuda()
    parents = i32([-1, 0, 0]).repeat(n)
    path, kept, following = B.ds4hc_draft_verify(p.repeat(3 * n, 1).cuda(), two, cu3, torch.rand(3 * n, generator=g).cuda(),
                                                 parents=parents)
    child = path.view(n, 3)[:, 1]
    first = torch.where(kept == 2, torch.where(child == 1, 4, 1), following).cpu()
    count = torch.bincount(first, minlength=v).double()
    assert ((count - n * p).abs() <= 5 * (n * p * (1 - p)).sqrt()).all(), count


def test_verify_without_tokens_and_without_sequences():
    empty = torch.empty(0, 5, device="cuda")
    no = torch.empty(0, dtype=torch.int64, device="cuda")
    got = B.ds4hc_draft_verify(empty, no, i32([0, 0, 0]), torch.empty(0, device="cuda"))
    assert got[1].tolist() == [0, 0] and got[2].tolist() == [-1, -1]
    got = B.ds4hc_draft_verify(torch.ones(3, 5, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0]),
                               torch.zeros(3, device="cuda"))
    assert got[1].shape == (0,)


# ------------------------------------------------------------------ moves

@pytest.mark.parametrize("shape,dtype", [((1, 8), torch.float32), ((3, 656), torch.uint8), ((5, 576), torch.bfloat16),
                                         ((2, 4096), torch.int32), ((43, 16), torch.uint8)])
@pytest.mark.parametrize("page", [1, 4, 64])
def test_compact(shape, dtype, page):
    say(f"[gpu] compact {shape} {dtype} page={page}")
    g = torch.Generator().manual_seed(page)
    layers, row = shape
    q_len, context = [1, 0, 70, 9, 200, 3], [5, 3, 0, 64, 31, 130]
    lens = [q + c for q, c in zip(q_len, context)]
    cu = sums_of(q_len)
    need = [-(-k // page) for k in lens]
    n_pages, most = sum(need) + 2, max(need)
    order = torch.randperm(n_pages, generator=g).tolist()
    table = [[order.pop() for _ in range(k)] + [-1] * (most - k) for k in need]
    keep, n_keep = [-9] * (cu[-1] + 2), []
    for b, q in enumerate(q_len):
        k = min(q, [1, 0, 33, 9, 150, 2][b])
        keep[cu[b]:cu[b] + k] = sorted(torch.randperm(q, generator=g)[:k].tolist())
        n_keep.append(k)
    size = row * torch.empty(0, dtype=dtype).element_size()
    cache = torch.randint(0, 256, (layers, n_pages, page, size), generator=g, dtype=torch.uint8)
    ref = cache.clone().view(layers, -1, size)
    compact_rows(ref, table, page, cu, lens, keep, n_keep, most)
    dev = cache.cuda().view(dtype)
    got = B.ds4hc_cache_compact(dev, i32(cu), i32(lens), i32(table), i32(keep), i32(n_keep))
    assert got is dev
    assert torch.equal(dev.view(torch.uint8).cpu().view(layers, -1, size), ref)
    one = cache[0].cuda().view(dtype)  # a cache without the dimension of the layers
    B.ds4hc_cache_compact(one, i32(cu), i32(lens), i32(table), i32(keep), i32(n_keep))
    assert torch.equal(one.view(torch.uint8).cpu().view(-1, size), ref[0])


def test_compact_passes_over_what_is_not_there():
    """Entries outside the call's tokens, places before token 0 and in pages that are not in the cache, more kept than there
    are tokens, lengths behind the table: nothing else moves."""
    cache = torch.arange(8 * 4 * 16, dtype=torch.int64).to(torch.uint8).view(1, 8, 4, 16)
    table = [[0, 1], [2, -1], [99, 3], [4, 5]]
    q_len, lens = [3, 5, 4, 6], [8, 7, 8, 900]
    cu, keep, n_keep = sums_of(q_len), [-1, 2, 7] + [1, 3, 4, 0, 0] + [1, 2, 3, 9] + [0, 2, 3, 4, 5, 6], [3, 9, 4, 5]
    ref = cache.clone().view(1, 32, 16)
    compact_rows(ref, table, 4, cu, lens, keep, n_keep, 2)
    dev = cache.cuda()
    B.ds4hc_cache_compact(dev, i32(cu), i32(lens), i32(table), i32(keep), i32(n_keep))
    assert torch.equal(dev.cpu().view(1, 32, 16), ref)
    before = dev.clone()
    short = [1, 2, 3, 4]  # fewer tokens than the call's: places before token 0
    B.ds4hc_cache_compact(dev, i32(cu), i32(short), i32([[-1, -1]] * 4), i32(keep), i32([-5, 0, 3, 3]))
    assert torch.equal(dev, before)


def test_compact_moves_no_row_up():
    """A list that rises from an entry below 0 has entries smaller than their places: no row goes to a later place, where it
    would meet rows that are still to be moved, and those that follow are moved as ever."""
    page, few = 16, 40
    cache = torch.arange(4 * page * 16).remainder(251).to(torch.uint8).view(1, 4, page, 16)
    for keep, moves in ((list(range(-1, few - 1)), []), (list(range(-20, few - 20)), []),
                        ([-3, -2, -1, 0, 1, 5, 6, 9] + list(range(20, 40)), [(6, 6), (7, 9)] + [(8 + i, 20 + i) for i in range(20)])):
        ref = cache.clone().view(-1, 16)
        for to, source in moves:
            ref[10 + to] = cache.view(-1, 16)[10 + source]
        dev = cache.cuda()
        B.ds4hc_cache_compact(dev, i32([0, few]), i32([few + 10]), i32([[0, 1, 2, 3]]), i32(keep + [0] * (few - len(keep))),
                              i32([len(keep)]))
        assert torch.equal(dev.cpu().view(-1, 16), ref)


def test_compact_offsets_past_32_bits():
    """Layers far apart (their strides pass 2^32 bytes) and rows past 2^32 bytes within one."""
    n_pages, page = 60000, 64
    cache = torch.zeros(2, n_pages, page, 1152, dtype=torch.uint8, device="cuda")
    last = n_pages - 1
    cache[:, last, 10] = torch.tensor([5, 6], dtype=torch.uint8, device="cuda")[:, None]
    B.ds4hc_cache_compact(cache, i32([0, 4]), i32([11]), i32([[last]]), i32([0, 3, 0, 0]), i32([2]))
    assert (cache[0, last, 8] == 5).all() and (cache[1, last, 8] == 6).all() and cache.sum(dtype=torch.int64) == 2 * 11 * 1152
    B.ds4hc_pages_copy(cache, i32([[last, 1]]))
    assert torch.equal(cache[:, 1], cache[:, last])


@pytest.mark.parametrize("layers,page,row,dtype", [(1, 1, 16, torch.uint8), (3, 64, 656, torch.uint8), (2, 16, 576, torch.bfloat16),
                                                   (43, 2, 36, torch.int32)])
def test_pages_copy(layers, page, row, dtype):
    g = torch.Generator().manual_seed(row)
    size = row * torch.empty(0, dtype=dtype).element_size()
    wide = torch.randint(0, 256, (layers, 25, page, size), generator=g, dtype=torch.uint8).cuda()
    cache = wide.view(dtype)[:, :20]  # layers that do not lie one behind another
    pairs = [[3, 7], [-1, -1], [3, 8], [0, 20], [25, 1], [-4, 2], [5, 5], [19, 0], [12, -1]]
    ref = wide.clone()
    for a, b in ([3, 7], [3, 8], [19, 0]):
        ref[:, b] = ref[:, a]
    assert B.ds4hc_pages_copy(cache, i32(pairs)) is cache
    assert torch.equal(wide, ref)
    B.ds4hc_pages_copy(cache, i32(pairs)[:0])
    assert torch.equal(wide, ref)


# ------------------------------------------------------------------ pages

def same(pool, dev):
    for want, got in zip(pool.tensors(), dev):
        assert torch.equal(want, got.cpu())


@pytest.mark.parametrize("slots,max_pages,pages,page", [(5, 6, 12, 4), (40, 20, 300, 1), (300, 9, 40000, 16), (1100, 3, 5000, 2),
                                                        (3, 700, 1500, 64)])
def test_pages_follow_the_model(slots, max_pages, pages, page):
    """Random lengths and forks, some of them refused for want of pages: tables, lengths, counts, copies and what became of
    each item as in the model, which counts every page."""
    say(f"[gpu] pages slots={slots} max={max_pages} pages={pages} page={page}")
    g = torch.Generator().manual_seed(slots)
    pick = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=g).tolist()  # noqa: E731
    pool = Pool(slots, max_pages, pages, page)
    dev = pool.tensors("cuda")
    short = copied = 0
    for turn in range(24):
        if turn % 3 == 2:
            n = pick(1, slots + 1, 1)[0]
            empty = [s for s in range(slots) if pool.lens[s] == 0]
            children = [empty[i % len(empty)] if empty and i % 5 else s for i, s in enumerate(pick(-1, slots + 1, n))]
            parents = pick(-1, slots + 1, n)
            status = pool.fork(parents, children)
            got = B.ds4hc_pages_fork(*dev, page, i32(parents), i32(children))
            assert got.tolist() == status
        else:
            n = pick(1, slots + 3, 1)[0]
            which = pick(-1, slots + 1, n) if turn % 2 else torch.randperm(slots, generator=g)[:n].tolist()
            lens = [0 if k % 3 == 0 else k for k in pick(-1, max_pages * page + 2, len(which))]
            if turn % 4 == 1:  # a few tokens more
                lens = [(pool.lens[s] if 0 <= s < slots else 0) + d for s, d in zip(which, pick(0, 3, len(which)))]
            copies, status = pool.resize(which, lens)
            got, what = B.ds4hc_pages_resize(*dev, page, i32(which), i32(lens))
            assert got.tolist() == copies and what.tolist() == status
            short += status.count(1)
            copied += sum(c[0] >= 0 for c in copies)
        pool.check()
        same(pool, dev)
    say(f"[gpu] short {short}, copies {copied}")


def test_pages_all_share_one_and_all_grow():
    """Every holder of a shared last page that grows in one call gets its own, and the page is free afterwards."""
    pool = Pool(6, 4, 20, 4)
    dev = pool.tensors("cuda")
    for op, a, b in (("resize", [0], [6]), ("fork", [0] * 5, [1, 2, 3, 4, 5]), ("resize", [5, 3, 0, 1, 2, 4], [7, 7, 8, 9, 7, 13])):
        if op == "fork":
            pool.fork(a, b)
            B.ds4hc_pages_fork(*dev, 4, i32(a), i32(b))
        else:
            copies, _ = pool.resize(a, b)
            got, _ = B.ds4hc_pages_resize(*dev, 4, i32(a), i32(b))
            assert got.tolist() == copies
        pool.check()
        same(pool, dev)
    assert pool.refs[1] == 0 and pool.refs[0] == 6


def test_pages_a_pool_of_a_quarter_million():
    """Free pages at the far end of a large pool, found in ascending order; slots that end with many pages each."""
    page, pages = 16, 260001
    pool = Pool(9, 30000, pages, page)
    lens = [29000 * page] * 8 + [0]
    pool.resize(list(range(9)), lens)
    dev = pool.tensors("cuda")
    for which, new in (([8, 2], [400000, 5]), ([2, 8, 0], [464000, 0, 1]), ([0, 1, 3, 4, 5, 6, 7], [0] * 7), ([8], [480000])):
        want = pool.resize(which, new)
        got = B.ds4hc_pages_resize(*dev, page, i32(which), i32(new))
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        same(pool, dev)


def test_pages_survive_a_broken_pool():
    """Tables, lengths and counts that contradict one another: no access outside them (entries that are no page are left
    out, lengths are cut to the table's)."""
    table = i32([[7, -3, 1 << 30], [99, 0, 1], [2, 2, 2]])
    lens, refs = i32([1 << 30, 5, -7]), i32([1, -5, 3, 0, 0, 0, 0, 2])
    slots = i32([0, 1, 2])
    for new in ([0, 0, 0], [9, 6, 12], [12, 12, 1], [1, 2, 3]):
        B.ds4hc_pages_resize(table, lens, refs, 4, slots, i32(new))
    B.ds4hc_pages_fork(table, lens, refs, 4, i32([0, 1]), i32([2, 2]))
    torch.cuda.synchronize()


def test_pages_and_verify_in_a_graph():
    """Captured resize, fork, copy, verify and compact, replayed with other contents, with eager work between: as eager. All
    share one workspace, on one stream."""
    page = 4
    g = torch.Generator().manual_seed(2)
    pool = Pool(4, 8, 24, page)
    table, lens, refs = pool.tensors("cuda")
    cache = torch.randint(0, 256, (3, 24, page, 32), generator=g, dtype=torch.uint8).cuda()
    cu = i32([0, 5, 8])
    tokens, uniform = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, device="cuda")
    target = torch.zeros(8, 300, device="cuda")
    slots, grown, less, none = i32([0, 1]), i32([0, 0]), i32([0, 0]), i32([0, 0])
    copies, status = i32([[0, 0]] * 2), i32([0, 0])
    path, kept, following = i32([0] * 8), i32([0] * 2), torch.zeros(2, dtype=torch.int64, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        B.ds4hc_pages_resize(table, lens, refs, page, slots, grown, copies=copies, status=status, workspace=ws)
        B.ds4hc_pages_copy(cache, copies)
        B.ds4hc_draft_verify(target, tokens, cu, uniform, path=path, n_kept=kept, next_token=following, workspace=ws)
        B.ds4hc_cache_compact(cache, cu, lens[:2], table[:2], path, kept)
        B.ds4hc_pages_resize(table, lens, refs, page, slots, less, copies=copies, status=status, workspace=ws)
        B.ds4hc_pages_resize(table, lens, refs, page, i32_2, none, status=status, copies=copies, workspace=ws)
        B.ds4hc_pages_fork(table, lens, refs, page, slots, i32_2, status=status, workspace=ws)

    i32_2 = i32([2, 3])
    state = (table, lens, refs, cache, copies, path, kept, following)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        p, _ = distributions(g, 8, 300)
        target.copy_(p)
        tokens.copy_(torch.multinomial(p, 1, generator=g)[:, 0].roll(1))
        uniform.copy_(torch.rand(8, generator=g))
        grown.copy_(torch.tensor([10 + turn, 13 - turn], dtype=torch.int32))
        less.copy_(torch.tensor([7 + turn, 12 - turn], dtype=torch.int32))
        saved = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in state]
        for t, old in zip(state, saved):
            t.copy_(old)
        step()
        torch.cuda.synchronize()
        for a, b in zip(state, replayed):
            assert torch.equal(a, b)


def test_verify_two_at_once():
    """Two calls side by side on two streams, each with a workspace of its own: as one after another."""
    g = torch.Generator().manual_seed(3)
    both = []
    for q_len in ([5] * 20, [3, 9, 1]):
        n = sum(q_len)
        p, q = distributions(g, n, 9000)
        both.append(((p.cuda(), torch.randint(0, 9000, (n,), generator=g).cuda(), i32(sums_of(q_len)), torch.rand(n, generator=g).cuda()),
                     dict(draft=q.cuda())))
    want = [B.ds4hc_draft_verify(*a, **kw) for a, kw in both]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [B.ds4hc_draft_verify(*a, **kw, stream=s) for (a, kw), s in zip(both, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for one, other in zip(got, want) for x, y in zip(one, other))


def test_refusals_of_the_binding():
    dev = "cuda"
    target, tokens, cu, u = torch.zeros(4, 9, device=dev), torch.zeros(4, dtype=torch.int64, device=dev), i32([0, 2, 4]), torch.zeros(4, device=dev)
    small = torch.zeros(16, dtype=torch.uint8, device=dev)
    for call in (lambda: B.ds4hc_draft_verify(target.half(), tokens, cu, u), lambda: B.ds4hc_draft_verify(target.t(), tokens, cu, u),
                 lambda: B.ds4hc_draft_verify(target, tokens.int(), cu, u), lambda: B.ds4hc_draft_verify(target, tokens[:3], cu, u),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, draft=target, parents=i32([0] * 4)),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, draft=target[:, :8]),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, n_kept=i32([0])),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, workspace=small),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu.cpu(), u),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, path=tokens),
                 lambda: B.ds4hc_draft_verify(target, tokens, cu, u, n_kept=cu[:2])):
        with pytest.raises((TypeError, ValueError, B.Ds4hcError)):
            call()
    cache = torch.zeros(2, 8, 4, 32, device=dev)
    table, lens, refs = i32([[-1, -1]] * 2), i32([0, 0]), i32([0] * 8)
    for call in (lambda: B.ds4hc_cache_compact(cache[..., :30], cu, lens, table, tokens.int(), lens),
                 lambda: B.ds4hc_cache_compact(cache[..., :3].contiguous(), cu, lens, table, tokens.int(), lens),
                 lambda: B.ds4hc_cache_compact(cache[:, :, :3].contiguous(), cu, lens, table, tokens.int(), lens),
                 lambda: B.ds4hc_cache_compact(cache[0, 0], cu, lens, table, tokens.int(), lens),
                 lambda: B.ds4hc_cache_compact(cache, cu, lens, table, tokens, lens),
                 lambda: B.ds4hc_cache_compact(cache[:0], cu, lens, table, tokens.int(), lens),
                 lambda: B.ds4hc_pages_copy(cache, tokens.int()), lambda: B.ds4hc_pages_copy(cache, tokens.view(2, 2)),
                 lambda: B.ds4hc_pages_copy(cache.transpose(1, 2), i32([[0, 1]])),
                 lambda: B.ds4hc_pages_resize(table, lens, refs, 3, i32([0]), i32([1])),
                 lambda: B.ds4hc_pages_resize(table, lens, refs, 4, i32([0]), i32([1, 2])),
                 lambda: B.ds4hc_pages_resize(table, lens[:1], refs, 4, i32([0]), i32([1])),
                 lambda: B.ds4hc_pages_resize(table, lens, refs, 4, i32([0]), lens[:1]),
                 lambda: B.ds4hc_pages_resize(table, lens, refs, 4, i32([0]), i32([1]), workspace=small),
                 lambda: B.ds4hc_pages_fork(table, lens, refs, 4, i32([0]), i32([1]).long()),
                 lambda: B.ds4hc_pages_fork(table.t(), lens, refs, 4, i32([0]), i32([1]))):
        with pytest.raises((TypeError, ValueError, B.Ds4hcError)):
            call()
    assert (lens == 0).all() and (refs == 0).all() and (table == -1).all()


# ------------------------------------------------------------------ all of them

@pytest.mark.parametrize("trees", [False, True])
def test_a_serving_step(trees):
    """Room for the drafts, append, attention, verification, compaction, the accepted lengths: after it every layer's cache
    holds, for every sequence, its context and the accepted tokens' rows in order, and an attention over it has the bits that it
    has over a cache to which the same tokens were appended one call after another."""
    g = torch.Generator().manual_seed(17)
    layers, page, seqs, few, heads, vocab, d = 3, 16, 4, 6, 16, 500, 128
    pool = Pool(seqs, 12, 60, page)
    dev = table, lens, refs = pool.tensors("cuda")
    caches = torch.zeros(layers, 60, page, d + 144, dtype=torch.uint8, device="cuda")
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    every = i32(list(range(seqs)))
    context = [33, 0, 16, 90]
    B.ds4hc_pages_resize(*dev, page, every, i32(context))
    rows = torch.randn(layers, sum(context), d + 64, generator=g).to(torch.bfloat16).cuda()
    at = torch.cat([torch.arange(k) for k in context]).cuda()
    for layer in range(layers):
        B.ds4hc_latent_append8(rows[layer], at, f, caches[layer], i32(sums_of(context)), lens, table)
    known = [[rows[layer, a:b] for a, b in zip(sums_of(context), sums_of(context)[1:])] for layer in range(layers)]
    positions = [list(range(k)) for k in context]
    for turn in range(5):
        cu = i32([few * b for b in range(seqs + 1)])
        old = lens.tolist()
        copies, status = B.ds4hc_pages_resize(*dev, page, every, i32([k + few for k in old]))
        assert (status == 0).all() and (copies == -1).all()
        tree = random_trees(g, [few] * seqs) if trees else [list(range(-1, few - 1))] * seqs
        depth = []
        for t in tree:
            deep = [0] * few
            for i in range(1, few):
                deep[i] = deep[t[i]] + 1
            depth.append(deep)
        mask = []
        for t in tree:
            seen = []
            for i, p in enumerate(t):
                seen.append((1 << i) | (seen[p] if p >= 0 else 0))
            mask += [[s] for s in seen]
        new = torch.randn(layers, seqs * few, d + 64, generator=g).to(torch.bfloat16).cuda()
        pos = torch.tensor([old[b] + depth[b][i] for b in range(seqs) for i in range(few)]).cuda()
        ql = torch.randn(seqs * few, heads, d, generator=g).to(torch.bfloat16).cuda()
        qr = torch.randn(seqs * few, heads, 64, generator=g).to(torch.bfloat16).cuda()
        for layer in range(layers):
            B.ds4hc_latent_append8(new[layer], pos, f, caches[layer], cu, lens, table)
            B.ds4hc_latent_attn8(ql, qr, caches[layer], cu, lens, table, scale=0.1, tree_mask=torch.tensor(mask).cuda())
        target, _ = distributions(g, seqs * few, vocab)
        best = target.topk(few, -1).indices
        tokens = torch.tensor([0 if p < 0 else int(best[b * few + p, t[:i].count(p)]) for b, t in enumerate(tree)
                               for i, p in enumerate(t)]).cuda()
        parents = i32([p for t in tree for p in t]) if trees else None
        path, kept, _ = B.ds4hc_draft_verify(target.cuda(), tokens, cu, torch.rand(seqs * few, generator=g).cuda(),
                                             parents=parents)
        B.ds4hc_cache_compact(caches, cu, lens, table, path, kept)
        length = torch.tensor(old, dtype=torch.int32, device="cuda") + kept
        B.ds4hc_pages_resize(*dev, page, every, length)
        assert torch.equal(lens, length)
        for b in range(seqs):
            way = path.tolist()[b * few:b * few + kept.tolist()[b]]
            for layer in range(layers):
                known[layer][b] = torch.cat((known[layer][b], new[layer, [b * few + w for w in way]]))
            positions[b] += [old[b] + depth[b][w] for w in way]
    # afresh: everything that is known, in one append a layer, to pages of its own
    total = lens.tolist()
    assert total == [len(p) for p in positions]
    plain = torch.zeros_like(caches[0])
    own, have = torch.full((seqs, 12), -1, dtype=torch.int32), 0
    for b, k in enumerate(total):
        pages = -(-k // page)
        own[b, :pages] = torch.arange(have, have + pages, dtype=torch.int32)
        have += pages
    for layer in range(layers):
        plain.zero_()
        B.ds4hc_latent_append8(torch.cat(known[layer]), torch.tensor([p for q in positions for p in q]).cuda(), f, plain,
                               i32(sums_of(total)), lens, own.cuda())
        ql = torch.randn(seqs, heads, d, generator=g).to(torch.bfloat16).cuda()
        qr = torch.randn(seqs, heads, 64, generator=g).to(torch.bfloat16).cuda()
        a, b = (B.ds4hc_latent_attn8(ql, qr, c, i32(list(range(seqs + 1))), lens, t, scale=0.1, want_lse=True)
                for c, t in ((caches[layer], table), (plain, own.cuda())))
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
