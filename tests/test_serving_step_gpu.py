"""A serving step with drafts while the pool of pages runs out: what is refused stays as it was."""
import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from serve_testlib import Pool, distributions, random_trees, sums_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("eight", [True, False])
@pytest.mark.parametrize("trees", [False, True])
def test_a_step_that_finds_too_few_pages(trees, eight):
    """Six sequences want room for 6 tokens each. There is one free page: the first takes it, for its copy of the last page
    that it shares with the second; the second and the third get none, the fourth would pass its table, the others need none.
    Those refused are given to the other operators with a length of 0, on the device: their rows and pages keep their bytes,
    lengths, tables and counts are the model's, results of theirs are zeros, and once the last has ended they go on."""
    say(f"[gpu] a step with too few pages, trees={trees} eight={eight}")
    g = torch.Generator().manual_seed(19)
    layers, page, seqs, few, heads, vocab, d, max_pages = 2, 16, 6, 6, 16, 300, 128, 3
    pages = 3 + 1 + 3 + 1 + 2 + 1  # of the first (shared with the second), the third, fourth, fifth, sixth, and one free
    pool = Pool(seqs, max_pages, pages, page)
    dev = table, lens, refs = pool.tensors("cuda")
    context, slots = [33, 0, 16, 47, 3, 17], list(range(seqs))
    B.ds4hc_pages_resize(*dev, page, i32(slots), i32(context))
    pool.resize(slots, context)
    B.ds4hc_pages_fork(*dev, page, i32([0]), i32([1]))
    pool.fork([0], [1])
    context[1] = 33
    f = B.ds4hc_rope_frequencies(64)[0].cuda()
    if eight:
        caches = torch.zeros(layers, pages, page, d + 144, dtype=torch.uint8, device="cuda")
        append, attn = B.ds4hc_latent_append8, B.ds4hc_latent_attn8
    else:
        caches = torch.zeros(layers, pages, page, d + 64, dtype=BF, device="cuda")
        append, attn = B.ds4hc_latent_append, B.ds4hc_latent_attn
    first = [33, 0, 16, 47, 3, 17]  # (the second has the first one's rows)
    for layer in range(layers):
        rows = torch.randn(sum(first), d + 64, generator=g).to(BF).cuda()
        append(rows, torch.cat([torch.arange(k) for k in first]).cuda(), f, caches[layer], i32(sums_of(first)), lens, table)

    def rows_of(b, k):
        at = torch.tensor([pool.table[b][j // page] * page + j % page for j in range(k)], dtype=torch.long, device="cuda")
        return caches.view(layers, pages * page, -1)[:, at].clone()

    known = [rows_of(b, k) for b, k in enumerate(context)]
    cu = i32([few * b for b in range(seqs + 1)])
    drafted = few
    for turn in range(2):
        want = [k + few for k in context]
        if turn:  # the last has ended, and the fourth is at its end
            B.ds4hc_pages_resize(*dev, page, i32([5]), i32([0]))
            pool.resize([5], [0])
            known[5], context[5] = known[5][:, :0], 0
            want = [k + few if b != 5 else 0 for b, k in enumerate(context)]
        copies, status = B.ds4hc_pages_resize(*dev, page, i32(slots), i32(want))
        assert status.tolist() == pool.resize(slots, want)[1]
        assert status.tolist() == ([0, 1, 1, 2, 0, 0] if not turn else [0, 0, 0, 2, 0, 0])
        B.ds4hc_pages_copy(caches, copies)
        done = status == B.DS4HC_PAGES_DONE
        live = torch.where(done, lens, 0)
        if turn:
            live[5] = 0
        tree = random_trees(g, [few] * seqs) if trees else [list(range(-1, few - 1))] * seqs
        mask = []
        for t in tree:
            seen = []
            for i, p in enumerate(t):
                seen.append((1 << i) | (seen[p] if p >= 0 else 0))
            mask += [[s] for s in seen]
        ql = torch.randn(seqs * few, heads, d, generator=g).to(BF).cuda()
        qr = torch.randn(seqs * few, heads, 64, generator=g).to(BF).cuda()
        pos = torch.randint(0, 1000, (seqs * few,), generator=g).cuda()
        for layer in range(layers):
            new = torch.randn(seqs * few, d + 64, generator=g).to(BF).cuda()
            append(new, pos, f, caches[layer], cu, live, table)
            out, lse = attn(ql, qr, caches[layer], cu, live, table, scale=0.1, tree_mask=torch.tensor(mask).cuda(), want_lse=True)
            for b in range(seqs):
                rows = slice(few * b, few * (b + 1))
                if live[b]:
                    assert torch.isfinite(lse[rows]).all()
                else:
                    assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
        now = {b: rows_of(b, pool.lens[b]) for b in slots if live[b]}  # the context, and the drafts behind it
        target, _ = distributions(g, seqs * few, vocab)
        best = target.topk(few, -1).indices
        tokens = torch.tensor([0 if p < 0 else int(best[b * few + p, t[:i].count(p)]) for b, t in enumerate(tree)
                               for i, p in enumerate(t)]).cuda()
        path, kept, _ = B.ds4hc_draft_verify(target.cuda(), tokens, cu, torch.rand(seqs * few, generator=g).cuda(),
                                             parents=i32([p for t in tree for p in t]) if trees else None)
        B.ds4hc_cache_compact(caches, cu, live, table, path, kept)
        length = torch.where(done, lens - drafted + kept, lens)
        if turn:
            length[5] = 0
        _, status = B.ds4hc_pages_resize(*dev, page, i32(slots), length)
        assert (status == 0).all()
        pool.resize(slots, length.tolist())
        pool.check()
        for mine, theirs in zip(pool.tensors(), dev):
            assert torch.equal(mine, theirs.cpu())
        for b in slots:
            if b in now:
                way = path.tolist()[few * b:few * b + kept.tolist()[b]]
                assert torch.equal(now[b][:, :context[b]], known[b])
                known[b] = torch.cat((known[b], now[b][:, [context[b] + w for w in way]]), 1)
            context[b] = pool.lens[b]
            assert torch.equal(rows_of(b, context[b]), known[b]), (turn, b)


def test_a_captured_step_that_finds_too_few_pages():
    """The step of a chain of 4 for each of three sequences, captured whole: replays that find pages for all, for some and for
    none, with eager work between them, leave what the eager step leaves."""
    g = torch.Generator().manual_seed(23)
    layers, page, seqs, few, heads, vocab, d, pages = 2, 16, 3, 4, 16, 200, 128, 6
    table, lens, refs = Pool(seqs, 4, pages, page).tensors("cuda")
    caches = torch.randint(0, 120, (layers, pages, page, d + 144), generator=g, dtype=torch.uint8).cuda()
    caches[..., d:] = 0
    caches[..., d + 128] = 120
    f, cu, slots = B.ds4hc_rope_frequencies(64)[0].cuda(), i32([few * b for b in range(seqs + 1)]), i32(list(range(seqs)))
    new = torch.randn(layers, seqs * few, d + 64, generator=g).to(BF).cuda()
    pos = torch.arange(seqs * few).cuda()
    ql = torch.randn(seqs * few, heads, d, generator=g).to(BF).cuda()
    qr = torch.randn(seqs * few, heads, 64, generator=g).to(BF).cuda()
    target, draft = (t.cuda() for t in distributions(g, seqs * few, vocab))
    tokens, uniform = target.argmax(-1).roll(1), torch.zeros(seqs * few, device="cuda")
    copies, status, status2 = i32([[0, 0]] * seqs), i32([0] * seqs), i32([0] * seqs)
    out = torch.zeros(layers, seqs * few, heads, d, dtype=BF, device="cuda")
    path, kept, following = i32([0] * seqs * few), i32([0] * seqs), torch.zeros(seqs, dtype=torch.int64, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def step():
        B.ds4hc_pages_resize(table, lens, refs, page, slots, lens + few, copies=copies, status=status, workspace=ws)
        B.ds4hc_pages_copy(caches, copies)
        done = status == B.DS4HC_PAGES_DONE
        live = torch.where(done, lens, 0)
        for layer in range(layers):
            B.ds4hc_latent_append8(new[layer], pos, f, caches[layer], cu, live, table)
            B.ds4hc_latent_attn8(ql, qr, caches[layer], cu, live, table, scale=0.1, out=out[layer], workspace=ws)
        B.ds4hc_draft_verify(target, tokens, cu, uniform, draft=draft, path=path, n_kept=kept, next_token=following, workspace=ws)
        B.ds4hc_cache_compact(caches, cu, live, table, path, kept)
        B.ds4hc_pages_resize(table, lens, refs, page, slots, torch.where(done, lens - few + kept, lens), copies=copies,
                             status=status2, workspace=ws)

    state = (table, lens, refs, caches, out, path, kept, following, status, status2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = set()
    for want in ([15, 30, 2], [31, 30, 30], [32, 16, 32], [32, 32, 32], [64, 1, 0]):
        B.ds4hc_pages_resize(table, lens, refs, page, slots, i32([0] * seqs))
        _, what = B.ds4hc_pages_resize(table, lens, refs, page, slots, i32(want))
        assert (what == 0).all() and lens.tolist() == want
        saved = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in state]
        for t, old in zip(state, saved):
            t.copy_(old)
        step()
        torch.cuda.synchronize()
        for a, b in zip(state, replayed):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        seen.add(tuple(status.tolist()))
        for b, was in enumerate(want):
            assert lens[b].item() == (was + kept[b].item() if status[b].item() == 0 else was)
    assert {(0, 0, 0), (1, 1, 1)} < seen and len(seen) >= 3
