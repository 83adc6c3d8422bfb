"""64-bit references of the operators around the attention of drafted tokens, and batches over a
cache of 8-bit latents. Everything here runs on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch

from site_testlib import Batch

TOP = 448.0  # e4m3's largest number


def to_rows8(latents, rope):
    """Rows of an 8-bit cache: latents [n, d] in 64 bits, rope [n, 64] of a 16-bit type. Values that are not
    finite make their row NaN."""
    top = latents.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(top)
    e = torch.ceil(torch.log2(torch.where(bad | (top == 0), torch.ones_like(top), top) / TOP))
    e = torch.where(top == 0, torch.full_like(e, -117), e).clamp(-117, 119)
    eight = (latents / torch.exp2(e)).clamp(-TOP, TOP).float().to(torch.float8_e4m3fn).view(torch.uint8)
    eight = torch.where(bad, torch.full_like(eight, 0x7F), eight)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    rest = torch.zeros(len(latents), 15, dtype=torch.uint8)
    return torch.cat((eight, rope.contiguous().view(torch.uint8), scale, rest), -1)


def values8(rows, dtype):
    """(latent, rope) in 64 bits of rows of an 8-bit cache."""
    d = rows.shape[-1] - 144
    scale = torch.exp2(rows[..., d + 128].double() - 127)
    scale = torch.where(rows[..., d + 128] == 255, torch.full_like(scale, math.nan), scale)
    latent = rows[..., :d].contiguous().view(torch.float8_e4m3fn).double() * scale[..., None]
    return latent, rows[..., d:d + 128].contiguous().view(dtype).double()


class Batch8(Batch):
    """A paged batch over a cache of 8-bit latents: `rows8` [pages, page, d + 144] uint8 is the cache, whose unused
    places hold NaN, and `cache` the values that it stands for. spread: the tokens' sizes are powers of 2 up to that."""

    def __init__(self, *args, spread=0, **kw):
        super().__init__(*args, **kw)
        d = self.latent
        self.rows8 = torch.full((self.n_pages, self.page, d + 144), 0x7F, dtype=torch.uint8)
        self.rows8[..., d + 128] = 255
        flat, flat8 = self.cache.view(-1, d + 64), self.rows8.view(-1, d + 144)
        for b, k in enumerate(self.kv_len):
            if k:
                at = self.rows(b, k)
                size = torch.exp2(torch.randint(-spread, spread + 1, (k, 1), generator=self.g).double())
                flat8[at] = to_rows8(flat[at, :d].double() * size, flat[at, d:])
        self.refresh()

    def refresh(self):
        latent, rope = values8(self.rows8, self.dtype)
        self.cache = torch.cat((latent, rope), -1)


# ------------------------------------------------------------------ drafted tokens

def verify64(target, tokens, cu, uniform, draft=None, parents=None, limit=1024):
    """(path, kept, next, margin): margin is how far, of the total, the number that chose the next token lies from the
    nearest border, inf where there is none to look at."""
    n, vocab = target.shape
    clean = lambda x: torch.where((x > 0) & torch.isfinite(x), x, torch.zeros_like(x)).double()  # noqa: E731
    number = lambda u: min(float(u), 1 - 2.0 ** -24) if float(u) > 0 else 0.0  # noqa: E731  (NaN: 0)
    path, kept, following, margin = [None] * n, [], [], []
    for b in range(len(cu) - 1):
        t0, few = cu[b], max(cu[b + 1] - cu[b], 0)
        if few == 0:
            kept.append(0), following.append(-1), margin.append(math.inf)
            continue
        seen = min(few, limit)
        up = [-1] + (list(range(seen - 1)) if parents is None else [int(parents[t0 + i]) for i in range(1, seen)])
        node, way = 0, [0]
        while True:
            p, left, mass, nxt, tried = clean(target[t0 + node]), None, 1.0, None, set()
            left = p.clone()
            for c in range(node + 1, seen):
                if up[c] != node:
                    continue
                x, u = int(tokens[t0 + c]), number(uniform[t0 + c])
                inside = 0 <= x < vocab
                px = float(p[x]) if inside else 0.0
                if draft is not None:
                    q = clean(draft[t0 + node])
                    if inside and px > 0 and u * float(q[x]) < px:
                        nxt = c
                        break
                    left = (p - q).clamp(min=0)
                    continue
                if x in tried:
                    continue
                tried.add(x)
                if px > 0 and u * mass < px:
                    nxt = c
                    break
                mass -= px
                if inside:
                    left[x] = 0
            if nxt is None:
                break
            node = nxt
            way.append(nxt)
        for i in range(few):
            path[t0 + i] = way[i] if i < len(way) else -1
        kept.append(len(way))
        if left.sum() <= 0:
            left = p
        total = float(left.sum())
        if total <= 0:
            following.append(-1), margin.append(math.inf)
            continue
        sums = left.cumsum(0)
        goal = number(uniform[t0]) * float(sums[-1])
        x = int((sums <= goal).sum())
        if x >= vocab:
            x = int(left.nonzero()[-1])
        following.append(x)
        margin.append(float((sums - goal).abs().min()) / total)
    return path, kept, following, margin


# ------------------------------------------------------------------ pages

class Pool:
    """The pool of pages as lists, one item after another."""

    def __init__(self, slots, max_pages, pages, page):
        self.page, self.max_pages = page, max_pages
        self.table = [[-1] * max_pages for _ in range(slots)]
        self.lens, self.refs = [0] * slots, [0] * pages

    def tensors(self, device="cpu"):
        return tuple(torch.tensor(x, dtype=torch.int32, device=device) for x in (self.table, self.lens, self.refs))

    def resize(self, slots, lengths):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        copies, status, need, seen, drops, takes = [], [], 0, set(), [], []
        start = list(self.refs)
        for s, new in zip(slots, lengths):
            copies.append([-1, -1])
            earlier = s in seen
            seen.add(s)
            if not 0 <= s < len(self.lens) or earlier or not 0 <= new <= self.max_pages * self.page:
                status.append(2)
                continue
            old = self.lens[s]
            had, has = -(-old // self.page), -(-new // self.page)
            last = self.table[s][had - 1] if had else -1
            own = int(new > old and old % self.page != 0 and 0 <= last < len(start) and start[last] > 1)
            first, want = need, max(has - had, 0) + own
            need += want
            if want and need > len(free):
                status.append(1)
                continue
            status.append(0)
            got = free[first:first + want]
            if own:
                page = got.pop(0)
                copies[-1] = [last, page]
                self.table[s][had - 1] = page
                drops.append(last)
                takes.append(page)
            for e in range(had, has):
                self.table[s][e] = got.pop(0)
                takes.append(self.table[s][e])
            for e in range(has, had):
                if 0 <= self.table[s][e] < len(start):
                    drops.append(self.table[s][e])
                self.table[s][e] = -1
            self.lens[s] = new
        for p in drops:
            self.refs[p] -= 1
        for p in takes:
            self.refs[p] = 1
        return copies, status

    def fork(self, parents, children):
        lens, status, seen = list(self.lens), [], set()
        for p, c in zip(parents, children):
            ok = 0 <= c < len(lens) and c not in seen and 0 <= p < len(lens) and p != c and lens[c] == 0
            if 0 <= c < len(lens):
                seen.add(c)
            status.append(0 if ok else 2)
            if ok:
                for e in range(-(-lens[p] // self.page)):
                    self.table[c][e] = self.table[p][e]
                    self.refs[self.table[p][e]] += 1
                self.lens[c] = lens[p]
        return status

    def check(self):
        """Every entry counted, tables as long as the lengths say."""
        count = [0] * len(self.refs)
        for row, n in zip(self.table, self.lens):
            have = -(-n // self.page)
            assert all(0 <= e < len(count) for e in row[:have]) and all(e == -1 for e in row[have:])
            for e in row[:have]:
                count[e] += 1
        assert count == self.refs


def compact_rows(flat, table, page, cu, lens, keep, n_keep, max_pages):
    """ds4hc_cache_compact on flat [layers, rows, ...], one move after another."""
    n_pages = flat.shape[1] // page
    for b in range(len(lens)):
        few = cu[b + 1] - cu[b]
        base = min(max(lens[b], 0), max_pages * page) - few

        def place(i):
            j = base + i
            if not 0 <= j < max_pages * page or not 0 <= table[b][j // page] < n_pages:
                return None
            return table[b][j // page] * page + j % page

        for i in range(min(n_keep[b], few)):
            k = keep[cu[b] + i]
            if 0 <= k < few and place(k) is not None and place(i) is not None:
                flat[:, place(i)] = flat[:, place(k)].clone()


def random_trees(g, q_len):
    """Parents among each sequence's tokens, the first one's -1."""
    return [([-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, n)])[:n] for n in q_len]


def distributions(g, n, vocab, sharp=2.0, near=0.7):
    """A target and a draft near it, [n, vocab] float32."""
    logits = torch.randn(n, vocab, generator=g) * sharp
    return torch.softmax(logits, -1), torch.softmax(logits + near * torch.randn(n, vocab, generator=g), -1)


def sums_of(lengths):
    return [0] + np.cumsum(lengths).tolist()
