"""64-bit references of the attention-site operators and the bounds that their
results are held to. Everything here runs on the CPU.

Bounds. u = eps / 2 of the 16-bit type is the most that one rounding moves a value,
relative to it; e = 2^-24 that of float32.

Attention, per element of a row with weights w_j (they sum to 1) and values v_j:
the weights are rounded once (u), the output once (u); a logit is a float32 sum of D
products and two more operations, so it is off by at most (D + 8) e * scale *
sum |q||k| =: ds, and its weight by a factor within 1 +- 2 ds; sums over n tokens,
with a rescaling for at most every token, by (n + 64) e. Hence

    |out - exact| <= (u + 2 * (2 ds) + 2 (n + 64) e) * sum_j w_j |v_j| + u |exact|

where the numerator and the denominator each take 2 ds and (n + 64) e. The same
without the roundings to 16 bits for lse: |lse - exact| <= ds + (n + 64) e + 4 e |lse|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

E32 = 2.0 ** -24


def u_of(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def turn64(x, positions, inv_freq, amplitude=1.0, interleaved=True, inverse=False):
    """x [n, ..., dim] in 64 bits, rotated."""
    x = x.double()
    a = positions.double().view(-1, *[1] * (x.dim() - 1)) * inv_freq.double()
    if inverse:
        a = -a
    half = x.shape[-1] // 2
    x0, x1 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y0, y1 = (x0 * a.cos() - x1 * a.sin()) * amplitude, (x0 * a.sin() + x1 * a.cos()) * amplitude
    if interleaved:
        return torch.stack((y0, y1), -1).flatten(-2)
    return torch.cat((y0, y1), -1)


def rope_bound(x, positions, inv_freq, amplitude, interleaved, dtype):
    """Per element: the angle's 64-bit product and reduction leave its float32 part
    (half a turn at most) with an error of 2^-24 of it and a few of its last places in
    sincos (4 e in all, in cos and sin); two products and a sum in float32, one
    rounding at the store. |x0| + |x1| bounds the terms. 64-bit angle: |a| 2^-52 each."""
    x = x.double().abs()
    half = x.shape[-1] // 2
    x0, x1 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    s = (x0 + x1) * abs(amplitude)
    a = positions.double().abs().view(-1, *[1] * (x.dim() - 1)) * inv_freq.double()
    part = s * (16 * E32 + a * 2.0 ** -50)
    part = torch.stack((part, part), -1).flatten(-2) if interleaved else torch.cat((part, part), -1)
    return part, (0.0 if dtype == torch.float32 else u_of(dtype))


def attend64(q, k, v, seen, scale):
    """q [r, d], k [n, d], v [n, e], seen [r, n] -> out, lse, sum w|v|, ds. Keys and
    values that a row does not see do not enter it, whatever they hold."""
    r, n = seen.shape
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(r, v.shape[1], dtype=torch.float64)
    size, lse, ds = out.clone(), torch.full((r,), -math.inf, dtype=torch.float64), torch.zeros(r, dtype=torch.float64)
    same = bool((seen == seen[:1]).all()) if r else False
    for rows in ([slice(0, r)] if same else [slice(i, i + 1) for i in range(r)]):
        j = seen[rows][0].nonzero()[:, 0]
        if not len(j):
            continue
        kj, vj = k[j], v[j]
        s = q[rows] @ kj.T * scale
        lse[rows] = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[rows][:, None])
        out[rows], size[rows] = w @ vj, w @ vj.abs()
        ds[rows] = (q.shape[1] + 8) * E32 * scale * (q[rows].abs() @ kj.abs().T).amax(-1)
    return out, lse, size, ds


def assert_attention(got, lse, ref, seen_counts, dtype, where=""):
    """got [r, e] and lse [r] (None: not looked at) against attend64's `ref`."""
    out, ref_lse, size, ds = ref
    n = torch.as_tensor(seen_counts, dtype=torch.float64)
    u = u_of(dtype)
    got = got.double()
    empty = n == 0
    assert (got[empty] == 0).all(), where
    bound = (u + 4 * ds + 2 * (n + 64) * E32)[:, None] * size + u * out.abs() + 1e-30
    over = ((got - out).abs() / bound)
    assert torch.isfinite(got).all(), where
    assert (over <= 1.0).all(), f"{where}: {over.max().item():.3g} times the bound"
    if lse is not None:
        lse = lse.double()
        assert (lse[empty] == -math.inf).all(), where
        d = (lse - ref_lse).abs()[~empty]
        tol = (ds + (n + 64) * E32 + 4 * E32 * ref_lse.abs())[~empty]
        assert (d <= tol).all(), f"{where}: lse {(d / tol).max().item():.3g} times the bound"


class Batch:
    """A paged batch on the CPU: pages of the sequences in random order, the cache's
    unused places holding NaN."""

    def __init__(self, seed, q_len, kv_len, page, latent=512, dtype=torch.bfloat16, spare=3, extra_tokens=0,
                 max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.q_len, self.kv_len, self.page, self.latent, self.dtype = g, q_len, kv_len, page, latent, dtype
        need = [-(-k // page) for k in kv_len]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.max_pages = max(need + [1]) if max_pages is None else max_pages
        table = np.full((len(need), self.max_pages), -1, np.int32)
        for b, n in enumerate(need):
            table[b, :n] = [order.pop() for _ in range(n)]
        self.table = torch.from_numpy(table)
        self.cu = torch.tensor([0] + list(np.cumsum(q_len)), dtype=torch.int32)
        self.lens = torch.tensor(kv_len, dtype=torch.int32)
        self.N = int(self.cu[-1]) + extra_tokens
        self.cache = torch.full((self.n_pages, page, latent + 64), float("nan"), dtype=dtype)
        flat = self.cache.view(-1, latent + 64)
        for b, k in enumerate(kv_len):
            if k:
                flat[self.rows(b, k)] = torch.randn(k, latent + 64, generator=g).to(dtype)

    def rows(self, b, k):
        j = torch.arange(k)
        return self.table[b, j // self.page].long() * self.page + j % self.page

    def queries(self, heads, size=1.0):
        ql = (torch.randn(self.N, heads, self.latent, generator=self.g) * size).to(self.dtype)
        return ql, (torch.randn(self.N, heads, 64, generator=self.g) * size).to(self.dtype)

    def reference(self, ql, qr, scale, tree=None, holes=()):
        """Per token: (attend64's result over the heads, tokens seen). tree [N, words]
        int64; holes: (b, page index) whose tokens are not in the cache."""
        res = []
        heads = ql.shape[1]
        flat = self.cache.view(-1, self.latent + 64)
        for b, (q, k) in enumerate(zip(self.q_len, self.kv_len)):
            keys = flat[self.rows(b, k)]
            j = torch.arange(k)
            gone = torch.zeros(k, dtype=torch.bool)
            for hb, p in holes:
                if hb == b:
                    gone |= (j // self.page) == p
            for i in range(q):
                t = int(self.cu[b]) + i
                d = j - (k - q)
                if tree is None:
                    seen = d <= i
                else:
                    words = tree[t].tolist()
                    bit = torch.tensor([(words[x >> 6] >> (x & 63)) & 1 if 0 <= x < 64 * len(words) else 0
                                        for x in d.tolist()], dtype=torch.bool)
                    seen = (d < 0) | bit
                seen = seen & ~gone
                qs = torch.cat((ql[t], qr[t]), -1)
                res.append((attend64(qs, keys, keys[:, :self.latent], seen.expand(heads, k), scale),
                            [int(seen.sum())] * heads))
        return res


def random_tree(g, q_len, words):
    """[N, words] int64: each token sees itself and its ancestors."""
    rows = []
    for n in q_len:
        seen = []
        for i in range(n):
            up = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            seen.append((1 << i) | (seen[up] if up >= 0 else 0))
        rows += seen
    w = [[(r >> (64 * x)) & (2 ** 64 - 1) for x in range(words)] for r in rows]
    return torch.from_numpy(np.array(w, dtype=np.uint64).reshape(len(rows), words).view(np.int64))
