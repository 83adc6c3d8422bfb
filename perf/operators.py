"""The operators of an attention site, as cases to time: rotary positions, the append to a paged latent cache, latent
attention over that cache (absorbed form: single tokens, drafted chains and trees) and latent attention over expanded
keys and values (prompts).

A case is a dict of plain values. ``prepare`` makes what a program holds before the call, ``run`` is one pass through
the operator: in plain torch where ``own`` is false, through the library where it is true. ``exact`` gives the same
outputs in 64 bits, ``work`` the bytes and operations that a pass cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE = 64          # rotated part of a latent row and of a head
NOPE, VALUE = 128, 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a drafted chain of four tokens through one layer: the rotated part of 128 heads, cut out of the query rows
        dict(name="rope_verify", op="rope", dtype="bf16", tokens=4, heads=128, head_dim=192, dim=64, interleaved=True,
             start=1000, factor=1.0),
        # a prompt of the benchmark's length, all heads
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=4096, heads=128, head_dim=192, dim=64,
             interleaved=True, start=0, factor=1.0),
        # odd sizes, float32, half layout, positions far behind the trained length (scaled frequencies)
        dict(name="rope_far", op="rope", dtype="f32", tokens=1021, heads=7, head_dim=80, dim=80, interleaved=False,
             start=900000, factor=40.0),
        # one decode step of 32 sequences: a row each
        dict(name="append_decode", op="append", dtype="bf16", source="bf16", seqs=32, q=1, kv=2048, ragged=True,
             latent=512, page=64, norm=True, interleaved=True),
        # prompts of four sequences of unequal length, float32 projections into a bfloat16 cache
        dict(name="append_prompts", op="append", dtype="bf16", source="f32", seqs=4, q=2048, kv=2500, ragged=True,
             latent=512, page=64, norm=True, interleaved=True),
        # the smallest call: one token of one sequence, a share of 16 heads, a short context
        dict(name="attn_one", op="attn", dtype="bf16", seqs=1, q=1, heads=16, kv=500, ragged=False, latent=512,
             page=64, mask="causal"),
        # one sequence with a long context: the work has to be split over the tokens
        dict(name="attn_long", op="attn", dtype="bf16", seqs=1, q=1, heads=128, kv=131000, ragged=False, latent=512,
             page=64, mask="causal"),
        # a serving batch: 64 sequences of unequal length, one token each, all heads
        dict(name="attn_batch", op="attn", dtype="bf16", seqs=64, q=1, heads=128, kv=8192, ragged=True, latent=512,
             page=64, mask="causal"),
        # trees of up to 40 drafted tokens over contexts of unequal length, float16, a share of 16 heads, small pages
        dict(name="attn_tree", op="attn", dtype="f16", seqs=8, q=40, heads=16, kv=5000, ragged=True, latent=512,
             page=16, mask="tree"),
        # drafted chains of four tokens, all heads
        dict(name="attn_verify", op="attn", dtype="bf16", seqs=24, q=4, heads=128, kv=4096, ragged=True, latent=512,
             page=64, mask="causal"),
        # one prompt of the benchmark's length, a share of 32 heads
        dict(name="prefill_prompt", op="prefill", dtype="bf16", seqs=1, q=4096, prefix=0, heads=32, ragged=False),
        # prompts of unequal length behind prefixes that are already known, float16
        dict(name="prefill_ragged", op="prefill", dtype="f16", seqs=6, q=1500, prefix=700, heads=8, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "prefill"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        heads, dim = _log(rng, 1, 128), 2 * _log(rng, 8, 64)
        return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), tokens=_log(rng, 1, max(1, min(8192, 2 ** 24 // (heads * dim)))),
                    heads=heads, head_dim=dim + rng.choice([0, 16, 128]), dim=dim, interleaved=rng.random() < 0.5,
                    start=rng.randrange(0, 1000000), factor=rng.choice([1.0, 40.0]))
    if op == "append":
        seqs = _log(rng, 1, 64)
        q = _log(rng, 1, 4096 // seqs)
        return dict(op=op, dtype=half, source=rng.choice([half, "f32"]), seqs=seqs, q=q, kv=q + _log(rng, 1, 2000),
                    ragged=rng.random() < 0.7, latent=rng.choice([128, 256, 512]), page=2 ** rng.randrange(4, 8),
                    norm=rng.random() < 0.8, interleaved=rng.random() < 0.5)
    if op == "attn":
        seqs, mask = _log(rng, 1, 64), rng.choice(["causal", "causal", "tree"])
        q, heads = (rng.choice([1, 1, 2, 3, 4]) if mask == "causal" else rng.randrange(2, 65)), _log(rng, 1, 128)
        most = min(100000, 2 ** 18 // seqs, 2 ** 25 // (seqs * q * heads))
        return dict(op=op, dtype=half, seqs=seqs, q=q, heads=heads, kv=q + _log(rng, 1, max(2, most - q)),
                    ragged=rng.random() < 0.7, latent=rng.choice([128, 256, 512, 512]), page=2 ** rng.randrange(4, 8),
                    mask=mask)
    heads, seqs = _log(rng, 1, 32), _log(rng, 1, 6)
    q = _log(rng, 16, max(16, min(4096, int(math.sqrt(2 ** 27 // (heads * seqs))))))
    return dict(op=op, dtype=half, seqs=seqs, q=q, prefix=rng.choice([0, 0, _log(rng, 1, 500)]), heads=heads,
                ragged=rng.random() < 0.7)


# ------------------------------------------------------------------ what a program holds before the call

def _lengths(case):
    """Per sequence: tokens of this call, and tokens in all (those before this call included)."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    total = case.get("kv") or case["q"] + case["prefix"]
    q_len, kv_len = [], []
    for b in range(case["seqs"]):
        first = b == 0 or not case["ragged"]
        few = case["q"] if first or case["q"] < 5 else rng.randrange(1, case["q"] + 1)
        q_len.append(few)
        kv_len.append(total if first else rng.randrange(few, total + 1))
    return q_len, kv_len


def _sums(lengths):
    return [0] + np.cumsum(lengths).tolist()


def _frequencies(dim, factor, length=4096, base=10000.0, fast=32.0, slow=1.0):
    """Angle a position of each pair, and the amplitude; slow pairs are stretched by `factor` (the ramp of Peng et al.
    2023, "YaRN")."""
    i = np.arange(dim // 2, dtype=np.float64)
    f = base ** (-2.0 * i / dim)
    if factor == 1.0:
        return f, 1.0
    turn = lambda beta: dim * math.log(length / (2.0 * math.pi * beta)) / (2.0 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(turn(fast)), 0), min(math.ceil(turn(slow)), dim // 2 - 1)
    kept = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f * (kept + (1.0 - kept) / factor), 0.1 * math.log(factor) + 1.0


def _tree(rng, q_len, words):
    """Random trees of drafted tokens: each token sees itself and its ancestors, as bits over its sequence's tokens."""
    rows, depth = [], []
    for n in q_len:
        seen, deep = [], []
        for i in range(n):
            up = rng.randrange(-1, i) if i else -1
            seen.append((1 << i) | (seen[up] if up >= 0 else 0))
            deep.append(deep[up] + 1 if up >= 0 else 0)
        rows += seen
        depth += deep
    word = [[(r >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for r in rows]
    return np.array(word, dtype=np.uint64).reshape(len(rows), words).view(np.int64), depth


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape, dtype=dt: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "op": case["op"]}
    if case["op"] == "rope":
        freq, s["amplitude"] = _frequencies(case["dim"], case["factor"])
        s["freq"] = torch.from_numpy(freq).cuda()
        s["x"] = normal(case["tokens"], case["heads"], case["head_dim"])[..., case["head_dim"] - case["dim"]:]
        s["positions"] = case["start"] + rng.randrange(64) + torch.arange(case["tokens"], device="cuda")
        s["interleaved"] = case["interleaved"]
        return s
    q_len, kv_len = _lengths(case)
    cu, n = _sums(q_len), sum(q_len)
    s["cu_q"] = ints(cu)
    s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
    s["seq"] = torch.tensor(np.repeat(np.arange(len(q_len)), q_len), device="cuda")
    s["nth"] = torch.tensor(np.concatenate([np.arange(k) for k in q_len]), device="cuda")
    if case["op"] == "prefill":
        h = case["heads"]
        s["cu_k"], total = ints(_sums(kv_len)), sum(kv_len)
        s["q"], s["kv"] = normal(n, h, NOPE + ROPE), normal(total, h, NOPE + VALUE)
        s["k_rope"] = normal(total, 512 + ROPE)[:, 512:]  # beside the latent in the projection that makes both
        s["scale"] = (NOPE + ROPE) ** -0.5
        return s
    latent, page = case["latent"], case["page"]
    s["kv_len"] = ints(kv_len)
    need = [-(-k // page) for k in kv_len]
    pages = sum(need) + 3
    order = list(range(pages))
    rng.shuffle(order)
    table = np.full((len(need), max(need)), -1, np.int32)  # -1: no page there yet
    for b, k in enumerate(need):
        table[b, :k] = [order.pop() for _ in range(k)]
    s["table"] = torch.from_numpy(table).cuda()
    s["cache"] = normal(pages, page, latent + ROPE)
    if case["op"] == "append":
        freq, s["amplitude"] = _frequencies(ROPE, 1.0)
        s["freq"], s["interleaved"] = torch.from_numpy(freq).cuda(), case["interleaved"]
        s["rows"] = normal(n, latent + ROPE, dtype=DTYPES[case["source"]])
        s["weight"] = (1.0 + 0.1 * normal(latent, dtype=torch.float32)) if case["norm"] else None
        s["positions"] = s["kv_len"].long()[s["seq"]] - ints(q_len).long()[s["seq"]] + s["nth"]
        return s
    h = case["heads"]
    s["ql"], s["qr"], s["scale"] = normal(n, h, latent), normal(n, h, ROPE), (NOPE + ROPE) ** -0.5
    s["tree"] = None
    if case["mask"] == "tree":
        word, _ = _tree(rng, q_len, -(-max(q_len) // 64))
        s["tree"] = torch.from_numpy(word).cuda()
    return s


# ------------------------------------------------------------------ one pass

def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)


def _angles(positions, freq, amplitude):
    a = positions.double()[:, None] * freq  # 64 bits: float32 has no fraction left for far positions
    return (a.cos() * amplitude).float(), (a.sin() * amplitude).float()


def _softmax(x, seen):
    """Weights that are not yet divided by their sum, the sum, and the logarithm of the sum of exponentials."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def _divide(x, total):
    return torch.where(total > 0, x / total, torch.zeros_like(x))


def _plain_append(s):
    cache, latent, page = s["cache"], s["cache"].shape[-1] - ROPE, s["cache"].shape[1]
    x = s["rows"].float()
    c, r = x[:, :latent], x[:, latent:]
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    cos, sin = _angles(s["positions"], s["freq"], s["amplitude"])
    row = torch.cat((c, _rotate(r, cos, sin, s["interleaved"])), -1).to(cache.dtype)
    at = s["kv_len"][s["seq"]].long() - (s["cu_q"][s["seq"] + 1] - s["cu_q"][s["seq"]]).long() + s["nth"]
    cache[s["table"][s["seq"], at // page].long(), at % page] = row
    return cache


def _plain_attn(s):
    cache, latent, page = s["cache"], s["cache"].shape[-1] - ROPE, s["cache"].shape[1]
    n, h = s["ql"].shape[:2]
    b, most_q, most_k = s["kv_len"].shape[0], s["max_q"], s["max_kv"]
    j = torch.arange(most_k, device="cuda")
    i = torch.arange(most_q, device="cuda")
    keys = cache[s["table"][:, j // page].long().clamp(min=0), j % page].float()  # [b, k, latent + rope]
    token = (s["cu_q"][:-1, None].long() + i).clamp(max=n - 1)
    q = torch.cat((s["ql"], s["qr"]), -1)[token].float()  # [b, q, h, latent + rope]
    x = torch.matmul(q.flatten(1, 2), keys.transpose(1, 2)).view(b, most_q, h, most_k) * s["scale"]
    few = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    context = (s["kv_len"].long() - few)[:, None, None]
    if s["tree"] is None:
        seen = j <= context + i[:, None]
    else:
        at = (j - context).clamp(0, 64 * s["tree"].shape[1] - 1)  # [b, 1, k]
        word = torch.gather(s["tree"][token], 2, (at // 64).expand(b, most_q, most_k))
        seen = (j < context) | (((word >> (at % 64)) & 1) != 0)
    seen = seen & (j < s["kv_len"][:, None, None])
    p, total, lse = _softmax(x, seen[:, :, None])
    o = torch.matmul(p.flatten(1, 2), keys[..., :latent]).view(b, most_q, h, latent)
    o = _divide(o, total)[s["seq"], s["nth"]]
    return o.to(s["ql"].dtype), lse[s["seq"], s["nth"]]


def _plain_prefill(s):
    q, kv = s["q"], s["kv"]
    (n, h), b = q.shape[:2], s["cu_q"].shape[0] - 1
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    at_q = (cu_q[:-1, None] + i).clamp(max=n - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=kv.shape[0] - 1)
    few, many = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qs = q[at_q].float().transpose(1, 2)  # [b, h, q, 192]
    kvs = kv[at_k].float().transpose(1, 2)
    kr = s["k_rope"][at_k].float()[:, None].expand(b, h, -1, -1)
    x = torch.matmul(qs, torch.cat((kvs[..., :NOPE], kr), -1).transpose(2, 3)) * s["scale"]
    seen = (j <= (many - few)[:, None, None] + i[:, None]) & (j < many[:, None, None])
    p, total, lse = _softmax(x, seen[:, None])
    o = _divide(torch.matmul(p, kvs[..., NOPE:]), total)
    return o[s["seq"], :, s["nth"]].to(q.dtype), lse[s["seq"], :, s["nth"]]


def run(s):
    op = s["op"]
    if own:
        import deepseek_v4_hyper_amd as ds4hc
        if op == "rope":
            return ds4hc.ds4hc_rope(s["x"], s["positions"], s["freq"], interleaved=s["interleaved"],
                                    amplitude=s["amplitude"])
        if op == "append":
            return ds4hc.ds4hc_latent_append(s["rows"], s["positions"], s["freq"], s["cache"], s["cu_q"], s["kv_len"],
                                             s["table"], norm_weight=s["weight"], rms_eps=1e-6,
                                             interleaved=s["interleaved"], amplitude=s["amplitude"])
        if op == "attn":
            return ds4hc.ds4hc_latent_attn(s["ql"], s["qr"], s["cache"], s["cu_q"], s["kv_len"], s["table"],
                                           scale=s["scale"], tree_mask=s["tree"], want_lse=True)
        return ds4hc.ds4hc_latent_prefill(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], scale=s["scale"],
                                          want_lse=True)
    if op == "rope":
        cos, sin = _angles(s["positions"], s["freq"], s["amplitude"])
        return _rotate(s["x"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(s["x"].dtype)
    if op == "append":
        return _plain_append(s)
    return _plain_attn(s) if op == "attn" else _plain_prefill(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * e + 8 * case["tokens"] + 4 * case["dim"], "flops": 3 * n}
    q_len, kv_len = _lengths(case)
    n = sum(q_len)
    if case["op"] == "append":
        row = case["latent"] + ROPE
        return {"bytes": n * row * (SIZE[case["source"]] + e) + 12 * n + 4 * case["latent"], "flops": 4 * n * row}
    if case.get("mask") == "tree":  # a token of a random tree sees few of the others: the context is what counts
        pairs = sum(q * (k - q) for q, k in zip(q_len, kv_len))
    else:
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(q_len, kv_len))
    h = case["heads"]
    if case["op"] == "attn":
        row = case["latent"] + ROPE
        return {"bytes": sum(kv_len) * row * e + n * h * ((row + case["latent"]) * e + 4),
                "flops": 2 * h * pairs * (row + case["latent"])}
    return {"bytes": n * h * ((NOPE + ROPE + VALUE) * e + 4) + sum(kv_len) * (h * (NOPE + VALUE) + ROPE) * e,
            "flops": 2 * h * pairs * (NOPE + ROPE + VALUE)}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _turn(x, positions, freq, amplitude, interleaved):
    """Pairs as complex numbers, turned by exp(i a). x [n, ..., dim] in 64 bits."""
    half = x.shape[-1] // 2
    z = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) if interleaved else torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    a = positions.double().view(-1, *[1] * (x.dim() - 1)) * freq
    z = z * torch.polar(torch.full_like(a, amplitude), a)
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)


def _attend(q, k, v, seen, scale):
    """q [r, d], k [t, d], v [t, e], seen [r, t], all of one head; rows that see nothing are 0 and -inf."""
    x = torch.where(seen, q @ k.T * scale, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.nan_to_num(torch.exp(x - lse[:, None])) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _turn(s["x"].double(), s["positions"], s["freq"], s["amplitude"], s["interleaved"])
    q_len, kv_len = _lengths(case)
    cu = _sums(q_len)
    if s["op"] == "append":
        cache, x = s["cache"].double(), s["rows"].double()
        c, latent, page = x[:, :case["latent"]], case["latent"], case["page"]
        if s["weight"] is not None:
            c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / latent + 1e-6) * s["weight"].double()
        row = torch.cat((c, _turn(x[:, latent:], s["positions"], s["freq"], s["amplitude"], s["interleaved"])), -1)
        flat = cache.view(-1, latent + ROPE)
        for b, (q, k) in enumerate(zip(q_len, kv_len)):
            at = torch.arange(k - q, k, device="cuda")
            flat[s["table"][b, at // page].long() * page + at % page] = row[cu[b]:cu[b + 1]]
        return cache
    out, lse = [], []
    if s["op"] == "attn":
        latent, page, h = case["latent"], case["page"], case["heads"]
        for b, (q, k) in enumerate(zip(q_len, kv_len)):
            j = torch.arange(k, device="cuda")
            keys = s["cache"].view(-1, latent + ROPE)[s["table"][b, j // page].long() * page + j % page].double()
            o, m = [], []
            for i in range(q):
                t = cu[b] + i
                seen = j <= k - q + i
                if s["tree"] is not None:
                    bits = s["tree"][t].tolist()
                    seen = torch.cat((torch.ones(k - q, dtype=torch.bool), torch.tensor([bits[d // 64] >> (d % 64) & 1 == 1 for d in range(q)]))).cuda()
                a, w = _attend(torch.cat((s["ql"][t], s["qr"][t]), -1).double(), keys, keys[:, :latent], seen.expand(h, k), s["scale"])
                o.append(a)
                m.append(w)
            out += [torch.stack(o)]
            lse += [torch.stack(m)]
        return torch.cat(out), torch.cat(lse)
    cu_k = _sums(kv_len)
    for b, (q, k) in enumerate(zip(q_len, kv_len)):
        here, there = slice(cu[b], cu[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = torch.ones(q, k, dtype=torch.bool, device="cuda").tril(k - q)
        each = []
        for h in range(case["heads"]):
            keys = torch.cat((s["kv"][there, h, :NOPE], s["k_rope"][there]), -1).double()
            each.append(_attend(s["q"][here, h].double(), keys, s["kv"][there, h, NOPE:].double(), seen, s["scale"]))
        out.append(torch.stack([e[0] for e in each], 1))
        lse.append(torch.stack([e[1] for e in each], 1))
    return torch.cat(out), torch.cat(lse)
