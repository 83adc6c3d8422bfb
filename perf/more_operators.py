"""The operators of serving drafted tokens over a paged latent cache, as cases to time: the append to a cache held in 8
bits and the attention over it, the verification of drafted tokens from given random numbers, the move of accepted tokens
to their places, and the taking, forking, copying and freeing of pages.

A case is a dict of plain values. ``prepare`` makes what a program holds before the call, ``run`` is one pass: in plain
torch where ``own`` is false, through the library where it is true. ``exact`` gives computed numbers in 64 bits, ``work``
the bytes and operations that a pass cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE = 64                # rotated part of a latent row, 16 bits an element
LAYERS = 43              # layers of the benchmark's decode chain, each with a cache of its own
BYTES = ROPE * 2 + 16    # of an 8-bit row behind its latent: rotated part, scale, 15 unused
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
TOP, LOWEST, HIGHEST = 448.0, -117, 119  # largest e4m3 value, exponents of scales


def listed():
    return [
        # one decode step of 32 sequences: a row each
        dict(name="append8_decode", op="append8", dtype="bf16", source="bf16", seqs=32, q=1, kv=2048, ragged=True,
             latent=512, page=64, norm=True, interleaved=True),
        # prompts of four sequences of unequal length, float32 projections
        dict(name="append8_prompts", op="append8", dtype="bf16", source="f32", seqs=4, q=2048, kv=2500, ragged=True,
             latent=512, page=64, norm=True, interleaved=True),
        # the smallest attention: one token of one sequence, a share of 16 heads, a short context
        dict(name="attn8_one", op="attn8", dtype="bf16", seqs=1, q=1, heads=16, kv=500, ragged=False, latent=512,
             page=64, mask="causal"),
        # a large serving batch on a share of 16 heads: the cache's bytes are what counts
        dict(name="attn8_share", op="attn8", dtype="bf16", seqs=128, q=1, heads=16, kv=8192, ragged=True, latent=512,
             page=64, mask="causal"),
        # a serving batch with all heads
        dict(name="attn8_batch", op="attn8", dtype="bf16", seqs=64, q=1, heads=128, kv=8192, ragged=True, latent=512,
             page=64, mask="causal"),
        # trees of up to 40 drafted tokens over contexts of unequal length, float16, small pages
        dict(name="attn8_tree", op="attn8", dtype="f16", seqs=8, q=40, heads=16, kv=5000, ragged=True, latent=512,
             page=16, mask="tree"),
        # drafted chains of four tokens for 64 sequences, a vocabulary of odd size
        dict(name="verify_chain", op="verify", seqs=64, q=5, vocab=100003, tree=False, ragged=True),
        # a small batch of drafted trees, judged by the target alone
        dict(name="verify_tree", op="verify", seqs=4, q=40, vocab=32000, tree=True, ragged=True),
        # accepted tokens of 64 drafted trees moved behind their contexts, in the 8-bit caches of all layers
        dict(name="compact_step", op="compact", dtype="u8", seqs=64, q=32, keep=8, kv=300, layers=LAYERS, latent=512,
             page=64),
        # the same of one chain in one layer's 16-bit cache: nothing but latency
        dict(name="compact_one", op="compact", dtype="bf16", seqs=1, q=4, keep=3, kv=200, layers=1, latent=512, page=64),
        # a quarter of 256 sequences end and others of the same lengths begin, in a large pool
        dict(name="pages_turnover", op="turnover", seqs=256, kv=8192, moved=64, page=64, pool=65536),
        # beams: four branches of each of 16 sequences are forked anew, grow by a token, and get their own copy of the
        # last page in all layers
        dict(name="pages_beam", op="beam", dtype="u8", seqs=16, branches=4, kv=500, page=64, layers=LAYERS, latent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append8", "attn8", "attn8", "verify", "verify", "compact", "turnover", "beam"])
    half, latent, page = rng.choice(["bf16", "bf16", "f16"]), rng.choice([128, 256, 512, 512]), 2 ** rng.randrange(4, 8)
    ragged = rng.random() < 0.7
    if op == "append8":
        seqs = _log(rng, 1, 64)
        q = _log(rng, 1, 4096 // seqs)
        return dict(op=op, dtype=half, source=rng.choice([half, "f32"]), seqs=seqs, q=q, kv=q + _log(rng, 1, 2000),
                    ragged=ragged, latent=latent, page=page, norm=rng.random() < 0.8, interleaved=rng.random() < 0.5)
    if op == "attn8":
        seqs, mask = _log(rng, 1, 128), rng.choice(["causal", "causal", "tree"])
        q, heads = (rng.choice([1, 1, 2, 3, 4]) if mask == "causal" else rng.randrange(2, 65)), _log(rng, 1, 128)
        most = min(100000, 2 ** 18 // seqs, 2 ** 25 // (seqs * q * heads))
        return dict(op=op, dtype=half, seqs=seqs, q=q, heads=heads, kv=q + _log(rng, 1, max(2, most - q)), ragged=ragged,
                    latent=latent, page=page, mask=mask)
    if op == "verify":
        seqs, tree = _log(rng, 1, 64), rng.random() < 0.5
        vocab = _log(rng, 1000, 150000)
        most = max(2, min(64 if tree else 9, 32000000 // (seqs * vocab)))
        return dict(op=op, seqs=seqs, q=rng.randrange(2, most + 1), vocab=vocab, tree=tree, ragged=ragged)
    if op == "compact":
        q, seqs, layers = rng.randrange(2, 65), _log(rng, 1, 64), _log(rng, 1, LAYERS)
        return dict(op=op, dtype=rng.choice(["u8", half]), seqs=seqs, q=q, keep=rng.randrange(1, min(q, 9) + 1),
                    kv=q + _log(rng, 1, min(2000, 2 ** 19 // (seqs * layers))), layers=layers, latent=latent, page=page)
    if op == "turnover":
        seqs = _log(rng, 2, 256)
        kv = _log(rng, 1, 8192)
        return dict(op=op, seqs=seqs, kv=kv, moved=_log(rng, 1, seqs), page=page,
                    pool=_log(rng, seqs * (kv // page + 2) + 8, 262144))
    return dict(op=op, dtype=rng.choice(["u8", half]), seqs=_log(rng, 1, 16), branches=rng.randrange(1, 5),
                kv=_log(rng, 1, 500), page=2 ** rng.randrange(4, 7), layers=_log(rng, 1, LAYERS), latent=latent)


# ------------------------------------------------------------------ what a program holds before the call

def _random(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """Per sequence: tokens of this call, and tokens in all (those before this call included)."""
    rng, ragged = _random(case), case.get("ragged", True)
    q_len, kv_len = [], []
    for b in range(case["seqs"]):
        first = b == 0 or not ragged
        few = case["q"] if first or case["q"] < 4 else rng.randrange(1, case["q"] + 1)
        q_len.append(few)
        kv_len.append(case.get("kv", few) if first else rng.randrange(few, max(few, case.get("kv", few)) + 1))
    return q_len, kv_len


def _sums(lengths):
    return [0] + np.cumsum(lengths).tolist()


def _trees(rng, q_len):
    """Random trees of drafted tokens: each token's parent among its sequence's tokens (-1: the first)."""
    return [[-1] + [rng.randrange(0, i) for i in range(1, n)] for n in q_len]


def _tree_bits(trees, words):
    """Each token sees itself and its ancestors, as bits over its sequence's tokens."""
    rows = []
    for up in trees:
        seen = []
        for i, p in enumerate(up):
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        rows += seen
    word = [[(r >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for r in rows]
    return np.array(word, dtype=np.uint64).reshape(len(rows), words).view(np.int64)


def _table(rng, kv_len, page, spare=3):
    """A block table over pages in random order, and their number."""
    need = [-(-k // page) for k in kv_len]
    order = list(range(sum(need) + spare))
    rng.shuffle(order)
    table = np.full((len(need), max(max(need), 1)), -1, np.int32)  # -1: no page there yet
    for b, k in enumerate(need):
        table[b, :k] = [order.pop() for _ in range(k)]
    return table, sum(need) + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES.get(case.get("dtype"))
    normal = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)  # noqa: E731
    ints = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    some = lambda *shape: torch.randint(-2 ** 31, 2 ** 31, (*shape[:-1], shape[-1] // 4), generator=g, device="cuda", dtype=torch.int32).view(torch.uint8)  # noqa: E731
    s = {"case": case, "op": case["op"]}

    if case["op"] == "turnover":
        return s | _turnover(case, rng, ints)
    if case["op"] == "beam":
        return s | _beam(case, rng, ints, some, normal, dt)

    q_len, kv_len = _lengths(case)
    cu, n = _sums(q_len), sum(q_len)
    s["cu_q"], s["max_q"], s["max_kv"] = ints(cu), max(q_len), max(kv_len)
    s["seq"] = torch.tensor(np.repeat(np.arange(len(q_len)), q_len), device="cuda")
    s["nth"] = torch.tensor(np.concatenate([np.arange(k) for k in q_len]), device="cuda")
    if case["op"] == "verify":
        return s | _drafts(case, q_len, rng, g, normal)

    latent, page = case["latent"], case["page"]
    table, pages = _table(rng, kv_len, page)
    s["kv_len"], s["table"] = ints(kv_len), ints(table)
    if case["op"] == "compact":
        shape = (case["layers"], pages, page)
        s["cache"] = some(*shape, latent + BYTES) if case["dtype"] == "u8" else normal(*shape, latent + ROPE, dtype=dt)
        keep = np.zeros(n, np.int32)
        kept = [rng.randrange(1, min(case["keep"], k) + 1) if b else min(case["keep"], k) for b, k in enumerate(q_len)]
        for b, k in enumerate(kept):  # the first, and an ascending choice of the others
            keep[cu[b]:cu[b] + k] = [0] + sorted(rng.sample(range(1, q_len[b]), k - 1))
        s["keep"], s["n_keep"], s["most"] = ints(keep), ints(kept), case["keep"]
        return s

    # an 8-bit cache as the append leaves it: latents of normed tokens, some channels larger than others
    width = torch.exp(0.4 * normal(latent))
    s["cache"] = torch.empty(pages, page, latent + BYTES, dtype=torch.uint8, device="cuda")
    for at in range(0, pages, 512):  # (a part at a time: the values in 32 bits take eight times the cache)
        part = s["cache"][at:at + 512]
        part.copy_(_to_bytes(normal(*part.shape[:2], latent) * width, normal(*part.shape[:2], ROPE, dtype=dt)))
    if case["op"] == "append8":
        s["freq"], s["interleaved"] = torch.from_numpy(10000.0 ** (-np.arange(ROPE // 2) * 2.0 / ROPE)).cuda(), case["interleaved"]
        s["rows"] = normal(n, latent + ROPE, dtype=DTYPES[case["source"]])
        s["weight"] = width if case["norm"] else None
        s["positions"] = s["kv_len"].long()[s["seq"]] - ints(q_len).long()[s["seq"]] + s["nth"]
        return s
    h = case["heads"]
    s["ql"], s["qr"], s["scale"] = normal(n, h, latent, dtype=dt), normal(n, h, ROPE, dtype=dt), 192 ** -0.5
    s["tree"] = None
    if case["mask"] == "tree":
        s["tree"] = torch.from_numpy(_tree_bits(_trees(rng, q_len), -(-max(q_len) // 64))).cuda()
    return s


def _drafts(case, q_len, rng, g, normal):
    """Distributions of a target and of a draft that is near it, tokens drawn from the draft (trees: its most likely, a
    different one for each child of a token), and the random numbers."""
    n, vocab = sum(q_len), case["vocab"]
    logits = 3.0 * normal(n, vocab)
    draft = logits + 0.5 * normal(n, vocab)
    s = {"target": torch.softmax(logits, -1), "uniform": torch.rand(n, generator=g, device="cuda")}
    trees = _trees(rng, q_len) if case["tree"] else [list(range(-1, k - 1)) for k in q_len]
    start = _sums(q_len)
    up = torch.tensor(np.concatenate([[start[b] + max(p, 0) for p in t] for b, t in enumerate(trees)]), device="cuda")
    if case["tree"]:
        rank = torch.tensor(np.concatenate([[t[:i].count(p) for i, p in enumerate(t)] for t in trees]), device="cuda")
        best = torch.topk(draft, min(vocab, 64), -1).indices
        s["tokens"] = best[up, rank]
        s["parents"] = torch.tensor(np.concatenate(trees), dtype=torch.int32, device="cuda")
        s["ancestors"], s["older"] = _relations(trees, case["q"])
    else:
        noise = -torch.log(-torch.log(torch.rand(n, vocab, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
        s["tokens"] = (draft + noise).argmax(-1)[up]
        s["draft"] = torch.softmax(draft, -1)
    return s


def _relations(trees, most):
    """[sequence, token, token]: the second is an ancestor of the first or itself; is an earlier child of the first's parent."""
    above, older = np.zeros((2, len(trees), most, most), bool)
    for b, t in enumerate(trees):
        for i, p in enumerate(t):
            above[b, i, i] = True
            if p >= 0:
                above[b, i] |= above[b, p]
                older[b, i, [k for k in range(1, i) if t[k] == p]] = True
    return torch.from_numpy(above).cuda(), torch.from_numpy(older).cuda()


def _turnover(case, rng, ints):
    """A pool whose pages are in use in random order; some sequences end, and as many of the same lengths begin."""
    of = _random(case)
    lens = [case["kv"]] + [of.randrange(0, case["kv"] + 1) for _ in range(case["seqs"] - 1)]
    page, pool = case["page"], case["pool"]
    table, _ = _table(rng, lens, page, pool - sum(-(-k // page) for k in lens))
    wide = np.full((len(lens), -(-case["kv"] // page) + 1), -1, np.int32)
    wide[:, :table.shape[1]] = table
    refs = np.zeros(pool, np.int32)
    np.add.at(refs, wide[wide >= 0], 1)
    moved = rng.sample(range(len(lens)), case["moved"])
    again = rng.sample(moved, len(moved))  # the new ones take their slots in another order
    return {"table": ints(wide), "lens": ints(lens), "refs": ints(refs), "page": page, "ended": ints(moved),
            "none": ints([0] * len(moved)), "begun": ints(again), "new": ints([lens[b] for b in again])}


def _beam(case, rng, ints, some, normal, dt):
    """`seqs` sequences in the first slots, their branches in those behind."""
    of = _random(case)
    lens = [case["kv"]] + [of.randrange(1, case["kv"] + 1) for _ in range(case["seqs"] - 1)]
    page, each = case["page"], case["branches"]
    slots = case["seqs"] * (1 + each)
    table, pages = _table(rng, lens, page, 2 * case["seqs"] * each + 3)
    wide = np.full((slots, -(-case["kv"] // page) + 1), -1, np.int32)
    wide[:case["seqs"], :table.shape[1]] = table
    refs = np.zeros(pages, np.int32)
    np.add.at(refs, wide[wide >= 0], 1)
    child = list(range(case["seqs"], slots))
    parent = [k // each for k in range(len(child))]
    shape = (case["layers"], pages, page)
    cache = some(*shape, case["latent"] + BYTES) if dt is None else normal(*shape, case["latent"] + ROPE, dtype=dt)
    return {"table": ints(wide), "lens": ints(lens + [0] * len(child)), "refs": ints(refs), "page": page, "cache": cache,
            "parent": ints(parent), "child": ints(child), "none": ints([0] * len(child)), "longer": ints([lens[p] + 1 for p in parent])}


# ------------------------------------------------------------------ one pass: the 8-bit cache

def _to_bytes(latents, rope):
    """Rows of an 8-bit cache: latents [.., latent] in 32 bits, rotated parts [.., 64] in 16."""
    top = latents.abs().amax(-1, keepdim=True)
    part, exponent = torch.frexp(top)  # top = part * 2^exponent, part in [0.5, 1): the smallest scale that fits 448
    exponent = torch.where(top > 0, exponent - 9 + (part > TOP / 512.0), LOWEST).clamp(LOWEST, HIGHEST)
    eight = torch.ldexp(latents, -exponent).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    scale = (exponent + 127).to(torch.uint8)
    rest = torch.zeros(*latents.shape[:-1], 15, dtype=torch.uint8, device=latents.device)
    return torch.cat((eight.view(torch.uint8), rope.contiguous().view(torch.uint8), scale, rest), -1)


def _parts(rows, dtype):
    """Rows of bytes as latents, scales and rotated parts, each in its own type."""
    latent = rows.shape[-1] - BYTES
    return (rows[..., :latent].view(torch.float8_e4m3fn), rows[..., latent + 2 * ROPE:latent + 2 * ROPE + 1].view(torch.float8_e8m0fnu),
            rows[..., latent:latent + 2 * ROPE].view(dtype))


def _from_bytes(rows, dtype):
    eight, _, rope = _parts(rows, dtype)
    scale = (rows[..., -16].int() << 23).view(torch.float32)
    return torch.cat((eight.float() * scale[..., None], rope.float()), -1)


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)


def _plain_append(s):
    cache, latent, page = s["cache"], s["cache"].shape[-1] - BYTES, s["cache"].shape[1]
    x = s["rows"].float()
    c, r = x[:, :latent], x[:, latent:]
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    a = s["positions"].double()[:, None] * s["freq"]  # 64 bits: float32 has no fraction left for far positions
    r = _rotate(r, a.cos().float(), a.sin().float(), s["interleaved"]).to(DTYPES[s["case"]["dtype"]])
    at = s["kv_len"][s["seq"]].long() - (s["cu_q"][s["seq"] + 1] - s["cu_q"][s["seq"]]).long() + s["nth"]
    cache[s["table"][s["seq"], at // page].long(), at % page] = _to_bytes(c, r)
    return cache


def _softmax(x, seen):
    """Weights that are not yet divided by their sum, the sum, and the logarithm of the sum of exponentials."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def _plain_attn(s):
    cache, latent, page = s["cache"], s["cache"].shape[-1] - BYTES, s["cache"].shape[1]
    n, h = s["ql"].shape[:2]
    b, most_q, most_k = s["kv_len"].shape[0], s["max_q"], s["max_kv"]
    j = torch.arange(most_k, device="cuda")
    i = torch.arange(most_q, device="cuda")
    keys = _from_bytes(cache[s["table"][:, j // page].long().clamp(min=0), j % page], s["ql"].dtype)  # [b, k, latent + rope]
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
    o = torch.where(total > 0, o / total, torch.zeros_like(o))[s["seq"], s["nth"]]
    return o.to(s["ql"].dtype), lse[s["seq"], s["nth"]]


# ------------------------------------------------------------------ one pass: drafted tokens

def _plain_verify(s):
    """[b, q]: a sequence's tokens side by side. Sums and products that are compared are of 64 bits."""
    n, b, most = s["tokens"].shape[0], s["cu_q"].shape[0] - 1, s["max_q"]
    i = torch.arange(most, device="cuda")
    few = (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None]
    token = (s["cu_q"][:-1, None].long() + i).clamp(max=n - 1)
    real = i < few
    x, u = s["tokens"][token], s["uniform"][token].double()
    if "draft" in s:
        before = (token - 1).clamp(min=0)
        p, q = s["target"][before, x].double(), s["draft"][before, x].double()
        taken = (u * q < p) & real
        taken[:, 0] = True
        reached = taken.long().cumprod(-1).bool()
        last = reached.sum(-1) - 1
        row = s["cu_q"][:-1].long() + last
        weights = s["target"][row].double()
        rest = torch.where((last + 1 < few[:, 0])[:, None], (weights - s["draft"][row].double()).clamp(min=0), weights)
    else:
        parent = s["parents"][token].long().clamp(min=0)
        above, older = s["ancestors"][:, :most, :most], s["older"][:, :most, :most]
        p = torch.where(real, s["target"][torch.gather(token, 1, parent), x].double(), 0.0)
        mass = 1.0 - (older * p[:, None, :]).sum(-1)  # what the earlier children of the token's parent leave
        would = (u * mass < p) & real
        would[:, 0] = True
        chosen = would & ~(older & would[:, None, :]).any(-1)
        reached = ~(above & ~chosen[:, None, :]).any(-1) & real
        last = (reached * (i + 1)).amax(-1) - 1
        row = s["cu_q"][:-1].long() + last
        weights = s["target"][row].double()
        out = torch.zeros_like(weights).scatter_add_(1, x, ((parent == last[:, None]) & real & (i > 0)).double())
        rest = torch.where(out > 0, 0.0, weights)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, weights)
    sums = rest.cumsum(-1)
    number = s["uniform"][s["cu_q"][:-1].long()].double()
    following = torch.searchsorted(sums, (number * sums[:, -1])[:, None], right=True)[:, 0]
    kept = reached.sum(-1)
    place = torch.where(reached, reached.long().cumsum(-1) - 1, most)  # an accepted token's place on the path
    path = torch.full((b, most + 1), -1, dtype=torch.int32, device="cuda").scatter_(1, place, i.int().expand(b, most))
    return path[s["seq"], s["nth"]], kept.int(), following


# ------------------------------------------------------------------ one pass: places and pages

def _plain_compact(s):
    cache, page = s["cache"], s["cache"].shape[2]
    i = torch.arange(s["most"], device="cuda")
    few = (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None]
    nth = torch.where(i < s["n_keep"][:, None], i, 0)  # behind the last: the first once more, in its own place
    keep = s["keep"][s["cu_q"][:-1, None].long() + nth].long()
    base = s["kv_len"][:, None].long() - few
    row = lambda j: torch.gather(s["table"], 1, j // page).long() * page + j % page  # noqa: E731
    flat = cache.view(cache.shape[0], -1, cache.shape[3])
    flat[:, row(base + nth)] = flat[:, row(base + keep)]
    return cache


def _plain_resize(s, slots, lengths):
    """Pages of the given slots for their new lengths; pairs of pages to be copied. (Here there is always room.)"""
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    at, new = slots.long(), lengths.long()
    old = lens[at].long()
    had, has = -(-old // page), -(-new // page)
    last = (had - 1).clamp(min=0)
    end = torch.gather(table[at], 1, last[:, None])[:, 0]
    shared = (new > old) & (old % page != 0) & (refs[end.long().clamp(min=0)] > 1)
    need = (has - had).clamp(min=0) + shared
    first = need.cumsum(0) - need
    free = (refs == 0).cumsum(0)
    take = lambda rank: torch.searchsorted(free, rank + 1)  # noqa: E731
    e = torch.arange(table.shape[1], device="cuda")
    fresh = (e >= had[:, None]) & (e < has[:, None])
    mine = shared[:, None] & (e == last[:, None])
    rank = first[:, None] + torch.where(mine, 0, shared[:, None] + e - had[:, None])
    rows = table[at]
    taken = take(rank.clamp(min=0)).int()
    gone = (mine | ((e >= has[:, None]) & (e < had[:, None]))) & (rows >= 0)
    count = torch.zeros_like(refs).index_add_(0, rows.clamp(min=0).flatten().long(), gone.flatten().int())
    refs -= count
    got = fresh | mine
    refs.index_add_(0, torch.where(got, taken, 0).flatten().long(), got.flatten().int())
    table[at] = torch.where(got, taken, torch.where(e >= has[:, None], -1, rows))
    lens[at] = new.int()
    return torch.where(shared[:, None], torch.stack((end, take(first).int()), -1), -1)


def _plain_fork(s):
    rows = s["table"][s["parent"].long()]
    s["table"][s["child"].long()] = rows
    s["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().int())
    s["lens"][s["child"].long()] = s["lens"][s["parent"].long()]


def _plain_copy(s, pairs):
    pairs = torch.where((pairs[:, :1] >= 0), pairs, s["table"][0, 0]).long()  # no copy: a page in use onto itself
    s["cache"][:, pairs[:, 1]] = s["cache"][:, pairs[:, 0]]


def _pages(s, turnover):
    """Sequences end and begin, or branches are made anew and grow into their own copies of the last pages."""
    if own:
        import deepseek_v4_hyper_amd as ds4hc
        pool = s["table"], s["lens"], s["refs"], s["page"]
        if turnover:
            ds4hc.ds4hc_pages_resize(*pool, s["ended"], s["none"])
            ds4hc.ds4hc_pages_resize(*pool, s["begun"], s["new"])
            return s["table"], s["lens"], s["refs"]
        ds4hc.ds4hc_pages_resize(*pool, s["child"], s["none"])
        ds4hc.ds4hc_pages_fork(*pool, s["parent"], s["child"])
        pairs, _ = ds4hc.ds4hc_pages_resize(*pool, s["child"], s["longer"])
        ds4hc.ds4hc_pages_copy(s["cache"], pairs)
        return s["table"], s["lens"], s["refs"], pairs, s["cache"]
    if turnover:
        _plain_resize(s, s["ended"], s["none"])
        _plain_resize(s, s["begun"], s["new"])
        return s["table"], s["lens"], s["refs"]
    _plain_resize(s, s["child"], s["none"])
    _plain_fork(s)
    pairs = _plain_resize(s, s["child"], s["longer"])
    _plain_copy(s, pairs)
    return s["table"], s["lens"], s["refs"], pairs, s["cache"]


def run(s):
    op = s["op"]
    if op in ("turnover", "beam"):
        return _pages(s, op == "turnover")
    if own:
        import deepseek_v4_hyper_amd as ds4hc
        if op == "append8":
            dtype = DTYPES[s["case"]["dtype"]]
            return _parts(ds4hc.ds4hc_latent_append8(s["rows"], s["positions"], s["freq"], s["cache"], s["cu_q"], s["kv_len"],
                                                     s["table"], dtype=dtype, norm_weight=s["weight"], rms_eps=1e-6,
                                                     interleaved=s["interleaved"]), dtype)
        if op == "attn8":
            return ds4hc.ds4hc_latent_attn8(s["ql"], s["qr"], s["cache"], s["cu_q"], s["kv_len"], s["table"],
                                            scale=s["scale"], tree_mask=s["tree"], want_lse=True)
        if op == "verify":
            return ds4hc.ds4hc_draft_verify(s["target"], s["tokens"], s["cu_q"], s["uniform"], draft=s.get("draft"),
                                            parents=s.get("parents"))
        return ds4hc.ds4hc_cache_compact(s["cache"], s["cu_q"], s["kv_len"], s["table"], s["keep"], s["n_keep"])
    if op == "append8":
        return _parts(_plain_append(s), DTYPES[s["case"]["dtype"]])
    if op == "attn8":
        return _plain_attn(s)
    return _plain_verify(s) if op == "verify" else _plain_compact(s)


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    return case["latent"] + BYTES if case["dtype"] == "u8" else (case["latent"] + ROPE) * 2


def work(case):
    op = case["op"]
    if op == "turnover":  # the moved slots' entries and their pages' counts, each written twice; their lengths
        of = _random(case)
        lens = [case["kv"]] + [of.randrange(0, case["kv"] + 1) for _ in range(case["seqs"] - 1)]
        entries = case["moved"] * sum(-(-k // case["page"]) for k in lens) / len(lens)  # (which slots: by the seed)
        return {"bytes": 16 * entries + 16 * case["moved"], "flops": 2 * entries}
    if op == "beam":  # a page read and written for each branch and layer, less those that end with a page
        of = _random(case)
        lens = [case["kv"]] + [of.randrange(1, case["kv"] + 1) for _ in range(case["seqs"] - 1)]
        copies = case["branches"] * sum(k % case["page"] != 0 for k in lens)
        entries = case["branches"] * sum(-(-k // case["page"]) for k in lens)
        return {"bytes": 2 * copies * case["layers"] * case["page"] * _row_bytes(case) + 16 * entries, "flops": 2 * entries}
    q_len, kv_len = _lengths(case)
    n = sum(q_len)
    if op == "verify":  # one row of each distribution a sequence (a chain's last one: the target's alone), and the numbers
        rows = len(q_len) * (1 if case["tree"] else 2)
        return {"bytes": 4 * rows * case["vocab"] + 28 * n, "flops": rows * case["vocab"]}
    if op == "compact":
        kept = len(q_len) * (case["keep"] + 1) / 2  # (how many: by the seed, and the first stays in place)
        return {"bytes": 2 * kept * case["layers"] * _row_bytes(case) + 8 * kept, "flops": kept}
    row, h = case["latent"] + ROPE, case.get("heads")
    stored = case["latent"] + 2 * ROPE + 1
    if op == "append8":
        return {"bytes": n * (row * SIZE[case["source"]] + stored) + 12 * n + 4 * case["latent"], "flops": 5 * n * row}
    if case["mask"] == "tree":  # a token of a random tree sees few of the others: the context is what counts
        pairs = sum(q * (k - q) for q, k in zip(q_len, kv_len))
    else:
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(q_len, kv_len))
    return {"bytes": sum(kv_len) * stored + n * h * ((row + case["latent"]) * 2 + 4), "flops": 2 * h * pairs * (row + case["latent"])}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _decode(rows, dtype):
    """The values that bytes stand for, from their bits: a sign, four bits of exponent, three of fraction."""
    latent = rows.shape[-1] - BYTES
    w = rows[..., :latent].long()
    e, f = (w >> 3) & 15, (w & 7).double()
    value = torch.where(e > 0, (8.0 + f) * torch.exp2(e.double() - 10.0), f * 2.0 ** -9)
    value = torch.where(w >= 128, -value, value) * torch.exp2(rows[..., latent + 2 * ROPE].double() - 127.0)[..., None]
    return value, rows[..., latent:latent + 2 * ROPE].contiguous().view(dtype).double()


def exact(case, seed):
    """Of what is stored in 8 bits: the values before their rounding, over the scale. Nothing for whole numbers."""
    if case["op"] not in ("append8", "attn8"):
        return None
    s = prepare(case, seed)
    dtype, latent, page = DTYPES[case["dtype"]], case["latent"], case["page"]
    q_len, kv_len = _lengths(case)
    cu = _sums(q_len)
    flat = s["cache"].view(-1, latent + BYTES)
    if s["op"] == "append8":
        c, r = _decode(flat, dtype)
        scale = torch.exp2(flat[:, latent + 2 * ROPE].double() - 127.0)
        eight = c / scale[:, None]
        x = s["rows"].double()
        n = x[:, :latent]
        if s["weight"] is not None:
            n = n / torch.sqrt(n.square().sum(-1, keepdim=True) / latent + 1e-6) * s["weight"].double()
        half = ROPE // 2
        pair = x[:, latent:].unflatten(-1, (half, 2)) if case["interleaved"] else x[:, latent:].unflatten(-1, (2, half)).transpose(1, 2)
        a = s["positions"].double()[:, None] * s["freq"]
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(a), a))
        z = z.flatten(-2) if case["interleaved"] else z.transpose(1, 2).flatten(-2)
        power = torch.ceil(torch.log2(n.abs().amax(-1) / TOP))
        for b, (q, k) in enumerate(zip(q_len, kv_len)):
            j = torch.arange(k - q, k, device="cuda")
            at, here = s["table"][b, j // page].long() * page + j % page, slice(cu[b], cu[b + 1])
            scale[at] = torch.exp2(power[here])
            eight[at] = n[here] * torch.exp2(-power[here])[:, None]
            r[at] = z[here]
        shape = s["cache"].shape[:2]
        return eight.view(*shape, latent), scale.view(*shape, 1), r.view(*shape, ROPE)
    out, lse = [], []
    for b, (q, k) in enumerate(zip(q_len, kv_len)):
        j = torch.arange(k, device="cuda")
        values, rope = _decode(flat[s["table"][b, j // page].long() * page + j % page], dtype)
        keys = torch.cat((values, rope), -1)
        seen = j <= (k - q + torch.arange(q, device="cuda"))[:, None]  # [q, k]
        if s["tree"] is not None:
            bits = s["tree"][cu[b]:cu[b + 1]].tolist()
            own_part = [[row[d // 64] >> (d % 64) & 1 == 1 for d in range(q)] for row in bits]
            seen = torch.cat((torch.ones(q, k - q, dtype=torch.bool), torch.tensor(own_part)), -1).cuda()
        for i in range(q):
            t = cu[b] + i
            x = torch.cat((s["ql"][t], s["qr"][t]), -1).double() @ keys.T * s["scale"]
            x = torch.where(seen[i], x, -math.inf)
            m = torch.logsumexp(x, -1)
            out.append(torch.nan_to_num(torch.exp(x - m[:, None])) @ values)
            lse.append(m)
    return torch.stack(out), torch.stack(lse)
