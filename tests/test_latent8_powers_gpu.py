"""Attention over a cache of 8-bit latents where the tokens' powers of 2 lie far apart, against 64-bit references (bounds
derived in site_testlib)."""
import math

import pytest
import torch

from deepseek_v4_hyper_amd import binding as B
from hc_testlib import say
from site_testlib import E32, assert_attention, attend64

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def many_beside_one(dtype, latent, page, n, kind, g):
    """A cache of one sequence: n tokens of logit 0 and, as its fourth, one of `latent` ordinary values whose rotated key is
    (4, 0, ..). kind "zero": half of the n are rows of a zeroed cache, half zero latents that were appended; "tiny": latents
    of sizes near 2^-105. Returns the cache, its table, and the one token's values."""
    pages = -(-(n + 1) // page)
    cache = torch.zeros(pages, page, latent + 144, dtype=torch.uint8, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    f = B.ds4hc_rope_frequencies(64)[0].cuda()

    def append(rows, end):
        B.ds4hc_latent_append8(rows, torch.zeros(len(rows), dtype=torch.int64, device="cuda"), f, cache, i32([0, len(rows)]),
                               i32([end]), table, dtype=dtype)

    few = n + 1 if kind == "tiny" else n // 2
    rows = torch.zeros(few, latent + 64, device="cuda")
    if kind == "tiny":
        rows[:, :latent] = torch.randn(few, latent, generator=g, device="cuda") * 2.0 ** -105
    append(rows, n + 1)
    at = 3
    one = torch.zeros(1, latent + 64, device="cuda")
    one[0, :latent] = torch.randn(latent, generator=g, device="cuda")
    one[0, latent] = 4.0
    append(one, at + 1)
    row = cache.view(-1, latent + 144)[table[0, at // page].long() * page + at % page]
    values = row[:latent].view(torch.float8_e4m3fn).double() * 2.0 ** (int(row[latent + 128]) - 127)
    return cache, table, values


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["zero", "tiny"])
@pytest.mark.parametrize("power,seqs", [(10, 1), (10, 256), (14, 24), (14, 256), (18, 24), (18, 256), (22, 24), (22, 256)])
@pytest.mark.parametrize("heads,latent,page", [(16, 512, 64), (64, 128, 16), (128, 512, 64), (128, 128, 8)])
def test_attn8_tokens_that_weigh_but_add_nothing(dtype, kind, power, seqs, heads, latent, page):
    """A quarter of 2^power tokens, each with 2^-power of the largest weight and a latent of zeros, or next to it: they add
    nothing to a row, but a fifth of its weight is theirs. Of 256 sequences each is one part, of fewer several."""
    if power == 22 and latent != 128:
        pytest.skip("700 MB of cache; smaller latents have the same tiles")
    say(f"[gpu] attn8 {kind} latents {dtype} 2^-{power} seqs={seqs} heads={heads} latent={latent} page={page}")
    g = torch.Generator(device="cuda").manual_seed(power + heads)
    n = 2 ** power // 4
    cache, table, values = many_beside_one(dtype, latent, page, n, kind, g)
    qr = torch.zeros(seqs, heads, 64, dtype=dtype, device="cuda")
    qr[..., 0] = power * math.log(2.0) / 4 * torch.linspace(1.0, 0.95, heads, device="cuda")
    out, lse = B.ds4hc_latent_attn8(torch.zeros(seqs, heads, latent, dtype=dtype, device="cuda"), qr, cache,
                                    torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), i32([n + 1] * seqs),
                                    table.expand(seqs, -1).contiguous(), scale=1.0, want_lse=True)
    x = qr[0, :, 0].double() * 4.0
    rest = n * torch.exp(-x)
    want = values / (1 + rest)[:, None]
    ref = [t.cpu() for t in (want, x + torch.log1p(rest), want.abs(), (latent + 72) * E32 * x)]
    for b in range(0, seqs, 17):
        assert_attention(out[b].cpu(), lse[b].cpu(), ref, [n + 1] * heads, dtype, f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_attn8_every_scale_byte(dtype, heads):
    """A sequence for each scale byte, of one token with values of +-2^-9 times its power, the smallest there are: bytes outside
    10..246 are taken as the nearest of these, values are exact, in float16 infinite beyond 65504, and 255 is a NaN. (Queries are
    zeros where the values are beyond 2^16: logits beyond 2^30 are not promised.)"""
    say(f"[gpu] attn8 scale bytes {dtype} heads={heads}")
    page, d, n = 16, 128, 256
    cache = torch.full((n, page, d + 144), 0x7F, dtype=torch.uint8)
    cache[:, 0] = 0
    cache[:, 0, 0:d:3], cache[:, 0, 1:d:3] = 0x01, 0x81
    cache[:, 0, d + 128] = torch.arange(n).to(torch.uint8)
    cache[:, 1:, d + 128] = 255
    ql, qr = torch.zeros(n, heads, d, dtype=dtype), torch.zeros(n, heads, 64, dtype=dtype)
    ql[:153, :, 0] = 2.0 ** -12 * torch.linspace(0.5, 1.0, heads)
    out, lse = B.ds4hc_latent_attn8(ql.cuda(), qr.cuda(), cache.cuda(), torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                                    i32([1] * n), torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(), scale=1.0,
                                    want_lse=True)
    out, lse = out.cpu(), lse.cpu()
    for b in range(n):
        value = 2.0 ** -9 * 2.0 ** (min(max(b, 10), 246) - 127)
        if b == 255 or dtype == HF and value > 65504:
            assert not torch.isfinite(out[b].float()).all(-1).any(), b
            continue
        key = torch.zeros(1, d + 64, dtype=torch.float64)
        key[0, 0:d:3], key[0, 1:d:3] = value, -value
        ref = attend64(torch.cat((ql[b], qr[b]), -1), key, key[:, :d], torch.ones(heads, 1, dtype=torch.bool), 1.0)
        # (half of float16's smallest number, where values and results are multiples of that)
        small = 2.0 ** -25 if dtype == HF else 0.0
        keep = (out[b].double() - ref[0]).abs() > small
        assert_attention(torch.where(keep, out[b].double(), ref[0]), lse[b], ref, [1] * heads, dtype, f"scale byte {b}")
