"""The ramp of the rotary frequencies for long trained lengths, against fractions worked out
by hand and against what the ramp is for; needs no GPU."""
import math
from fractions import Fraction as F

import pytest

from deepseek_v4_hyper_amd import binding as B


def kept_of(dim, base, factor, length, **kw):
    """Per pair: its frequency over the one that is not stretched."""
    f, _ = B.ds4hc_rope_frequencies(dim, base, factor=factor, original_length=length, **kw)
    return [x / base ** (-2 * i / dim) for i, x in enumerate(f.tolist())]


# dim 64, base 10^4: pair i makes L / (2 pi) 10^(-i / 8) turns over the trained length L, so b turns lie at
# i = 8 log10(L / (2 pi b)).
@pytest.mark.parametrize("factor,length,lo,hi", [
    (16, 65536, 20, 33),      # 8 log10(325.95) = 20.1 and 8 log10(10430.4) = 32.15
    (4, 131072, 22, 35),      # 22.5, 34.6
    (40, 4096, 10, 23),       # 10.5, 22.5: both ends are among the pairs
    (8, 10 ** 6, 29, 42),     # 29.6, 41.6: only the last pairs are stretched
])
def test_ramp_ends_where_its_turns_do(factor, length, lo, hi):
    """The ramp runs from pair lo to pair hi, also where hi lies behind the last pair. pow and the
    quotient are off by a few last places."""
    got = kept_of(64, 10000.0, factor, length)
    for i, x in enumerate(got):
        k = F(1) - min(max(F(i - lo, hi - lo), F(0)), F(1))
        assert abs(x - float((1 - k) / factor + k)) <= 1e-13, i


@pytest.mark.parametrize("dim,base", [(64, 1e4), (128, 1e4), (64, 5e5), (128, 1e6), (32, 1e3)])
def test_pairs_of_more_turns_than_beta_slow_are_not_stretched_fully(dim, base):
    """A pair that makes more than beta_slow turns lies before the ramp's end, and one that makes
    more than beta_fast by a pair's step before its begin. Frequencies fall from pair to pair."""
    for length in (512, 4096, 16384, 50000, 65536, 131072, 262144, 10 ** 6):
        kept = kept_of(dim, base, 16.0, length)
        f = [x * base ** (-2 * i / dim) for i, x in enumerate(kept)]
        assert all(a > b for a, b in zip(f, f[1:]))
        for i, x in enumerate(kept):
            turns = length * base ** (-2 * i / dim) / (2 * math.pi)
            if turns > 1.0 + 1e-9:
                assert x > 1 / 16 + 1e-6, (length, i)
            if turns > 32.0 * base ** (2 / dim):
                assert x == pytest.approx(1.0, abs=1e-13), (length, i)
