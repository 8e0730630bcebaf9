"""How far the table of frequencies is off the formulas, against 60 decimal digits (host only)."""
from decimal import Decimal, getcontext

import pytest

import gated_deltanet_linear_spec_gb300 as gdn

getcontext().prec = 60


def pi():
    """16 atan(1/5) - 4 atan(1/239)."""
    def atan_of(n):
        term, total, k = Decimal(1) / n, Decimal(0), 0
        while abs(term) > Decimal(10) ** -58:
            total += (-1) ** k * term / (2 * k + 1)
            term /= n * n
            k += 1
        return total
    return 16 * atan_of(5) - 4 * atan_of(239)


PI = pi()
PLAIN, LINEAR, NTK, BANDS, RAMP = (gdn.GDN_ROPE_PLAIN, gdn.GDN_ROPE_LINEAR, gdn.GDN_ROPE_NTK, gdn.GDN_ROPE_BANDS, gdn.GDN_ROPE_RAMP)


def turns(rotary, base, scaling, factor, original):
    """Fractions of a turn a position."""
    base, factor, original, r = Decimal(base), Decimal(factor), Decimal(original), Decimal(rotary)
    of = lambda times: r * (original / (2 * PI * times)).ln() / (2 * base.ln())  # noqa: E731
    first = max(of(32).to_integral_value("ROUND_FLOOR"), 0)
    last = min(of(1).to_integral_value("ROUND_CEILING"), r - 1)
    if scaling == NTK and rotary > 2:
        base = base * (factor.ln() * r / (r - 2)).exp()
    out = []
    for i in range(rotary // 2):
        f = (-2 * i / r * base.ln()).exp()
        if scaling == LINEAR:
            f /= factor
        if scaling in (BANDS, RAMP):
            w = (original * f / (2 * PI) - 1) / 3 if scaling == BANDS else 1 - (i - first) / max(last - first, Decimal("0.001"))
            w = min(max(w, Decimal(0)), Decimal(1))
            f = w * f + (1 - w) * f / factor
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("rotary", [2, 6, 64, 90, 128, 254, 256])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0, 10000000.0])
@pytest.mark.parametrize("scaling,factor,original", [(PLAIN, 1, 1), (LINEAR, 8, 1), (NTK, 4, 1), (BANDS, 8, 8192), (RAMP, 40, 4096)])
def test_fractions_of_a_turn(rotary, base, scaling, factor, original):
    """At most 2^-53 of a turn: in units of 2^-53 turns, the power's last place, its exponent's rounding (0.37 of it: x e^-x), 2 pi's
    and the division's make 0.46, and the quotients and sums of a scaling four roundings of 1 / (2 pi) each more.  Where a
    weight between kept and divided frequencies has an error of its own (a few 2^-53 of it and of the logarithms), it
    moves them by as much of a frequency that is a tenth of a radian or less."""
    rope = gdn.Rope(rotary, base=base, scaling=scaling, factor=float(factor), original_len=float(original), device="cpu")
    for got, want in zip(rope.turns.tolist(), turns(rotary, base, scaling, factor, original)):
        off = abs(Decimal(got % (1 << 64)) / (1 << 64) - want)
        assert off <= Decimal(2) ** -53, float(off * (1 << 53))
