"""Rotary frequencies against 60 decimal digits, and what is left of their error at the farthest position.  CPU only."""
import math
from decimal import Decimal, localcontext

import pytest

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
SPECS = {
    "none": dict(),
    "linear": dict(scaling="linear", factor=4.0),
    "wavelength": dict(scaling="wavelength", factor=8.0, low=1.0, high=4.0, original_len=8192),
    "ramp": dict(scaling="ramp", factor=32.0, low=1.0, high=32.0, original_len=4096),
    "whole": dict(scaling="ramp", factor=32.0, low=1.0, high=32.0, original_len=4096, whole_pairs=True),
}


@pytest.fixture(scope="module")
def b():
    from paged_gqa_decode_step_gb300 import build
    build.build()
    from paged_gqa_decode_step_gb300 import binding
    return binding


def turns(theta, rot, scaling="none", factor=1.0, low=1.0, high=1.0, original_len=0, whole_pairs=False):
    """w_i / (2 pi) of every pair, from the definition."""
    with localcontext() as ctx:
        ctx.prec = 60
        pairs, factor, c = rot // 2, Decimal(factor), Decimal(original_len)
        log = Decimal(theta).ln()
        out = []
        for i in range(pairs):
            f = (-log * i / pairs).exp() / (2 * PI)
            s = Decimal(1)
            if scaling == "linear":
                s = Decimal(0)
            elif scaling == "wavelength":
                s = (c * f - Decimal(low)) / (Decimal(high) - Decimal(low))
            elif scaling == "ramp":
                ends = [pairs * (c / (2 * PI * Decimal(t))).ln() / log for t in (high, low)]
                if whole_pairs:
                    ends = [Decimal(min(max(round_(e), 0), rot - 1)) for e, round_ in zip(ends, (math.floor, math.ceil))]
                s = 1 - (i - ends[0]) / max(ends[1] - ends[0], Decimal("0.001"))
            s = min(max(s, Decimal(0)), Decimal(1))
            out.append(f * s + f / factor * (1 - s))
        return out


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("theta,rot", [(10000.0, 64), (500000.0, 128), (150000.0, 64), (1e7, 48), (1.5, 16)])
def test_frequencies_have_64_bits(b, theta, rot, spec):
    """In a format of 64 bits (rounding 2^-64 of a value): the logarithm, its product with i / pairs and the power are
    each off by 2^-64, the first two of an exponent of x <= log(theta), so a frequency, the product of two powers, by
    (2 x + 3) 2^-64 of itself, and e^-x (2 x + 3) <= 3; five more products and sums and 2 pi.  The share of a scaled one is off by as much times
    how steep it is: f by high / (high - low) on the wavelengths', and on the ramp's, whose ends (up to 128 pairs)
    are off by 6 roundings, by 128 * 6 over a width of two pairs at least, or by none where its ends are whole pairs.  The
    result is a whole number of 2^-64 turns, f at most 1 / (2 pi)."""
    r = b.make_rotary(128, theta, rot_dim=rot, **SPECS[spec])
    want = turns(theta, rot, **SPECS[spec])
    steep = {"wavelength": 4.0 * 4 / 3, "ramp": 384.0, "whole": 0.0}.get(spec, 0.0)
    off = (3 + 6 + steep) / (2 * math.pi) + 0.5
    worst = max(abs(Decimal(t) - w * 2 ** 64) for t, w in zip(r.turns, want))
    assert worst <= off, float(worst)


@pytest.mark.parametrize("spec", SPECS)
def test_angles_of_the_farthest_positions(b, spec):
    """Position 2^31 - 1 (any position that an int32 holds) is right to 2^-27 turns with what the kernel's f32 rest of an
    eighth of a turn leaves: 2^-28 turns and 2^-32 cut off leave 2^-29 for the frequency."""
    r = b.make_rotary(128, 500000.0, **SPECS[spec])
    pos = 2 ** 31 - 1
    for t, w in zip(r.turns, turns(500000.0, 128, **SPECS[spec])):
        off = (Decimal(pos * t) / 2 ** 64 - w * pos) % 1
        assert min(off, 1 - off) <= Decimal(2) ** -29, float(off)
