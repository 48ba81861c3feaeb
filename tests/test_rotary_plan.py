"""The rotary plan's frequencies against 60-digit decimal arithmetic (host only):
the relative error that the library documents, for bands whose exponents fp64
does not hold, long contexts and large bases."""

import math
from decimal import Decimal, getcontext

import pytest

import streaming_attention_block_gb300 as sab

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def _turns(bands, base, scaling, s, c, fast, slow):
    """Turns per position of every pair, in units of 2^-64."""
    getcontext().prec = 60
    out = []
    for n in bands:
        for i in range(n // 2):
            x = (Decimal(-2 * i) / n * Decimal(base).ln()).exp()
            if scaling == sab.ROTARY_SCALE_BASE:
                x *= (Decimal(-2 * i) / (n - 2) * Decimal(s).ln()).exp()
            if scaling == sab.ROTARY_SCALE_LINEAR:
                x /= Decimal(s)
            if scaling == sab.ROTARY_SCALE_RAMP:
                w = (Decimal(c) * x / (2 * PI) - Decimal(slow)) / (Decimal(fast) - Decimal(slow))
                w = min(max(w, Decimal(0)), Decimal(1))
                x *= w + (1 - w) / Decimal(s)
            out.append(x / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 1.5, 1e30])
@pytest.mark.parametrize("scaling", [sab.ROTARY_SCALE_NONE, sab.ROTARY_SCALE_LINEAR, sab.ROTARY_SCALE_BASE,
                                     sab.ROTARY_SCALE_RAMP], ids=["none", "linear", "base", "ramp"])
def test_frequencies_to_the_documented_error(scaling, base):
    s, c, fast, slow = (1.0, 0.0, 32.0, 1.0) if scaling == sab.ROTARY_SCALE_NONE else (40.0, 4096.0, 32.0, 1.0)
    worst = 0.0
    for bands in ((44, 42, 42), (64,), (80,), (96,), (128,), (6, 10, 14), (254,), (256,)):
        p = sab.rotary_plan(bands, base=base, scaling=scaling, factor=s, original_context=c, ramp_fast=fast,
                            ramp_slow=slow)
        for j, want in enumerate(_turns(bands, base, scaling, s, c, fast, slow)):
            # rounding to whole 2^-64 turns: half of one
            worst = max(worst, float((abs(Decimal(p.step[j]) - want) - Decimal("0.5000001")) / want))
    # in units of 2^-53: a power 2 and its correction 1, the constant 2 pi and the
    # quotient by it 1.4, the quotient by s 1: below 6 (2^-50.4) at worst, and below
    # 4 (2^-51) with a pow that is right to 0.6 units in the last place, as both
    # machines' is; a second power and its product make that below 8.  By-parts
    # scaling adds the weight's rounding, up to factor * fast / (fast - slow) as large
    limit = 2.0 ** -51 if scaling in (sab.ROTARY_SCALE_NONE, sab.ROTARY_SCALE_LINEAR) else 2.0 ** -50
    if scaling == sab.ROTARY_SCALE_RAMP:
        limit *= 1 + s * fast / (fast - slow)
    assert worst <= limit, f"2^{math.log2(worst):.2f}"


def test_a_magnitude_that_fp32_holds_as_zero_is_refused():
    """It would turn every pair to zero without an error."""
    for bad in (1e-60, 7e-46):
        with pytest.raises(sab.SabError):
            sab.rotary_plan((64,), magnitude=bad)
    assert sab.rotary_plan((64,), magnitude=2e-45).magnitude > 0
