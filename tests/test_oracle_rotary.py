"""Pins of the rotary oracle: the existing interleaved three-band oracle, a
complex-number restatement, integer reduction of far angles, the transpose
property, and the plan's fixed-point frequencies (host only)."""

import math

import numpy as np
import pytest

import streaming_attention_block_gb300 as sab
from oracle import qkrope as OQ
from oracle import rotary as OR

SCALINGS = {None: sab.ROTARY_SCALE_NONE, "linear": sab.ROTARY_SCALE_LINEAR, "base": sab.ROTARY_SCALE_BASE,
            "ramp": sab.ROTARY_SCALE_RAMP}


def test_equals_the_three_band_oracle():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 24, 2, 16))
    pos = OQ.positions(3, 24, (2, 3, 4))  # [24, 3]
    f, ax = OR.frequencies((8, 4, 4))
    got = OR.rotate(x, OR.angles(pos.T[:, None].astype(np.int64), f, ax), half=False)
    assert np.allclose(got, OQ.rope(x, OQ.angles(pos, (8, 4, 4))), atol=1e-13)


@pytest.mark.parametrize("half", [False, True])
def test_equals_complex_products(half):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 5, 3, 10))
    pos = rng.integers(-1000, 1000, (1, 2, 5))
    f, ax = OR.frequencies((6,))
    y = OR.rotate(x, OR.angles(pos, f, ax), half, magnitude=1.5)
    for i in range(3):
        j0, j1 = (i, i + 3) if half else (2 * i, 2 * i + 1)
        z = (x[..., j0] + 1j * x[..., j1]) * 1.5 * np.exp(1j * pos[0].astype(float)[:, :, None] * 10000.0 ** (-2 * i / 6))
        assert np.allclose(y[..., j0] + 1j * y[..., j1], z, atol=1e-12)
    assert np.array_equal(y[..., 6:], x[..., 6:])


@pytest.mark.parametrize("half", [False, True])
def test_backward_is_the_transpose(half):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 1, 7, 2, 12))
    f, ax = OR.frequencies((4, 2, 2), scaling="linear", factor=3.0)
    ang = OR.angles(rng.integers(0, 50, (3, 1, 7)), f, ax)
    y, dx = OR.rotate(x, ang, half, 1.25), OR.rotate(dy, ang, half, 1.25, backward=True)
    assert abs((y * dy).sum() - (x * dx).sum()) < 1e-12
    h = 1e-4  # central differences (the map is linear: exact up to rounding)
    for idx in [(0, 0, 0, 0), (0, 3, 1, 5), (0, 6, 0, 11)]:
        e = np.zeros_like(x)
        e[idx] = h
        num = ((OR.rotate(x + e, ang, half, 1.25) - OR.rotate(x - e, ang, half, 1.25)) * dy).sum() / (2 * h)
        assert abs(num - dx[idx]) < 1e-9


def test_far_angles_by_integer_powers():
    """Angle of position 2^k by repeated doubling of the rotation."""
    f, ax = OR.frequencies((8,))
    z = np.exp(1j * np.asarray(f, dtype=np.clongdouble))
    for k in range(41):
        if k in (0, 10, 20, 21, 33, 40):
            ang = OR.angles(np.full((1, 1, 1), 1 << k), f, ax)[0, 0]
            # each doubling doubles the error of the long double start
            assert np.all(np.abs(np.exp(1j * ang) - z) < 1e-14 + 2.0 ** (k - 58))
        z = z * z


def test_scalings_by_hand():
    f, _ = OR.frequencies((4,), base=100.0)
    assert np.allclose(f.astype(float), [1.0, 0.1])
    assert np.allclose(OR.frequencies((4,), 100.0, "linear", 4.0)[0].astype(float), [0.25, 0.025])
    assert np.allclose(OR.frequencies((4,), 100.0, "base", 4.0)[0].astype(float), [1.0, 1600.0 ** -0.5])
    # c = 20 pi: 10 turns and 1 turn; slow 2, fast 18 -> weights 0.5 and 0
    r = OR.frequencies((4,), 100.0, "ramp", 4.0, 20 * math.pi, fast=18.0, slow=2.0)[0].astype(float)
    assert np.allclose(r, [0.5 + 0.5 / 4, 0.1 / 4])


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("bands", [(128,), (44, 42, 42), (4,), (256,), (6, 8)])
def test_plan_frequencies(scaling, bands):
    """The plan's 2^-64 turns: fp64 pow and a few products, 2^-50 relative."""
    p = sab.rotary_plan(bands, scaling=SCALINGS[scaling], factor=1.0 if scaling is None else 8.0,
                        original_context=4096.0)
    f, ax = OR.frequencies(bands, scaling=scaling, factor=8.0, context=4096.0)
    n = sum(bands) // 2
    assert p.dims == 2 * n and p.axes == len(bands) and list(p.axis)[:n] == list(ax)
    got = np.array([int(x) for x in p.step[:n]], dtype=np.longdouble)
    want = f / (2 * np.arctan2(np.longdouble(0), np.longdouble(-1))) * np.longdouble(2) ** 64
    assert np.all(np.abs(got - want) <= want * 2.0 ** -50 + 1)


def test_plan_refusals():
    for kw in (dict(bands=(5,)), dict(bands=(0,)), dict(bands=()), dict(bands=(2, 2, 2, 2)), dict(bands=(258,)),
               dict(bands=(8,), layout=2), dict(bands=(8,), base=1.0), dict(bands=(8,), base=float("inf")),
               dict(bands=(8,), base=float("nan")), dict(bands=(8,), scaling=4), dict(bands=(8,), scaling=-1),
               dict(bands=(8,), scaling=1, factor=0.5), dict(bands=(8,), scaling=1, factor=float("nan")),
               dict(bands=(2,), scaling=2, factor=2.0), dict(bands=(8,), scaling=3, factor=2.0),
               dict(bands=(8,), scaling=3, factor=2.0, original_context=64, ramp_fast=1.0, ramp_slow=1.0),
               dict(bands=(8,), scaling=2, factor=1e300),
               dict(bands=(8,), magnitude=0.0), dict(bands=(8,), magnitude=float("inf"))):
        with pytest.raises(sab.SabError):
            sab.rotary_plan(**kw)
