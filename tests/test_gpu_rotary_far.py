"""Rotary positions to 2^40 with bands whose frequencies fp64 rounds, against the
oracle's long double angles.

An angle is off by the position times the frequency's documented error (2^-50
of it, and 2^-65 turns for the fixed-point step); the rest as for near
positions: 2^-21 of |a| + |b| and one rounding to the output type."""

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import rotary as OR

NAMES = {None: sab.ROTARY_SCALE_NONE, "linear": sab.ROTARY_SCALE_LINEAR, "base": sab.ROTARY_SCALE_BASE,
         "ramp": sab.ROTARY_SCALE_RAMP}


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", NAMES, ids=lambda s: s or "none")
@pytest.mark.parametrize("bands", [(44, 42, 42), (80,), (6, 10, 14)])
def test_far_positions(bands, scaling):
    dims, D = sum(bands), 128
    s = 1.0 if scaling is None else 8.0
    plan = sab.rotary_plan(bands, scaling=NAMES[scaling], factor=s, original_context=4096.0)
    f, ax = OR.frequencies(bands, scaling=scaling, factor=s, context=4096.0)
    p = np.array([0, 1, -1, (1 << 24) + 1, (1 << 31) + 5, (1 << 33) - 1, -(1 << 36) - 3, (1 << 40) + 7])
    pos = np.stack([np.roll(p, a) for a in range(len(bands))])[:, None]
    g = torch.Generator().manual_seed(dims)
    x = torch.randn((1, len(p), 2, D), generator=g).cuda()
    y = torch.empty_like(x)
    sab.rotary(plan, x, None, y, positions=torch.tensor(pos, device="cuda"))
    xd = x.double().cpu().numpy()
    ref = OR.rotate(xd, OR.angles(pos, f, ax), False)
    worse = 1 + s * 32 / 31 if scaling == "ramp" else 1.0
    fa = np.abs(pos[ax, 0].astype(float)).T * (f.astype(float) * worse * 2.0 ** -50 + 2 * np.pi * 2.0 ** -65)  # [L, pairs]
    pair = np.abs(xd[..., :dims:2]) + np.abs(xd[..., 1:dims:2])
    room = np.repeat((2.0 ** -21 + fa[None, :, None]) * pair, 2, axis=-1)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.array_equal(err[..., dims:], np.zeros_like(err[..., dims:]))
    assert np.all(err[..., :dims] <= room + 2.0 ** -24 * np.abs(ref[..., :dims]))
