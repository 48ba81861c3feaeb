"""Rotary positions in front of block-causal attention, and both gradients, as
a training step uses them, against the fp64 composition."""

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import attention as OA
from oracle import backward as OB
from oracle import rotary as OR

pytestmark = pytest.mark.gpu


def _n(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("D", [64, 128])
def test_rotary_then_block_causal_training(D, half):
    B, L, H, Lc, W = 2, 500, 2, 100, 2
    scale = D ** -0.5
    bands = (D // 2,) if half else (D - 4 * (D // 6), D // 6 * 2, D // 6 * 2)
    plan = sab.rotary_plan(bands, layout=sab.ROTARY_HALF if half else sab.ROTARY_INTERLEAVED)
    f, ax = OR.frequencies(bands)
    t = np.arange(L)
    pos = np.stack([t // 100, t // 10 % 10, t % 10] if not half else [t + 4096])[:, None].repeat(B, 1)
    dpos, ang = torch.tensor(pos, device="cuda"), OR.angles(pos, f, ax)
    g = torch.Generator().manual_seed(D)
    q, k, v, do = (torch.randn((B, L, H, D), generator=g).bfloat16().cuda() for _ in range(4))
    qr, kr, O, dqr, dkr, dv, dq, dk = (torch.empty_like(q) for _ in range(8))
    LSE = torch.empty((B, H, L), device="cuda")
    sab.rotary(plan, q, k, qr, kr, positions=dpos)
    sab.block_causal_attention(qr, kr, v, Lc, W, 1, scale, O, LSE)
    sab.block_causal_attention_backward(qr, kr, v, O, do, LSE, Lc, W, scale, dqr, dkr, dv)
    sab.rotary_backward(plan, dqr, dkr, dq, dk, positions=dpos)
    qn, kn = OR.rotate(_n(q), ang, half), OR.rotate(_n(k), ang, half)
    o = np.transpose(OA.block_causal_attention(qn, kn, _n(v), Lc, W, scale)[0], (0, 2, 1, 3))
    gq, gk, gv = OB.block_causal_attention_backward(qn, kn, _n(v), _n(do), Lc, W, scale)
    want = [o, OR.rotate(gq, ang, half, backward=True), OR.rotate(gk, ang, half, backward=True), gv]
    # independent roundings to bf16 in a row, each 2^-8 / sqrt(3) of the norm at
    # most.  O: q', k' (a score of unit variance moves by as much), P, O.  The
    # gradients: q', k' in the scores and k' or q' again in the product, P, dS,
    # O in delta, two stored results
    for name, got, ref, n in zip(("O", "dQ", "dK", "dV"), (O, dq, dk, dv), want, (4, 8, 8, 8)):
        err = np.linalg.norm(_n(got) - ref) / np.linalg.norm(ref)
        assert err <= np.sqrt(n / 3) * 2.0 ** -8, (name, err)
