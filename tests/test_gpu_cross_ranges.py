"""Cross attention on the GPU with values and scores far from 1.

Tolerances are those of the tests of the two directions, and for values near the
least of the type: products below 2^-126 keep multiples of 2^-149, half a step of
which is 2^-150 a key, and a sum of 2^-24 or more divides them.  So O is off by
at most Lk 2^-126 more."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import cross as OC
from tests.test_gpu_cross import BF, _np

gpu = pytest.mark.gpu


def _level(B, Lq, Lk, H, D, score, exponent, seed=0):
    """Every score is `score`; values between 2^(exponent - 1) and 2^exponent."""
    g = torch.Generator().manual_seed(seed)
    q = torch.ones((B, Lq, H, D)).bfloat16().cuda()
    k = torch.full((B, Lk, H, D), 1.0 if score >= 0 else -1.0).bfloat16().cuda()
    v = ((torch.rand((B, Lk, H, D), generator=g) + 1.0) * 2.0 ** (exponent - 1)).bfloat16().cuda()
    return q, k, v, max(abs(score), 2.0 ** -20) / D


@gpu
@pytest.mark.parametrize("B, Lq, Lk, H, D", [(64, 300, 16, 4, 64), (3, 300, 200, 2, 128), (1, 4, 1300, 1, 64)])
@pytest.mark.parametrize("score", [-60.0, -50.0, -30.0, -17.0, -10.0, 0.0, 40.0, 60.0])
def test_small_and_large_values_under_scores_of_all_sizes(B, Lq, Lk, H, D, score):
    """A row's weights are 1 / Lk each, whatever its scores are: O is the mean of the values."""
    for exponent in (-110, -100, -80, -60, 0, 60, 100):
        q, k, v, scale = _level(B, Lq, Lk, H, D, score, exponent)
        o = torch.full_like(q, float("nan"))
        sab.cross_attention(q, k, v, scale, o)
        ref = v[:1].double().mean(1, keepdim=True) if B == 1 else v.double().mean(1, keepdim=True)
        es = D * 2.0 ** -23 * abs(score) + 2.0 ** -20
        tol = (2 * BF + 2 * es + 2.0 ** -16) * ref + Lk * 2.0 ** -126
        err = (o.double() - ref).abs()
        assert bool((err <= tol).all()), (exponent, (err / ref).max().item())
    assert sab.get_last_device_error() == 0


@gpu
@pytest.mark.parametrize("Lk, lens", [(40, None), (300, None), (300, [300, 20])])
def test_a_row_whose_scores_all_overflow_below_has_no_say(Lk, lens):
    """Its scores are -inf: O is 0, LSE -inf as without keys, its dQ 0, and the other
    rows' gradients are those of a call with that row's dO at 0."""
    B, Lq, H, D = 2, 200, 2, 64
    g = torch.Generator().manual_seed(4)
    q, do = (torch.randn((B, Lq, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    k = ((torch.rand((B, Lk, H, D), generator=g) + 0.5) * 8.0).bfloat16().cuda()
    v = torch.randn((B, Lk, H, D), generator=g).bfloat16().cuda()
    scale, kl = 0.05, None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call():
        o, lse = torch.empty_like(q), torch.empty((B, H, Lq), device="cuda")
        sab.cross_attention(q, k, v, scale, o, lse, kv_len=kl)
        grads = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        sab.cross_attention_backward(q, k, v, o, do, lse, scale, *grads, kv_len=kl)
        torch.cuda.synchronize()
        return o, lse, grads

    q[0, 5], q[1, 130, 1] = -2.0 ** 127, -2.0 ** 127
    o, lse, grads = call()
    assert bool((o[0, 5] == 0).all()) and bool((lse[0, :, 5] == -float("inf")).all())
    assert bool((o[1, 130, 1] == 0).all()) and bool(torch.isfinite(lse[1, 0, 130]))
    assert bool((grads[0][0, 5] == 0).all()) and bool((grads[0][1, 130, 1] == 0).all())
    q[0, 5], q[1, 130, 1], do[0, 5], do[1, 130, 1] = 0.0, 0.0, 0.0, 0.0
    ref, bound = OC.backward(_np(q), _np(k), _np(v), _np(do), scale, None, lens)
    for x, r, b in zip(grads, ref, bound):  # 2^127 dS of those rows is 0 too
        assert bool((abs(_np(x) - r) <= (2 * BF + BF / 2) * b + BF * abs(r) + 1e-30).all())
