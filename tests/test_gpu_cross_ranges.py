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
