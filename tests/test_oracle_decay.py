"""Pins of the decay-attention oracle: the masked quadratic form, closed forms,
feeding in pieces, autograd and differences for the gradients."""

import numpy as np
import pytest
import torch

from oracle import decay as OD


def _inputs(B, L, H, D, seed):
    rng = np.random.default_rng(seed)
    q, k, v, do = rng.standard_normal((4, B, L, H, D))
    S, dS = rng.standard_normal((2, B, H, D, D))
    return q, k, v, do, S, dS


def test_equals_the_masked_quadratic_form():
    q, k, v, _, S, _ = _inputs(2, 9, 3, 4, 1)
    ld = np.array([-0.3, -1e-3, 0.0])
    O, S1, _, _ = OD.decay_attention(q, k, v, ld, 0.5, S)
    i = np.arange(9)
    for h in range(3):
        M = np.where(i[:, None] >= i, np.exp(ld[h] * (i[:, None] - i)), 0.0)
        for b in range(2):
            o = 0.5 * (((q[b, :, h] @ k[b, :, h].T) * M) @ v[b, :, h] + np.exp(ld[h] * (i + 1))[:, None] *
                       (q[b, :, h] @ S[b, h]))
            assert np.allclose(O[b, :, h], o)
            w = np.exp(ld[h] * (8 - i))[:, None]
            assert np.allclose(S1[b, h], np.exp(9 * ld[h]) * S[b, h] + (k[b, :, h] * w).T @ v[b, :, h])


def test_full_decay_keeps_one_token_and_positive_counts_as_none():
    q, k, v, _, _, _ = _inputs(1, 5, 2, 3, 2)
    O, S, _, _ = OD.decay_attention(q, k, v, np.array([-np.inf, 2.0]), 1.0)
    assert np.allclose(O[0, :, 0], (q[0, :, 0] * k[0, :, 0]).sum(-1, keepdims=True) * v[0, :, 0])
    assert np.allclose(S[0, 1], k[0, :, 1].T @ v[0, :, 1])


def test_pieces_equal_the_whole_and_padding_is_inert():
    q, k, v, _, S, _ = _inputs(2, 11, 2, 4, 3)
    ld = np.array([-0.2, -0.01])
    O, S1, _, _ = OD.decay_attention(q, k, v, ld, 0.7, S)
    St, parts = S, []
    for a, b in ((0, 4), (4, 5), (5, 11)):
        o, St, _, _ = OD.decay_attention(q[:, a:b], k[:, a:b], v[:, a:b], ld, 0.7, St)
        parts.append(o)
    assert np.allclose(np.concatenate(parts, 1), O) and np.allclose(St, S1)
    q2, k2, v2 = (x.copy() for x in (q, k, v))
    for x in (q2, k2, v2):
        x[1, 6:] = np.nan
    O2, S2, _, _ = OD.decay_attention(q2, k2, v2, ld, 0.7, S, lens=[11, 6])
    assert np.allclose(O2[0], O[0]) and np.allclose(O2[1, :6], O[1, :6]) and np.all(O2[1, 6:] == 0)
    O3, S3, _, _ = OD.decay_attention(q[:, :6], k[:, :6], v[:, :6], ld, 0.7, S)
    assert np.allclose(S2[1], S3[1])
    _, S0, _, _ = OD.decay_attention(q, k, v, ld, 0.7, S, lens=[0, -3])
    assert np.array_equal(S0, S)


def test_gradients_equal_autograd():
    q, k, v, do, S, dS = _inputs(2, 8, 2, 3, 4)
    ld = np.array([-0.4, 0.0])
    lens = [8, 5]
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, S)]
    tq, tk, tv, tS = t
    loss = 0.0
    for b in range(2):
        s = tS[b]
        for i in range(lens[b]):
            s = s * torch.exp(torch.tensor(ld))[:, None, None] + tk[b, i, :, :, None] * tv[b, i, :, None, :]
            loss = loss + (0.6 * torch.einsum("hd,hde->he", tq[b, i], s) * torch.tensor(do[b, i])).sum()
        loss = loss + (s * torch.tensor(dS[b])).sum()
    loss.backward()
    grads, bounds = OD.decay_attention_backward(q, k, v, do, ld, 0.6, S, dS, lens)
    for got, want, bnd in zip(grads, t, bounds):
        assert np.allclose(got, want.grad.numpy())
        assert np.all(np.abs(got) <= bnd + 1e-12)


@pytest.mark.parametrize("which", range(4))
def test_gradients_equal_differences(which):
    q, k, v, do, S, dS = _inputs(1, 6, 1, 3, 5)
    ld = np.array([-0.25])
    args = [q, k, v, S]

    def loss(a):
        O, S1, _, _ = OD.decay_attention(a[0], a[1], a[2], ld, 0.9, a[3])
        return (O * do).sum() + (S1 * dS).sum()

    g = OD.decay_attention_backward(q, k, v, do, ld, 0.9, S, dS)[0][which]
    rng = np.random.default_rng(6)
    for _ in range(5):
        e = np.zeros_like(args[which])
        e[tuple(rng.integers(0, n) for n in e.shape)] = 1e-5
        lo, hi = ([x - e if i == which else x for i, x in enumerate(args)],
                  [x + e if i == which else x for i, x in enumerate(args)])
        assert abs((loss(hi) - loss(lo)) / 2e-5 - g[e != 0].sum()) < 1e-6
