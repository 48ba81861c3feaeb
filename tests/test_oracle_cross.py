"""Pins of the cross-attention oracle: torch in fp64, its gradients, closed
forms, and padding that is never read."""

import numpy as np
import pytest
import torch

from oracle import cross as OC


def _case(B, Lq, Lk, H, Hk, D, Bk=None, seed=0):
    r = np.random.default_rng(seed)
    return r.normal(size=(B, Lq, H, D)), r.normal(size=(Bk or B, Lk, Hk, D)), r.normal(size=(Bk or B, Lk, Hk, D)), \
        r.normal(size=(B, Lq, H, D))


@pytest.mark.parametrize("B, Lq, Lk, H, Hk, Bk", [(1, 3, 5, 1, 1, 1), (2, 4, 3, 4, 2, 2), (3, 2, 6, 3, 1, 1)])
def test_against_torch_and_its_gradients(B, Lq, Lk, H, Hk, Bk):
    q, k, v, do = _case(B, Lq, Lk, H, Hk, 8, Bk)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    wide = [x.expand(B, -1, -1, -1).repeat_interleave(H // Hk, 2).transpose(1, 2) for x in (tk, tv)]
    o = torch.nn.functional.scaled_dot_product_attention(tq.transpose(1, 2), *wide, scale=0.3).transpose(1, 2)
    o.backward(torch.tensor(do))
    O, lse, W, _ = OC.forward(q, k, v, 0.3)
    assert np.allclose(O, o.detach().numpy(), atol=1e-12) and np.all(W >= np.abs(O) - 1e-12)
    s = torch.einsum("blhd,bhkd->bhlk", tq, wide[0]) * 0.3
    assert np.allclose(lse, torch.logsumexp(s, -1).detach().numpy(), atol=1e-12)
    got, bound = OC.backward(q, k, v, do, 0.3)
    for g, b, t in zip(got, bound, (tq, tk, tv)):
        assert np.allclose(g, t.grad.numpy(), atol=1e-10) and np.all(b >= np.abs(g) - 1e-10)


def test_lengths_cut_and_padding_is_never_read():
    q, k, v, do = _case(3, 4, 5, 2, 1, 4)
    q_len, kv_len = [4, 2, 3], [5, 3, 0]
    for b in range(3):
        q[b, q_len[b]:] = np.nan
        do[b, q_len[b]:] = np.inf
        k[b, kv_len[b]:] = np.nan
        v[b, kv_len[b]:] = np.inf
    O, lse, _, _ = OC.forward(q, k, v, 0.5, q_len, kv_len)
    (dq, dk, dv), _ = OC.backward(q, k, v, do, 0.5, q_len, kv_len)
    for x in (O, dq, dk, dv):
        assert np.all(np.isfinite(x))
    assert np.all(O[1, 2:] == 0) and np.all(lse[1, :, 2:] == -np.inf) and np.all(O[2] == 0)
    assert np.all(dk[1, 3:] == 0) and np.all(dv[2] == 0) and np.all(dq[2] == 0)
    cut = OC.forward(q[1:2, :2], k[1:2, :3], v[1:2, :3], 0.5)
    assert np.allclose(O[1:2, :2], cut[0]) and np.allclose(lse[1:2, :, :2], cut[1])


def test_closed_forms():
    q, k, v, _ = _case(1, 2, 4, 1, 1, 4)
    O, lse, _, _ = OC.forward(0 * q, k, v, 1.0)
    assert np.allclose(O[0, 0, 0], v[0, :, 0].mean(0)) and np.allclose(lse, np.log(4.0))
    O, lse, _, _ = OC.forward(q, k[:, :1], v[:, :1], 1.0)
    assert np.allclose(O[0, :, 0], v[0, 0, 0]) and np.allclose(lse[0, 0], q[0, :, 0] @ k[0, 0, 0])


def test_differences():
    q, k, v, do = _case(2, 3, 4, 2, 1, 4, 1, seed=5)
    (dq, dk, dv), _ = OC.backward(q, k, v, do, 0.7, [3, 2], [4])
    r = np.random.default_rng(6)
    for name, x, g in (("q", q, dq), ("k", k, dk), ("v", v, dv)):
        step, h = r.normal(size=x.shape), 1e-6

        def loss(t):
            a = {"q": q, "k": k, "v": v, name: x + t * step}
            return np.sum(OC.forward(a["q"], a["k"], a["v"], 0.7, [3, 2], [4])[0] * do)

        assert abs((loss(h) - loss(-h)) / (2 * h) - np.sum(g * step)) < 1e-6, name
