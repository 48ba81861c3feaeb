"""Pins of the layer-norm oracle: closed forms, torch in fp64, differences."""

import numpy as np
import pytest
import torch

from oracle import layer_norm as ON


def _case(rows, C, group_rows, seed=0):
    r = np.random.default_rng(seed)
    groups = -(-rows // group_rows)
    return r.normal(size=(rows, C)) * 2 + 0.5, r.normal(size=(groups, C)), r.normal(size=(groups, C)), \
        r.normal(size=(rows, C))


@pytest.mark.parametrize("rows, C, group_rows, offset", [(5, 7, 5, 0.0), (6, 4, 2, 1.0), (7, 9, 3, 0.5), (3, 1, 1, 0.0)])
def test_against_torch_and_its_gradients(rows, C, group_rows, offset):
    x, w, b, dy = _case(rows, C, group_rows)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    n = torch.nn.functional.layer_norm(tx, (C,), eps=1e-5)
    at = torch.arange(rows) // group_rows
    (n * (offset + tw[at]) + tb[at]).backward(torch.tensor(dy))
    y, mean, rstd = ON.forward(x, w, b, 1e-5, group_rows, offset)
    assert np.allclose(y, (n * (offset + tw[at]) + tb[at]).detach().numpy(), atol=1e-12)
    got, scale = ON.backward(x, dy, w, mean, rstd, group_rows, offset)
    for g, s, ref in zip(got, scale, (tx.grad, tw.grad, tb.grad)):
        assert np.allclose(g, ref.numpy(), atol=1e-9 * max(1.0, rstd.max()))
        assert np.all(s >= np.abs(g) - 1e-9)


def test_by_hand_and_without_weights():
    y, mean, rstd = ON.forward([[1.0, 3.0]], None, None, 0.0, 1)
    assert np.allclose(y, [[-1.0, 1.0]]) and mean[0] == 2.0 and rstd[0] == 1.0
    y, _, _ = ON.forward([[1.0, 3.0]], [[2.0, 4.0]], [[10.0, 20.0]], 0.0, 1, offset=1.0)
    assert np.allclose(y, [[7.0, 25.0]])
    assert np.all(ON.forward(np.full((2, 8), 4.0), None, None, 1e-6, 2)[0] == 0.0)


def test_differences():
    x, w, b, dy = _case(4, 6, 2, 3)
    _, mean, rstd = ON.forward(x, w, b, 1e-6, 2, 1.0)
    (dx, dw, db), _ = ON.backward(x, dy, w, mean, rstd, 2, 1.0)
    r = np.random.default_rng(4)
    for name, v, g in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        step = r.normal(size=v.shape)
        h = 1e-6

        def loss(t):
            a = {"x": x, "w": w, "b": b, name: v + t * step}
            return np.sum(ON.forward(a["x"], a["w"], a["b"], 1e-6, 2, 1.0)[0] * dy)

        assert abs((loss(h) - loss(-h)) / (2 * h) - np.sum(g * step)) < 1e-6, name
