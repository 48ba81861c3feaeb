"""Layer norm and its gradients over tensors of more than 2^31 elements: the last
rows against the fp64 oracle, the sums that only they feed, and rows in between.
Bounds are those of ``tests/test_gpu_layer_norm.py``."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests.test_gpu_layer_norm import EPS, _check_backward, _check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C, group", [(8192, None), (8191, None), (8192, 4096)])
def test_last_rows_and_the_sums_they_feed(C, group):
    rows, far = (1 << 31) // C + 100, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    x, y, dy, dx = (torch.empty((rows, C), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    x.fill_(1.0)
    x[-far:].normal_(generator=g)
    dy.zero_()
    dy[-far:].normal_(generator=g)
    y.fill_(float("nan"))
    dx.fill_(float("nan"))
    groups = 1 if group is None else -(-rows // group)
    first = 0 if group is None else (groups - 1) * group  # of the last group, which holds the far rows
    assert rows - far >= first
    w, b = (torch.randn((groups, C), generator=g, device="cuda") for _ in range(2))
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    dw, db = (torch.full((groups, C), float("nan"), device="cuda") for _ in range(2))
    sab.layer_norm(x, w, b, EPS, y, mean, rstd, group_rows=group)
    sab.layer_norm_backward(x, dy, w, mean, rstd, dx, dw, db, group_rows=group)
    tail = slice(rows - far, rows)
    _check_forward(x[tail], w[-1:], b[-1:], y[tail], mean[tail], rstd[tail], far, 0.0, "far rows")
    # a row of ones is its mean: y is the bias, dx of dy = 0 is 0
    for i in (0, 1, (rows - far) // 2, rows - far - 1):
        assert torch.equal(y[i], b[0 if group is None else i // group].bfloat16())
    assert bool((mean[:-far] == 1.0).all()) and not bool(dx[:-far].any())
    # what the other rows add to the sums is 0
    _check_backward(x[tail], dy[tail], w[-1:], mean[tail], rstd[tail], dx[tail], dw[-1:], db[-1:], far, 0.0, "far rows")
    assert not bool(dw[:-1].any()) and not bool(db[:-1].any())
    assert sab.get_last_device_error() == 0
