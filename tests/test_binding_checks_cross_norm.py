"""Checks of tensor arguments in the Python binding of cross attention and layer
norm, on the CPU: the binding is told that CPU tensors live on its device, and the
library's entry points are replaced by a recorder."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests.test_binding_checks import calls  # noqa: F401  (a fixture)

BF, F4, I4 = torch.bfloat16, torch.float32, torch.int32


def _forms():
    """(call, its tensors) of the entry points, with every optional tensor."""
    B, Lq, Lk, H, Hk, D = 2, 5, 7, 4, 2, 64
    q, k, rows = (B, Lq, H, D), (B, Lk, Hk, D), 6

    def z(shape, dtype=BF):
        return torch.zeros(shape, dtype=dtype)

    cross = dict(Q=z(q), K=z(k), V=z(k), O=z(q), LSE=z((B, H, Lq), F4), q_len=z(B, I4), kv_len=z(B, I4))
    grads = dict(cross, dO=z(q), dQ=z(q), dK=z(k), dV=z(k))
    norm = dict(X=z((rows, 32)), weight=z((3, 32), F4), bias=z((3, 32), F4), Y=z((rows, 32)), mean=z(rows, F4),
                rstd=z(rows, F4))
    back = dict(X=z((rows, 32)), dY=z((rows, 32)), weight=z((3, 32), F4), mean=z(rows, F4), rstd=z(rows, F4),
                dX=z((rows, 32)), dweight=z((3, 32), F4), dbias=z((3, 32), F4))
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    return {"cross_attention": (cross, dict(softmax_scale=0.1)),
            "cross_attention_backward": (grads, dict(softmax_scale=0.1, workspace=ws)),
            "layer_norm": (norm, dict(eps=1e-6, group_rows=2)),
            "layer_norm_backward": (back, dict(group_rows=2, workspace=ws))}


def _wrong(t):
    """The tensor with another type, another shape, not contiguous, none at all."""
    other = {BF: torch.float16, F4: torch.float64, I4: torch.int64}[t.dtype]
    return [t.to(other), torch.zeros((*t.shape[:-1], t.shape[-1] + 8), dtype=t.dtype),
            torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2], [0]]


@pytest.mark.parametrize("fn", list(_forms()))
def test_each_tensor_of_a_call_is_checked(calls, fn):  # noqa: F811
    """One wrong tensor at a time is refused by its name; nothing is launched."""
    good, rest = _forms()[fn]
    call = getattr(sab, fn)
    call(stream=0, **good, **rest)
    assert calls == ["sab_" + fn]
    for name, t in good.items():
        for i, bad in enumerate(_wrong(t)):
            if i == 1 and name in ("Q", "K", "X"):
                continue  # these are the call's shapes
            with pytest.raises((TypeError, ValueError), match=f"^{name}: "):
                call(stream=0, **dict(good, **{name: bad}), **rest)
    assert len(calls) == 1


def test_shapes_that_disagree(calls):  # noqa: F811
    good, rest = _forms()["cross_attention"]
    for bad in (dict(Q=good["Q"][:, :4]), dict(K=good["K"][:, :6]), dict(K=torch.zeros((2, 7, 2, 128), dtype=BF))):
        with pytest.raises(ValueError):
            sab.cross_attention(stream=0, **dict(good, **bad), **rest)
    same = good["O"][:, :, :1].expand(-1, -1, 4, -1)  # heads on top of each other
    for name in ("Q", "O"):
        with pytest.raises(ValueError, match=f"^{name}: "):
            sab.cross_attention(stream=0, **dict(good, **{name: same}), **rest)
    good, rest = _forms()["layer_norm"]
    for bad in (dict(weight=good["weight"][:2]), dict(bias=good["bias"].view(-1)), dict(mean=good["mean"][:5])):
        with pytest.raises(ValueError):
            sab.layer_norm(stream=0, **dict(good, **bad), **rest)
    assert not calls
