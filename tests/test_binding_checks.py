"""Checks of tensor arguments in the Python binding, on the CPU: the binding is
told that CPU tensors live on its device, and the library's entry points are
replaced by a recorder, so that a call that passes every check is seen."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from streaming_attention_block_gb300 import _abi


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library; its sizes are as they are."""
    seen = []
    real = sab.library()

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_workspace") or name.endswith("plan_init"):
                return getattr(real, name)

            def call(*args):
                seen.append(name)
                return 0

            return call

    monkeypatch.setattr(_abi, "_device", lambda: -1)  # get_device() of a CPU tensor
    monkeypatch.setattr(_abi, "library", lambda: Recorder())
    return seen


def _rotate(bands, B, L, positions, fn=None):
    x = torch.zeros((B, L, 2, 64), dtype=torch.bfloat16)
    (fn or sab.rotary)(sab.rotary_plan(bands), x, None, torch.empty_like(x), positions=positions, stream=0)


@pytest.mark.parametrize("fn", ["rotary", "rotary_backward"])
def test_positions_in_another_order_are_refused(calls, fn):
    """[axes, B, L] ([B, L] for one axis) and nothing that holds as many numbers
    in another order, which would be read as other positions."""
    three, one = (24, 20, 20), (64,)
    fn = getattr(sab, fn)
    i64 = torch.int64
    for bands, B, L, shape in ((three, 2, 5, (2, 5, 3)), (three, 2, 5, (5, 2, 3)), (three, 2, 5, (3, 5, 2)),
                               (three, 2, 5, (30,)), (three, 2, 5, (3, 10)), (three, 1, 5, (5, 3)), (one, 2, 5, (5, 2)),
                               (one, 2, 5, (5, 2, 1)), (one, 2, 5, (10,)), (one, 4, 6, (8, 3)), (one, 1, 6, (2, 3))):
        with pytest.raises(ValueError, match="positions"):
            _rotate(bands, B, L, torch.zeros(shape, dtype=i64), fn)
    assert not calls
    # as documented, and the same with axes of length one added or left out
    good = ((three, 2, 5, (3, 2, 5)), (three, 1, 5, (3, 1, 5)), (three, 1, 5, (3, 5)), (three, 2, 1, (3, 2, 1)),
            (one, 2, 5, (2, 5)), (one, 2, 5, (1, 2, 5)), (one, 1, 5, (5,)), (one, 1, 5, (1, 5)), (one, 1, 1, (1,)),
            (one, 5, 1, (5, 1)))
    for bands, B, L, shape in good:
        _rotate(bands, B, L, torch.zeros(shape, dtype=i64), fn)
    assert len(calls) == len(good)


def test_positions_of_another_kind_are_refused(calls):
    for bad in (torch.zeros((2, 5), dtype=torch.int32), torch.zeros((2, 5)), torch.zeros((5, 2), dtype=torch.int64).t(),
                torch.zeros((2, 6), dtype=torch.int64)):
        with pytest.raises(ValueError, match="positions"):
            _rotate((64,), 2, 5, bad)
    with pytest.raises(TypeError, match="positions"):
        _rotate((64,), 2, 5, [[0] * 5] * 2)
    assert not calls
