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


def _forms():
    """(call, its arguments, those that may be left out) of the decay entry points."""
    B, L, H, D = 2, 300, 3, 64
    bf, f4, i4 = torch.bfloat16, torch.float32, torch.int32
    x, st = (B, L, H, D), (B, H, D, D)

    def args(shape, *rows):
        a = {n: torch.zeros(shape, dtype=bf) for n in rows}
        a["log_decay"] = torch.zeros(H, dtype=f4)
        return a

    states = {"state_in": torch.zeros(st, dtype=f4)}
    fwd = dict(args(x, "Q", "K", "V", "O"), **states, state_out=torch.zeros(st, dtype=f4),
               seq_len=torch.zeros(B, dtype=i4))
    step = dict(args((B, H, D), "Q", "K", "V", "O"), **states, state_out=torch.zeros(st, dtype=f4),
                active=torch.zeros(B, dtype=i4))
    bwd = dict(args(x, "Q", "K", "V", "dO", "dQ", "dK", "dV"), **states, d_state_out=torch.zeros(st, dtype=f4),
               d_state_in=torch.zeros(st, dtype=f4), seq_len=torch.zeros(B, dtype=i4))
    return {"decay_attention": fwd, "decay_attention_step": step, "decay_attention_backward": bwd}


def _wrong(t):
    """The tensor with another type, with another length, and strided."""
    other = {torch.bfloat16: torch.float16, torch.float32: torch.float64, torch.int32: torch.int64}[t.dtype]
    return [("type", t.to(other)), ("shape", torch.zeros((*t.shape[:-1], t.shape[-1] + 4), dtype=t.dtype, device=t.device)),
            ("contiguous", torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=t.device)[..., ::2]),
            ("tensor", [0])]


@pytest.mark.parametrize("fn", list(_forms()))
def test_each_tensor_of_a_decay_call_is_checked(calls, fn):
    """One wrong tensor at a time is refused by its name; nothing is launched."""
    good = _forms()[fn]

    def call(**kw):
        if fn != "decay_attention_step":
            kw["workspace"] = torch.empty(1 << 24, dtype=torch.uint8)
        getattr(sab, fn)(**kw)

    call(scale=0.1, stream=0, **good)
    assert calls == ["sab_" + fn]
    for name, t in good.items():
        for what, bad in _wrong(t):
            if name == "Q" and what in ("shape", "tensor"):
                continue  # Q's shape is the call's
            with pytest.raises((TypeError, ValueError), match=f"^{name}: "):
                call(scale=0.1, stream=0, **dict(good, **{name: bad}))
    with pytest.raises(ValueError, match="^[KVOd]"):  # another shape of Q: the others disagree
        q = good["Q"]
        call(scale=0.1, stream=0, **dict(good, Q=torch.zeros((*q.shape[:-2], q.shape[-2] + 1, q.shape[-1]), dtype=q.dtype)))
    assert len(calls) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("fn", list(_forms()))
def test_each_tensor_of_a_decay_call_is_checked_on_the_gpu(fn):
    good = {n: t.cuda() for n, t in _forms()[fn].items()}
    call = getattr(sab, fn)
    reason = {"type": "expected torch", "shape": "expected shape", "contiguous": "must be contiguous",
              "tensor": "expected a torch tensor"}
    for name, t in good.items():
        for what, bad in _wrong(t) + [("device", t.cpu())]:
            if name == "Q" and what in ("shape", "tensor"):
                continue
            say = reason.get(what, "must be a CUDA tensor")
            with pytest.raises((TypeError, ValueError), match=f"^{name}: {say}"):
                call(scale=0.1, **dict(good, **{name: bad}))
    torch.cuda.synchronize()
    assert not any(bool(t.any()) for t in good.values())
    call(scale=0.1, **good)
    torch.cuda.synchronize()
