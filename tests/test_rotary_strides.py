"""Strides whose products pass 64 bits are refused by the rotary entry points
before any CUDA call (host only)."""

import ctypes

import pytest

import streaming_attention_block_gb300 as sab


@pytest.mark.parametrize("fn", ["sab_rotary", "sab_rotary_backward"])
@pytest.mark.parametrize("B,L,strides", [
    (2, 1 << 30, (128, 128, 128, 1 << 40)),   # 2^70 - 2^40 elements, -2^40 in 64 bits
    (2, 1 << 30, (128, 1 << 40, 1 << 40, 128)),
    (1 << 24, 1, (1 << 40, 128, 1 << 40, 128)),
    (1, 1 << 24, (128, 1 << 40, 128, 128)),
    (1, 1 << 24, (128, 128, 128, 1 << 40)),
])
def test_extents_beyond_any_memory_are_refused(fn, B, L, strides):
    plan = sab.rotary_plan((64,))
    rows = sab._abi.RotaryRows(4096, 8192, 2, *strides)
    call = getattr(sab.library(), fn)
    for q, k in ((rows, None), (sab._abi.RotaryRows(1 << 20, 1 << 21, 2, 1 << 37, 128, 1 << 37, 128), rows)):
        got = call(ctypes.byref(plan), ctypes.byref(q), ctypes.byref(k) if k else None, None, 0, B, L, 64, 0, None)
        assert got == 1, got
