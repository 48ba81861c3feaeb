"""Sizes that cross attention refuses before any CUDA call, through the C ABI, on
the CPU.  (Only refusals are called: the pointers are not memory.)"""

import ctypes

import pytest

import streaming_attention_block_gb300 as sab
from tests.test_gpu_cross import _desc, _rows

P = ctypes.c_void_p


def _status(d, ql, kl, back, scale=0.1):
    lib = sab.library()
    token = 64 * d.heads
    r = [_rows(4096 * (i + 1), token * max(d.q_tokens, d.kv_tokens), token) for i in range(8)]
    p = [ctypes.byref(x) for x in r]
    if back:
        return lib.sab_cross_attention_backward(ctypes.byref(d), *p[:5], P(4096), ql, kl, scale, *p[5:], P(1 << 20),
                                                1 << 60, None)
    return lib.sab_cross_attention(ctypes.byref(d), *p[:3], ql, kl, scale, p[3], P(4096), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [
    dict(batch=(1 << 26) + 1, kv_batch=1, q_tokens=1, heads=4, kv_heads=4, head_dim=64),  # four tiles a token
    dict(batch=(1 << 26) + 1, kv_batch=1, q_tokens=1, heads=4, kv_heads=1, head_dim=64),  # one
    dict(batch=1 << 20, kv_batch=1, q_tokens=129, heads=33, kv_heads=33, head_dim=64),
])
def test_more_query_tiles_of_unequal_sequences_than_are_cleared_in_time(back, kw):
    for ql, kl in ((P(4096), None), (None, P(4096)), (P(4096), P(8192))):
        assert _status(_desc(**kw), ql, kl, back) == 1


@pytest.mark.parametrize("back", [False, True])
def test_scales_that_are_infinite_to_base_2(back):
    """3e38 log2 e is no fp32 number, and 0 times it none at all."""
    for scale in (3.0e38, 2.4e38, float("inf")):
        assert _status(_desc(), None, None, back, scale) == 1
