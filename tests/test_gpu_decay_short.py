"""Decay attention on both sides of the lengths at which it changes from single
tokens to tiles, for few heads, for a block per SM and for several waves,
against the fp64 recurrence (bounds: tests/test_gpu_decay.py)."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests.test_gpu_decay import _check, _fp64_back_on_gpu, _fp64_on_gpu, _n, _out, _randn, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H", [(2, 3), (8, 6), (10, 8), (25, 8)])
@pytest.mark.parametrize("L", [1, 2, 3, 4, 5, 8, 9, 12, 13, 16, 17, 40, 41])
def test_lengths_around_the_change(B, H, D, L):
    scale = D ** -0.5
    q, k, v, do = (_randn((B, L, H, D), 500 + L + i) for i in range(4))
    ld = torch.tensor([-0.3, -0.02, 0.0, -1e-3, -4.0, -0.7, -1e-5, -0.1][:H], device="cuda")
    S, dS = (_randn((B, H, D, D), 510 + i, torch.float32) for i in range(2))
    zero = torch.zeros_like(S)
    for s_in, d_out in ((S, dS), (None, None)):
        a, r = (x.double() for x in ((S, dS) if s_in is not None else (zero, zero)))
        o, s, oa, sa = _fp64_on_gpu(q, k, v, ld, scale, a)
        refs, bnds = _fp64_back_on_gpu(q, k, v, do, ld, scale, a, r)
        O, g = _out(q.shape), [_out(q.shape) for _ in range(3)]
        So, d_in = ((_out(S.shape, torch.float32), _out(S.shape, torch.float32)) if s_in is not None else (None, None))
        sab.decay_attention(q, k, v, ld, scale, O, state_in=s_in, state_out=So,
                            workspace=_ws(sab.decay_attention_workspace(B, L, H, D)))
        sab.decay_attention_backward(q, k, v, do, ld, scale, *g, state_in=s_in, d_state_out=d_out, d_state_in=d_in,
                                     workspace=_ws(sab.decay_attention_backward_workspace(B, L, H, D)))
        _check(O, _n(o), _n(oa), "O")
        for name, got, ref, bnd in zip(("dQ", "dK", "dV"), g, refs, bnds):
            _check(got, _n(ref), _n(bnd), name)
        if s_in is not None:
            _check(So, _n(s), _n(sa), "state", state=True)
            _check(d_in, _n(refs[3]), _n(bnds[3]), "d_state_in", state=True)
