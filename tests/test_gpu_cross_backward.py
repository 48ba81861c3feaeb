"""Gradients of cross attention on the GPU against the fp64 oracle
(``oracle/cross.py``), through the C ABI.

Bound per element, derived from the arithmetic.  P and dS are rounded to bf16
before their products (2^-8 each); P is recomputed from LSE with the forward's
score error e_s (below 2^-10 at these sizes); delta comes from the bf16 output
(2^-8 of sum |dO| |O|, inside the error scale, which holds |dP| + |delta| for
dS); sums are fp32.  So each gradient is off by at most (2 * 2^-8 + 2^-9) of
the sum of its absolute terms, and one rounding of its own."""

import ctypes

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import cross as OC
from tests.test_gpu_cross import BF, RAGGED, ROW_REFUSALS, SHAPE_REFUSALS, SHAPES, _case, _desc, _heads_first, _lens, _np, \
    _rows, _spoil

gpu = pytest.mark.gpu


def _forward(q, k, v, scale, q_len, kv_len):
    o = torch.empty_like(q)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), device="cuda")
    sab.cross_attention(q, k, v, scale, o, lse, q_len=q_len, kv_len=kv_len)
    return o, lse


def _backward(q, k, v, do, scale, q_len=None, kv_len=None, **kw):
    ql, kl = _lens(q_len), _lens(kv_len)
    o, lse = _forward(q, k, v, scale, ql, kl)
    _spoil(o, q_len, float("nan"))
    grads = [torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    sab.cross_attention_backward(q, k, v, o, do, lse, scale, *grads, q_len=ql, kv_len=kl, **kw)
    torch.cuda.synchronize()
    assert sab.get_last_device_error() == 0
    return grads


def _check(q, k, v, do, scale, grads, q_len, kv_len, what):
    ref, bound = OC.backward(_np(q), _np(k), _np(v), _np(do), scale, q_len, kv_len)
    for name, g, r, b in zip(("dQ", "dK", "dV"), grads, ref, bound):
        tol = (2 * BF + BF / 2) * b + BF * np.abs(r) + 1e-30
        err = np.abs(_np(g) - r)
        assert np.all(err <= tol), f"{what}: {name} off by {np.max(err - tol):.3e} at {np.argwhere(~(err <= tol))[:3]}"


@gpu
@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D, Bk", SHAPES)
def test_shapes(B, Lq, Lk, H, Hk, D, Bk):
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D, Bk, fused=Lk % 2 == 1)
    _check(q, k, v, do, D ** -0.5, _backward(q, k, v, do, D ** -0.5), None, None, f"{B} {Lq} {Lk} {H}/{Hk} {D}")


@gpu
@pytest.mark.parametrize("Lq, Lk, H, Hk, D, q_len, kv_len", RAGGED)
@pytest.mark.parametrize("junk", [0.0, float("nan"), float("inf")])
def test_lengths_and_what_lies_past_them(Lq, Lk, H, Hk, D, q_len, kv_len, junk):
    B = len(q_len or kv_len)
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D, fused=Hk == 2)
    for t, n in ((q, q_len), (do, q_len), (k, kv_len), (v, kv_len)):
        _spoil(t, n, junk)
    grads = _backward(q, k, v, do, D ** -0.5, q_len, kv_len)
    for t in (q, k, v, do):  # the oracle may not read it either
        t.nan_to_num_(0.0, 0.0, 0.0)
    _check(q, k, v, do, D ** -0.5, grads, q_len, kv_len, "ragged")


@gpu
@pytest.mark.parametrize("Lq, H, Hk, D", [(1, 24, 8, 128), (3, 6, 6, 64), (129, 4, 4, 64)])
def test_many_sequences_of_unequal_lengths(Lq, H, Hk, D):
    B, Lk = 64, 400
    lens = [(97 * b) % (Lk + 1) for b in range(B)]
    lens[5] = lens[40] = 0
    lens[7], lens[8], lens[9], lens[10] = 128, 129, 1, 64
    q_len = [(5 * b) % (Lq + 1) for b in range(B)]
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D)
    _check(q, k, v, do, D ** -0.5, _backward(q, k, v, do, D ** -0.5, q_len, lens), q_len, lens, "many")


@gpu
@pytest.mark.parametrize("H, Hk", [(4, 4), (6, 2), (10, 1)])
def test_states_that_all_sequences_share(H, Hk):
    """Heads and sequences summed into one gradient; most queries padding."""
    q, k, v, do = _case(9, 150, 300, H, Hk, 64, 1)
    q_len = [150, 0, 3, 1, 64, 65, 0, 149, 0]
    _check(q, k, v, do, 0.125, _backward(q, k, v, do, 0.125, q_len, [260]), q_len, [260], "shared")
    _check(q, k, v, do, 0.125, _backward(q, k, v, do, 0.125, [0] * 9, [260]), [0] * 9, [260], "no query")
    _check(q, k, v, do, 0.125, _backward(q, k, v, do, 0.125, None, [0]), None, [0], "no key")


@gpu
def test_long_queries_in_shares_and_equal_bits():
    q, k, v, do = _case(1, 9000, 130, 3, 3, 128)
    first = _backward(q, k, v, do, 0.08)
    _check(q, k, v, do, 0.08, first, None, None, "long")
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, _backward(q, k, v, do, 0.08)))


@gpu
@pytest.mark.parametrize("q_scale", [0.0, 20.0])
def test_sharp_and_flat_rows(q_scale):
    q, k, v, do = _case(1, 200, 300, 2, 2, 64, q_scale=q_scale)
    _check(q, k, v, do, 0.125, _backward(q, k, v, do, 0.125), None, None, "sharp")


@gpu
def test_directional_derivatives():
    """Against differences of the fp64 oracle's loss along random directions."""
    q, k, v, do = _case(2, 70, 90, 4, 2, 64, 1)
    grads = _backward(q, k, v, do, 0.125, [70, 40], [77])
    r = np.random.default_rng(0)
    x = [_np(t) for t in (q, k, v)]
    bound = OC.backward(*x, _np(do), 0.125, [70, 40], [77])[1]
    for i in range(3):
        step, h = r.normal(size=x[i].shape), 1e-5

        def loss(t):
            y = list(x)
            y[i] = x[i] + t * step
            return np.sum(OC.forward(*y, 0.125, [70, 40], [77])[0] * _np(do))

        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - np.sum(_np(grads[i]) * step)) <= 3.5 * BF * np.sum(bound[i] * np.abs(step)) + 1e-4


@gpu
def test_strides_and_what_lies_between():
    B, Lq, Lk, H, Hk, D = 2, 200, 150, 4, 2, 128
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D)
    ref = _backward(q, k, v, do, 0.1)
    o, lse = _forward(q, k, v, 0.1, None, None)
    wide = torch.full((B, Lq + 3, 3, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, t in enumerate((q, do, o)):
        wide[:, :Lq, i] = t
    kv = torch.stack([k, v], 2)
    dkv = torch.full((Lk + 2, B, 2, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")  # tokens outermost
    dq = torch.full((B, Lq + 2, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qs, ds, os_ = (wide[:, :Lq, i] for i in range(3))
    out = [dq[:, 1:Lq + 1, 1:], dkv[:Lk, :, 0].transpose(0, 1), dkv[:Lk, :, 1].transpose(0, 1)]
    sab.cross_attention_backward(qs, kv[:, :, 0], kv[:, :, 1], os_, ds, lse, 0.1, *out)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    dq[:, 1:Lq + 1, 1:] = 7.0
    assert bool((dq == 7).all()) and bool((dkv[Lk:] == 7).all())


@gpu
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [(2, 200, 150, 4, 2, 128), (3, 65, 300, 6, 2, 64), (1, 900, 77, 4, 4, 128)])
def test_heads_before_tokens(B, Lq, Lk, H, Hk, D):
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D)
    for lens in (None, [Lk] * (B - 1) + [0]):
        ref = _backward(q, k, v, do, 0.1, None, lens)
        o, lse = _forward(q, k, v, 0.1, None, _lens(lens))
        out = [_heads_first(t, 7.0) for t in (q, k, v)]
        sab.cross_attention_backward(*(_heads_first(t) for t in (q, k, v, o, do)), lse, 0.1, *out, kv_len=_lens(lens))
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@gpu
def test_other_stream_and_graph_beside_autograd():
    """A captured call while an eager graph of the same leaves lives."""
    q, k, v, do = _case(2, 600, 200, 6, 3, 64)
    ref = _backward(q, k, v, do, 0.125)
    o, lse = _forward(q, k, v, 0.125, None, None)
    ws = torch.empty(sab.cross_attention_backward_workspace(2, 600, 200, 6, 3, 64), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in ref]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sab.cross_attention_backward(q, k, v, o, do, lse, 0.125, *out, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    leaf = q.float().requires_grad_()
    alive = (leaf * 2).sum()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sab.cross_attention_backward(q, k, v, o, do, lse, 0.125, *out, workspace=ws)
    for _ in range(2):
        for t in out:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    alive.backward()
    assert bool((leaf.grad == 2).all())


def test_refusals_before_any_cuda_call():
    lib = sab.library()
    names = ("q", "k", "v", "o", "do", "dq", "dk", "dv")
    P = ctypes.c_void_p

    def call(d=_desc(), lse=P(4096), ql=None, kl=None, scale=0.1, ws=P(1 << 20), n=1 << 40, **kw):
        r = [kw.get(x) if kw.get(x) is not None else _rows(4096 * (i + 1)) for i, x in enumerate(names)]
        p = [ctypes.byref(x) if x != 0 else None for x in r]
        return lib.sab_cross_attention_backward(ctypes.byref(d) if d else None, *p[:5], lse, ql, kl, scale, *p[5:], ws,
                                                n, None)

    assert call(d=None) == 1
    for kw in SHAPE_REFUSALS:
        assert call(d=_desc(**kw)) == 1, kw
    for name in names:
        assert call(**{name: 0}) == 1
        for kw in ROW_REFUSALS:
            assert call(**{name: _rows(**kw)}) == 1, (name, kw)
    for i, name in enumerate(names[5:]):
        for j in range(8):
            if j != 5 + i:
                assert call(**{name: _rows(4096 * (j + 1))}) == 1, (name, j)
    for kw in (dict(lse=None), dict(lse=P(4104)), dict(ql=P(4098)), dict(kl=P(4097)), dict(scale=0.0),
               dict(scale=float("nan"))):
        assert call(**kw) == 1, kw
    need = sab.cross_attention_backward_workspace(2, 4, 8, 4, 2, 64)
    assert need > 0 and sab.cross_attention_backward_workspace(2, 4, 8, 4, 3, 64) == 0
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=P((1 << 20) + 16))):
        assert call(**kw) == 4, kw
