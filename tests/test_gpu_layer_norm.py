"""Layer norm and its gradients on the GPU against the fp64 oracle
(``oracle/layer_norm.py``), through the C ABI.

Bounds per element, with e = 2^-24 and one rounding of the output type on top.
Sums are at most 64 additions deep in a thread and then over at most 5 + 32
partial sums: 128 e of the absolute terms covers them and the few roundings
around them.  Forward: the mean is within 128 e of A = mean |x|, which moves
x - mean by as much, and rstd, relative to itself, by 64 e for the sum of
squares and by that shift over the deviation.  Backward is given the same
moments as the oracle.  A group's sums run over its rows one after the other
within a block and over the blocks: at most rows + 64 additions."""

import ctypes

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import layer_norm as ON

gpu = pytest.mark.gpu
E = 2.0 ** -24
EPS = 1e-6


def _np(t):
    return t.double().cpu().numpy()


def _inputs(rows, C, group_rows, dtype, seed=0, center=0.3, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    groups = -(-rows // group_rows)
    x = (torch.randn((rows, C), generator=g) * spread + center).to(dtype).cuda()
    dy = torch.randn((rows, C), generator=g).to(dtype).cuda()
    w, b = (torch.randn((groups, C), generator=g).cuda() for _ in range(2))
    return x, dy, w, b


def _check_forward(x, w, b, y, mean, rstd, group_rows, offset, what):
    xd = _np(x)
    ref, m_ref, r_ref = ON.forward(xd, None if w is None else _np(w), None if b is None else _np(b), EPS, group_rows,
                                   offset)
    rows = len(xd)
    at = np.arange(rows) // group_rows
    f = np.ones((1, 1)) if w is None else np.abs(offset + _np(w)[at])
    A, r = np.abs(xd).mean(1, keepdims=True), r_ref[:, None]
    d = np.abs(xd - m_ref[:, None])
    rel_r = 64 * E + 2 * 128 * E * A * r  # of rstd
    off = r * (128 * E * A + 2 * E * np.abs(xd)) + d * r * (rel_r + 4 * E)
    bias = 0.0 if b is None else np.abs(_np(b)[at])
    tol = f * off * (1 + 1e-3) + 4 * E * (f * d * r + bias) + torch.finfo(x.dtype).eps / 2 * np.abs(ref) + 1e-30
    err = np.abs(_np(y) - ref)
    assert np.all(err <= tol), f"{what}: y off by {np.max(err - tol):.3e} at {np.argwhere(err > tol)[:3]}"
    if mean is not None:
        assert np.all(np.abs(_np(mean) - m_ref) <= 128 * E * A[:, 0] + 1e-30), what
    if rstd is not None:
        assert np.all(np.abs(_np(rstd) - r_ref) <= r_ref * (rel_r[:, 0] + 4 * E)), what


def _check_backward(x, dy, w, mean, rstd, dx, dw, db, group_rows, offset, what):
    ref, scale = ON.backward(_np(x), _np(dy), None if w is None else _np(w), _np(mean), _np(rstd), group_rows, offset)
    deep = (128 + group_rows + 64) * E
    tols = [128 * E * scale[0] + torch.finfo(x.dtype).eps / 2 * np.abs(ref[0]), deep * scale[1], deep * scale[2]]
    for name, g, r, tol in zip(("dx", "dweight", "dbias"), (dx, dw, db), ref, tols):
        if g is None:
            continue
        err = np.abs(_np(g) - r)
        tol = tol + 1e-30
        assert np.all(err <= tol), f"{what}: {name} off by {np.max(err - tol):.3e} at {np.argwhere(err > tol)[:3]}"


def _moments(x):
    _, m, r = ON.forward(_np(x), None, None, EPS, len(x))
    return (torch.tensor(v, dtype=torch.float32).cuda() for v in (m, r))


def _both(x, dy, w, b, group_rows, offset, what, out=None, **kw):
    y = torch.empty_like(x) if out is None else out
    mean, rstd = (torch.empty(len(x), device="cuda") for _ in range(2))
    sab.layer_norm(x, w, b, EPS, y, mean, rstd, group_rows=group_rows, weight_offset=offset, **kw)
    _check_forward(x, w, b, y, mean, rstd, group_rows, offset, what)
    m, r = _moments(x)
    C = x.shape[1]
    dx = torch.empty_like(x) if out is None else out
    dw, db = (torch.full((-(-len(x) // group_rows), C), float("nan"), device="cuda") for _ in range(2))
    sab.layer_norm_backward(x, dy, w, m, r, dx, dw, db, group_rows=group_rows, weight_offset=offset, **kw)
    _check_backward(x, dy, w, m, r, dx, dw, db, group_rows, offset, what)


SHAPES = [
    # rows, C, group_rows
    (1, 1, 1), (1, 8, 1), (2, 7, 1), (3, 64, 3), (33, 65, 10), (5, 80, 2), (129, 100, 50), (300, 96, 300),
    (70, 256, 70), (1023, 257, 300), (64, 511, 64), (1536, 1536, 500), (40, 1001, 40), (17, 2048, 8),
    (9, 5120, 9), (6, 8184, 4), (5, 8191, 5), (3, 8192, 3), (5000, 24, 5000), (700, 40, 1),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, C, group_rows", SHAPES)
def test_shapes(rows, C, group_rows, dtype):
    x, dy, w, b = _inputs(rows, C, group_rows, dtype)
    _both(x, dy, w, b, group_rows, 1.0 if rows % 2 else 0.0, f"{rows}x{C}/{group_rows}")


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [64, 72, 1536])
def test_strides_and_rows_off_16_bytes(C, dtype):
    rows, group = 37, 11
    x, dy, w, b = _inputs(rows, C, group, dtype)
    for first, step in ((0, C + 8), (1, C + 8), (8, C + 9), (0, 2 * C)):
        wide = torch.full((rows, step + 8), float("nan"), dtype=dtype, device="cuda")
        xs = wide[:, first:first + C]
        xs.copy_(x)
        out = torch.full((rows, step + 8), 7.0, dtype=dtype, device="cuda")
        _both(xs, dy, w, b, group, 0.0, f"strided {first} {step}", out=out[:, first:first + C])
        assert bool((out[:, :first] == 7).all()) and bool((out[:, first + C:] == 7).all())


@gpu
def test_missing_weights_and_unwanted_outputs():
    x, dy, w, b = _inputs(50, 264, 50, torch.bfloat16)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y = torch.empty_like(x)
        sab.layer_norm(x, ww, bb, EPS, y)
        _check_forward(x, ww, bb, y, None, None, 50, 0.0, "no weights")
    m, r = _moments(x)
    for want in ((0, 0), (1, 0), (0, 1)):
        dx = torch.empty_like(x)
        dw, db = (torch.empty((1, 264), device="cuda") if on else None for on in want)
        sab.layer_norm_backward(x, dy, None, m, r, dx, dw, db)
        _check_backward(x, dy, None, m, r, dx, dw, db, 50, 0.0, f"wanted {want}")


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_off_centre_and_constant_rows(dtype):
    x, dy, w, b = _inputs(40, 512, 40, dtype, center=1000.0, spread=0.01 if dtype == torch.float32 else 8.0)
    x[3] = 5.0
    x[4] = 0.0
    _both(x, dy, w, b, 40, 0.0, "off centre")


@gpu
def test_in_place_and_leading_axes():
    x, dy, w, b = _inputs(60, 1536, 20, torch.bfloat16)
    y = torch.empty_like(x)
    sab.layer_norm(x, w, b, EPS, y, group_rows=20)
    z = x.clone().view(3, 20, 1536)
    sab.layer_norm(z, w, b, EPS, z, group_rows=20)
    assert torch.equal(z.view(60, 1536), y)
    m, r = _moments(x)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    dx = torch.empty_like(x)
    sab.layer_norm_backward(x, dy, w, m, r, dx, dw, db, group_rows=20)
    g = dy.clone()
    dw2, db2 = torch.empty_like(w), torch.empty_like(b)
    sab.layer_norm_backward(x, g, w, m, r, g, dw2, db2, group_rows=20)
    assert torch.equal(g, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)


@gpu
def test_a_bad_row_stays_in_its_row_and_equal_calls_give_equal_bits():
    x, dy, w, b = _inputs(2000, 1536, 2000, torch.bfloat16)
    y = torch.empty_like(x)
    sab.layer_norm(x, w, b, EPS, y)
    bad = x.clone()
    bad[77, 5] = float("inf")
    bad[78, 0] = float("nan")
    z = torch.empty_like(x)
    sab.layer_norm(bad, w, b, EPS, z)
    keep = [i for i in range(2000) if i not in (77, 78)]
    assert torch.equal(z[keep], y[keep]) and bool(z[77:79].isnan().any(1).all())
    m, r = _moments(x)
    first = None
    for _ in range(3):
        out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)]
        sab.layer_norm_backward(x, dy, w, m, r, *out)
        assert first is None or all(torch.equal(p, q) for p, q in zip(first, out))
        first = out


@gpu
def test_other_stream_and_graph():
    x, dy, w, b = _inputs(3000, 640, 1000, torch.bfloat16)
    m, r = _moments(x)

    def call(stream=None, ws=None):
        out = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)]
        torch.cuda.synchronize()
        sab.layer_norm(x, w, b, EPS, out[0], group_rows=1000, stream=stream)
        sab.layer_norm_backward(x, dy, w, m, r, *out[1:], group_rows=1000, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        return out

    ref = call()
    assert all(torch.equal(p, q) for p, q in zip(ref, call(torch.cuda.Stream())))
    ws = torch.empty(sab.layer_norm_backward_workspace(3000, 640, 1000), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sab.layer_norm(x, w, b, EPS, out[0], group_rows=1000)
        sab.layer_norm_backward(x, dy, w, m, r, *out[1:], group_rows=1000, workspace=ws)
    for _ in range(2):
        for t in out:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ref, out))


@gpu
def test_rows_past_2_31_elements():
    rows, C = (1 << 31) // 8192 + 2, 8192
    x = torch.empty((rows, C), dtype=torch.bfloat16, device="cuda")
    x[:2].normal_()
    x[-2:] = x[:2]
    x[2:-2] = 1.0
    sab.layer_norm(x, None, None, EPS, x)
    assert torch.equal(x[:2], x[-2:]) and bool(x[-1].any()) and not bool(x[2:-2:4096].any())
    _, m, r = (None, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"))
    db = torch.empty(C, device="cuda")
    sab.layer_norm_backward(x, x, None, m, r, x, None, db)
    assert torch.equal(x[:2], x[-2:])


def _desc(**kw):
    d = dict(rows=4, channels=64, group_rows=4, weight_offset=0.0, eps=1e-6, dtype=0)
    d.update(kw)
    return sab.NormDesc(*(d[n] for n, _ in sab.NormDesc._fields_))


def test_refusals_before_any_cuda_call():
    lib = sab.library()
    P = lambda a: None if a is None else ctypes.c_void_p(a)  # noqa: E731

    def fwd(d=_desc(), x=4096, xs=64, w=8192, b=12288, y=16384, ys=64, m=20480, r=24576):
        return lib.sab_layer_norm(ctypes.byref(d) if d else None, P(x), xs, P(w), P(b), P(y), ys, P(m), P(r), None)

    def bwd(d=_desc(), x=4096, xs=64, g=8192, gs=64, w=12288, m=16384, r=20480, dx=24576, ds=64, dw=28672, db=32768,
            ws=None, n=0):
        return lib.sab_layer_norm_backward(ctypes.byref(d) if d else None, P(x), xs, P(g), gs, P(w), P(m), P(r), P(dx),
                                           ds, P(dw), P(db), P(ws), n, None)

    shapes = [dict(d=None)] + [dict(d=_desc(**k)) for k in (
        dict(rows=0), dict(rows=1 << 31), dict(channels=0), dict(channels=8193), dict(group_rows=0), dict(eps=0.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("nan")), dict(dtype=2),
        dict(dtype=-1))]
    for kw in shapes + [dict(x=None), dict(x=4097), dict(xs=-64), dict(xs=1 << 60), dict(y=None), dict(ys=63),
                        dict(y=16385), dict(w=8194), dict(b=12289), dict(m=20482), dict(r=24577),
                        dict(y=4096, ys=128)]:
        assert fwd(**kw) == 1, kw
    for kw in shapes + [dict(x=None), dict(g=None), dict(g=8193), dict(gs=-1), dict(dx=None), dict(ds=10), dict(m=None),
                        dict(r=None), dict(m=16386), dict(dw=28673), dict(db=28672), dict(dx=8192, ds=128)]:
        assert bwd(**kw) == 1, kw
    need = sab.layer_norm_backward_workspace(4096, 64, 4096)
    assert need > 0 and sab.layer_norm_backward_workspace(4, 64, 4) == 0
    assert sab.layer_norm_backward_workspace(0, 64, 4) == 0
    big = _desc(rows=4096, group_rows=4096)
    for kw in (dict(), dict(ws=65536, n=need - 1), dict(ws=65536 + 16, n=need)):
        assert bwd(d=big, **kw) == 4, kw


def test_python_refusals():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        sab.layer_norm(x, None, None, 1e-6, x)  # not on the GPU
    with pytest.raises((TypeError, ValueError)):
        sab.layer_norm([1.0], None, None, 1e-6, x)
