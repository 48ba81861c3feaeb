"""Rotary positions and their gradient on the GPU against the fp64 oracle
(``oracle/rotary.py``), through the C ABI.

Bound per element, derived from the arithmetic: the angle's fraction of half a
turn is rounded to fp32 (2^-25, times pi), sine and cosine are within 2 ulp,
two products and a sum round in fp32; on |a| + |b| times the magnitude that
stays below 2^-21.  One rounding to the output type adds eps / 2 of the value."""

import ctypes

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import rotary as OR

gpu = pytest.mark.gpu
NAMES = {None: sab.ROTARY_SCALE_NONE, "linear": sab.ROTARY_SCALE_LINEAR, "base": sab.ROTARY_SCALE_BASE,
         "ramp": sab.ROTARY_SCALE_RAMP}


def _plan(bands, half, scaling=None, factor=1.0, magnitude=1.0):
    plan = sab.rotary_plan(bands, layout=sab.ROTARY_HALF if half else sab.ROTARY_INTERLEAVED, scaling=NAMES[scaling],
                           factor=factor, original_context=2048.0, magnitude=magnitude)
    return plan, OR.frequencies(bands, scaling=scaling, factor=factor, context=2048.0)


def _check(got, x, ang, half, magnitude, backward, dtype, what):
    xd = x.double().cpu().numpy()
    ref = OR.rotate(xd, ang, half, magnitude, backward)
    m = ang.shape[-1]
    mag = np.abs(xd).copy()
    i0 = np.arange(m) if half else 2 * np.arange(m)
    i1 = i0 + (m if half else 1)
    both = (np.abs(xd[..., i0]) + np.abs(xd[..., i1])) * magnitude
    mag[...] = 0.0
    mag[..., i0] = both
    mag[..., i1] = both
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = 2.0 ** -21 * mag + (torch.finfo(dtype).eps / 2) * np.abs(ref) * (mag > 0)
    assert np.all(err <= tol), f"{what}: worst {np.max(err - tol):.3e} at {np.argwhere(err > tol)[:3]}"


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


CASES = [
    # B, L, Hq, Hk, D, bands
    (1, 1, 1, 1, 8, (2,)),
    (1, 1, 12, 12, 128, (44, 42, 42)),
    (2, 37, 3, 1, 64, (64,)),
    (3, 5, 8, 2, 128, (64,)),
    (2, 19, 2, 2, 80, (80,)),
    (1, 130, 5, 5, 80, (30,)),
    (2, 9, 4, 1, 256, (256,)),
    (1, 33, 1, 1, 256, (2,)),
    (1, 7, 24, 24, 128, (10, 6, 4)),
    (1, 1037, 6, 3, 64, (32,)),
]


@gpu
@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}_h{c[2]}_{c[3]}_d{c[4]}_{'_'.join(map(str, c[5]))}" for c in CASES])
def test_rotary_and_gradient(case, dtype, half):
    B, L, Hq, Hk, D, bands = case
    scaling = [None, "linear", "ramp", "base"][(L + Hq) % 4] if min(bands) > 2 else None
    factor = 1.0 if scaling is None else 6.0
    plan, (f, ax) = _plan(bands, half, scaling, factor, magnitude=1.25)
    q, k = _rand((B, L, Hq, D), dtype, L), _rand((B, L, Hk, D), dtype, L + 1)
    rng = np.random.default_rng(L)
    pos = rng.integers(-5000, 1 << 24, (len(bands), B, L))
    dpos = torch.tensor(pos, device="cuda")
    ang = OR.angles(pos, f, ax)
    for backward, fn in ((False, sab.rotary), (True, sab.rotary_backward)):
        qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        fn(plan, q, k, qo, ko, positions=dpos)
        _check(qo, q, ang, half, 1.25, backward, dtype, "q")
        _check(ko, k, ang, half, 1.25, backward, dtype, "k")
        q1, k1 = q.clone(), k.clone()  # in place, then keys left out
        fn(plan, q1, k1, q1, k1, positions=dpos)
        assert torch.equal(q1, qo) and torch.equal(k1, ko)
        q2 = torch.empty_like(q)
        fn(plan, q, None, q2, positions=dpos)
        assert torch.equal(q2, qo)


@gpu
@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
def test_positions_of_any_size(half):
    """int64 positions to 2^40, negative ones, and the implied first_position + t."""
    plan, (f, ax) = _plan((64,), half)
    pos = np.array([[[0, 1, -1, 1 << 20, (1 << 31) + 5, (1 << 33) - 1, -(1 << 33), (1 << 40) + 7]]])
    x = _rand((1, 8, 2, 64), torch.float32, 3)
    y = torch.empty_like(x)
    sab.rotary(plan, x, None, y, positions=torch.tensor(pos, device="cuda"))
    # the plan's fp64 frequency is within 2^-52 relative, the oracle's is not
    # rounded: their angles part by |pos| f 2^-52
    ref = OR.rotate(x.double().cpu().numpy(), OR.angles(pos, f, ax), half)
    xa = np.abs(x.double().cpu().numpy())
    pair = xa + np.concatenate([xa[..., 32:], xa[..., :32]], -1) if half else xa + xa.reshape(1, 8, 2, 32, 2)[..., ::-1].reshape(xa.shape)
    tol = (2.0 ** -21 + np.abs(pos[0, :, :, None, None].astype(float)).reshape(1, 8, 1, 1) * 2.0 ** -52) * pair + 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)
    for first in (0, 77, -3, 1 << 35):
        a, b = torch.empty_like(x), torch.empty_like(x)
        sab.rotary(plan, x, None, a, first_position=first)
        sab.rotary(plan, x, None, b, positions=torch.arange(first, first + 8, device="cuda"))
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
def test_strided_rows(half):
    """Slices of a fused projection, of a longer buffer, and a sequence-first
    layout; what lies between the rows stays as it was."""
    B, L, Hq, Hk, D = 2, 21, 4, 2, 64
    plan, (f, ax) = _plan((D,), half)
    fused = _rand((B, L, (Hq + 2 * Hk) * D), torch.bfloat16, 5)
    before = fused.clone()
    q, k = (fused[..., a * D:b * D].unflatten(-1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hk)))
    pos = np.arange(L)[None, None].repeat(B, 1)
    ang = OR.angles(pos, f, ax)
    qc, kc = q.clone(), k.clone()
    sab.rotary(plan, q, k, q, k)  # in place in the fused buffer
    _check(q, qc, ang, half, 1.0, False, torch.bfloat16, "fused q")
    _check(k, kc, ang, half, 1.0, False, torch.bfloat16, "fused k")
    assert torch.equal(fused[..., (Hq + Hk) * D:], before[..., (Hq + Hk) * D:])
    long = torch.full((B, 50, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sab.rotary(plan, qc, kc, torch.empty_like(qc), long[:, 11:11 + L])
    assert torch.equal(long[:, 11:11 + L], k)
    assert bool((long[:, :11] == 7).all()) and bool((long[:, 11 + L:] == 7).all())
    seq_first = torch.empty((L, B, Hk, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    sab.rotary(plan, kc, None, seq_first)
    assert torch.equal(seq_first, k)
    same = kc[:1].expand(B, L, Hk, D)  # a broadcast input
    out = torch.empty_like(kc)
    sab.rotary(plan, same, None, out)
    assert torch.equal(out[1], out[0]) and torch.equal(out[0], k[0])


@gpu
def test_gradient_against_differences():
    """<rotary(x + e) - rotary(x - e), dy> / 2 = <e, rotary_backward(dy)> (the
    map is linear): fp32, relative to the sums of absolute products."""
    plan, _ = _plan((24, 20, 20), False, magnitude=0.75)
    x, e, dy = (_rand((2, 33, 3, 64), torch.float32, s) for s in (1, 2, 3))
    pos = torch.randint(0, 9000, (3, 2, 33), device="cuda")
    up, dn, dx = (torch.empty_like(x) for _ in range(3))
    sab.rotary(plan, x + e, None, up, positions=pos)
    sab.rotary(plan, x - e, None, dn, positions=pos)
    sab.rotary_backward(plan, dy, None, dx, positions=pos)
    lhs = ((up.double() - dn.double()) * dy.double()).sum() / 2
    rhs = (e.double() * dx.double()).sum()
    # 2^-21 on each of |x|, |e| (each element meets two outputs)
    room = 2.0 ** -20 * ((x.abs() + e.abs()).double().sum() * dy.abs().max() * 2)
    assert abs(lhs - rhs) <= room


@gpu
def test_special_values_stay_in_their_pair():
    """An infinity or NaN reaches its own pair only; -0 and the unrotated part keep their bits."""
    for half in (False, True):
        plan, _ = _plan((32,), half)
        x = _rand((1, 3, 2, 64), torch.bfloat16, 9)
        clean = torch.empty_like(x)
        sab.rotary(plan, x, None, clean)
        x[0, 1, 0, 4], x[0, 2, 1, 40] = float("nan"), float("-inf")
        x[0, 2, 1, 41] = -0.0
        y = torch.empty_like(x)
        sab.rotary(plan, x, None, y)
        mate = 4 + 16 if half else 5
        bad = torch.isnan(y)
        assert bool(bad[0, 1, 0, 4]) and bool(bad[0, 1, 0, mate]) and int(bad.sum()) == 2
        assert y[0, 2, 1, 40] == float("-inf") and torch.signbit(y[0, 2, 1, 41])
        keep = ~bad
        keep[0, 2, 1, 40:42] = False
        assert torch.equal(y[keep], clean[keep])


@gpu
def test_stream_and_graph():
    plan, (f, ax) = _plan((64,), True)
    x = _rand((2, 40, 3, 64), torch.bfloat16, 4)
    pos = torch.arange(80, device="cuda").view(1, 2, 40)
    want, y = torch.empty_like(x), torch.zeros_like(x)
    sab.rotary(plan, x, None, want, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sab.rotary(plan, x, None, y, positions=pos, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sab.rotary(plan, x, None, y, positions=pos)
    pos += 1000
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    _check(y, x, OR.angles(pos.cpu().numpy(), f, ax), True, 1.0, False, torch.bfloat16, "replay")


@gpu
def test_more_than_2_to_31_elements():
    """Rows behind 2^31 elements: the last tokens against the oracle."""
    B, L, H, D = 1, 4200000, 4, 128
    plan, (f, ax) = _plan((D,), True)
    x = torch.zeros((B, L, H, D), dtype=torch.bfloat16, device="cuda")
    x[:, -64:] = _rand((B, 64, H, D), torch.bfloat16, 8)
    tail = x[:, -64:].clone()
    sab.rotary(plan, x, None, x)
    pos = np.arange(L - 64, L)[None, None]
    _check(x[:, -64:], tail, OR.angles(pos, f, ax), True, 1.0, False, torch.bfloat16, "tail")
    assert not bool(x[:, :-64].any())


def _rows(**kw):
    r = dict(inp=4096, out=8192, heads=2, in_batch=0, in_token=128, out_batch=0, out_token=128)
    r.update(kw)
    return sab._abi.RotaryRows(*[r[n] for n, _ in sab._abi.RotaryRows._fields_])


def test_refusals_before_any_cuda_call():
    lib = sab.library()
    plan = sab.rotary_plan((64,))
    multi = sab.rotary_plan((16, 16, 16))
    P = ctypes.c_void_p(4096)

    def call(pl=plan, q=None, k=None, pos=None, B=1, L=4, D=64, dt=0, fn="sab_rotary"):
        q = _rows() if q is None else q
        return getattr(lib, fn)(ctypes.byref(pl) if pl is not None else None,
                                ctypes.byref(q) if q != 0 else None, ctypes.byref(k) if k is not None else None, pos, 0,
                                B, L, D, dt, None)

    for fn in ("sab_rotary", "sab_rotary_backward"):
        bad = [dict(pl=None), dict(pl=sab.RotaryPlan()), dict(q=0), dict(q=_rows(inp=None)), dict(q=_rows(out=None)),
               dict(q=_rows(inp=4104)), dict(q=_rows(out=8200)), dict(q=_rows(heads=0)), dict(q=_rows(in_token=132)),
               dict(q=_rows(out_token=64)), dict(q=_rows(in_token=-128)), dict(B=2),  # batches on top of each other
               dict(q=_rows(out=4096, out_token=256)), dict(k=_rows()), dict(k=_rows(inp=8192, out=12288)),
               dict(k=_rows(out=4096)), dict(k=_rows(heads=-1)), dict(k=_rows(inp=None)),
               dict(pl=multi), dict(pos=ctypes.c_void_p(4100)), dict(D=60), dict(D=0), dict(D=264), dict(D=32),
               dict(B=0), dict(L=0), dict(L=(1 << 30) + 1), dict(dt=2), dict(dt=-1),
               dict(pl=multi, pos=ctypes.c_void_p(4097))]
        for kw in bad:
            assert call(fn=fn, **kw) == 1, (fn, kw)
    for field, value in (("axes", 0), ("axes", 4), ("dims", 0), ("dims", 63), ("dims", 258), ("magic", 1)):
        broken = sab.rotary_plan((64,))
        setattr(broken, field, value)
        assert call(pl=broken) == 1, field
    broken = sab.rotary_plan((64,))
    broken.axis[31] = 1
    assert call(pl=broken) == 1
    assert P.value == 4096


def test_python_refusals():
    plan = sab.rotary_plan((64,))
    x = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sab.rotary(plan, x, None, x)  # not on the GPU
    with pytest.raises(TypeError):
        sab.rotary(plan, x[0], None, x[0])


@gpu
def test_more_tokens_than_32_bits_are_refused():
    plan = sab.rotary_plan((8,))
    x = torch.ones((1, 1, 1, 8), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sab.SabError):  # not taken for one token
        sab.rotary(plan, x.expand((1 << 32) + 1, 1, 1, 8), None, x.expand((1 << 32) + 1, 1, 1, 8), first_position=1)
    torch.cuda.synchronize()
    assert bool((x == 1).all())
