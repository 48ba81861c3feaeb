"""Decay attention, its single-token form and its gradients on the GPU against
the fp64 recurrence (``oracle/decay.py``), through the C ABI.

Bounds, from the documented roundings (a rounding to bf16 moves a value by at
most 2^-8 of it).  Every output is a sum of products; the oracle returns the
same sum over absolute values, A.  Rounding the masked scores (tokens of the
same block) or the state's copy (tokens before it) to bf16 changes the output
by at most 2^-8 A; k on its way into the state carries 16 bits (2^-16 A); the
decay powers and fp32 sums stay below 2^-13 A.  The bf16 output rounds once
more: 2^-8 |value|.  A state gets only the 2^-16, the powers (the exponent's
fp32 argument, at most 40 where the power matters: 40 * 2^-23) and the sums:
2^-15 A.  On random inputs the roundings are independent, so the error's norm
is also below 2^-8 of the output's norm: two uniform errors of 2^-8 / sqrt(3)
each give 0.82 * 2^-8."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import decay as OD
from oracle import rotary as OR
from streaming_attention_block_gb300._abi import _guarded

gpu = pytest.mark.gpu

DECAYS = [-0.5, -0.02, 0.0, -1e-3, -4.0, float("-inf"), 0.7, -2e4]


def _ld(H, start=0):
    return torch.tensor([DECAYS[(start + h) % len(DECAYS)] for h in range(H)], device="cuda")


def _n(t):
    return None if t is None else t.double().cpu().numpy()


def _randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _out(shape, dtype=torch.bfloat16):
    """An output between canary bands (checked after every test), holding NaN."""
    n = int(np.prod(shape)) * dtype.itemsize
    t = _guarded(n, 4096, "cuda")[1].view(dtype).view(shape)
    t.fill_(float("nan"))
    return t


def _ws(n):
    return _guarded(n, 4096, "cuda")[1] if n else None


def _check(got, ref, bound, what, state=False, norm=True):
    g, r = _n(got), ref
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    err = np.abs(g - r)
    tol = 2.0 ** -15 * bound if state else 2.0 ** -8 * np.abs(r) + (2.0 ** -8 + 2.0 ** -12) * bound
    tol = tol + 1e-30
    assert np.all(err <= tol), f"{what}: worst ratio {np.max(err / tol):.2f} at {np.argwhere(err > tol)[:3].tolist()}"
    if norm and r.size >= 4096:
        lim = 2.0 ** (-15 if state else -8) * np.linalg.norm(r)
        assert np.linalg.norm(err) <= lim, f"{what}: norm ratio {np.linalg.norm(err) / lim:.3f}"


def _forward(q, k, v, ld, scale, state=None, lens=None, inplace=False, want_state=True):
    B, L, H, D = q.shape
    O = _out(q.shape)
    So = None
    if want_state:
        So = _out((B, H, D, D), torch.float32)
        if inplace:
            So.copy_(state)
            state = So
    sab.decay_attention(q, k, v, ld, scale, O, state_in=state, state_out=So, seq_len=lens,
                        workspace=_ws(sab.decay_attention_workspace(B, L, H, D)))
    return O, So


SHAPES = [
    # B, L, H, D, lens
    (1, 1, 1, 64, None),
    (1, 2, 3, 128, None),
    (2, 16, 2, 64, (16, 3)),
    (1, 17, 2, 128, None),
    (3, 127, 2, 64, (0, 127, 64)),
    (2, 128, 3, 128, None),
    (2, 129, 4, 64, (129, 128)),
    (2, 129, 2, 128, (1, 129)),
    (3, 300, 8, 128, (300, 257, 0)),
    (2, 300, 8, 64, None),
    (1, 700, 8, 128, (613,)),
    (4, 513, 3, 64, (600, -5, 512, 100)),
    (1, 1536, 2, 128, None),
    (40, 130, 8, 64, None),
]
IDS = [f"{b}x{l}_h{h}_d{d}{'_ragged' if n else ''}" for b, l, h, d, n in SHAPES]


@gpu
@pytest.mark.parametrize("with_state", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_forward(case, with_state):
    B, L, H, D, lens = case
    q, k, v = (_randn((B, L, H, D), 10 * L + i) for i in range(3))
    ld = _ld(H, L)
    S = _randn((B, H, D, D), L + 7, torch.float32) * 3 if with_state else None
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:  # padding holds anything
        for b, n in enumerate(lens):
            n = min(max(n, 0), L)
            q[b, n:], k[b, n:], v[b, n:] = float("nan"), float("inf"), float("nan")
    O, So = _forward(q, k, v, ld, D ** -0.5, S, dl)
    o, s, oa, sa = OD.decay_attention(_n(q), _n(k), _n(v), _n(ld), D ** -0.5, _n(S), lens)
    _check(O, o, oa, "O")
    _check(So, s, sa, "state", state=True)
    if lens is not None:
        for b, n in enumerate(lens):
            assert not bool(O[b, min(max(n, 0), L):].any())
    O2, none = _forward(q, k, v, ld, D ** -0.5, S, dl, want_state=False)
    # (k enters a state that nobody asked for with 16 bits instead of 24: other bits, same bounds)
    _check(O2, o, oa, "O without state_out")
    assert none is None
    if with_state:
        O3, S3 = _forward(q, k, v, ld, D ** -0.5, S, dl, inplace=True)
        assert torch.equal(O3, O) and torch.equal(S3, So)


@gpu
@pytest.mark.parametrize("with_state", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_backward(case, with_state):
    B, L, H, D, lens = case
    q, k, v, do = (_randn((B, L, H, D), 20 * L + i) for i in range(4))
    ld = _ld(H, L + 1)
    scale = D ** -0.5
    S = _randn((B, H, D, D), L + 7, torch.float32) * 3 if with_state else None
    dS = _randn((B, H, D, D), L + 8, torch.float32) if with_state else None
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:
        for b, n in enumerate(lens):
            n = min(max(n, 0), L)
            q[b, n:], k[b, n:], v[b, n:], do[b, n:] = float("inf"), float("nan"), float("inf"), float("nan")
    refs, bnds = OD.decay_attention_backward(_n(q), _n(k), _n(v), _n(do), _n(ld), scale, _n(S), _n(dS), lens)
    outs = []
    for inplace in (False, True):
        g = [_out(q.shape) for _ in range(3)]
        dSi = _out((B, H, D, D), torch.float32)
        d_out = dS
        if inplace and with_state:
            dSi.copy_(dS)
            d_out = dSi
        sab.decay_attention_backward(q, k, v, do, ld, scale, *g, state_in=S, d_state_out=d_out, d_state_in=dSi,
                                     seq_len=dl, workspace=_ws(sab.decay_attention_backward_workspace(B, L, H, D)))
        outs.append(g + [dSi])
    for n, got, ref, bnd in zip(("dQ", "dK", "dV"), outs[0], refs, bnds):
        _check(got, ref, bnd, n)
        if lens is not None:
            for b, m in enumerate(lens):
                assert not bool(got[b, min(max(m, 0), L):].any())
    _check(outs[0][3], refs[3], bnds[3], "d_state_in", state=True)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def _fp64_on_gpu(q, k, v, ld, scale, S):
    """The recurrence in fp64 torch operations (long sequences)."""
    B, L, H, D = q.shape
    g = torch.exp(ld.double().clamp(max=0))[:, None, None]
    O = torch.empty((B, L, H, D), dtype=torch.float64, device=q.device)
    A, Oa = S.abs(), torch.empty_like(O)
    for t in range(L):
        kk, vv, qq = (x[:, t].double() for x in (k, v, q))
        kv = kk.unsqueeze(-1) * vv.unsqueeze(-2)
        S = g * S + kv
        A = g * A + kv.abs()
        O[:, t] = scale * (qq.unsqueeze(-2) @ S).squeeze(-2)
        Oa[:, t] = scale * (qq.abs().unsqueeze(-2) @ A).squeeze(-2)
    return O, S, Oa, A


def _fp64_back_on_gpu(q, k, v, do, ld, scale, S, R):
    """Gradients by the adjoint recurrence, and their absolute sums."""
    B, L, H, D = q.shape
    g = torch.exp(ld.double().clamp(max=0))[:, None, None]
    A, Ra = S.abs(), R.abs()
    out = [torch.empty((B, L, H, D), dtype=torch.float64, device=q.device) for _ in range(6)]
    dq, dk, dv, dqa, dka, dva = out
    for t in range(L):
        kv = k[:, t].double().unsqueeze(-1) * v[:, t].double().unsqueeze(-2)
        S = g * S + kv
        A = g * A + kv.abs()
        d = do[:, t].double().unsqueeze(-1)
        dq[:, t] = scale * (S @ d).squeeze(-1)
        dqa[:, t] = scale * (A @ d.abs()).squeeze(-1)
    for t in range(L - 1, -1, -1):
        w = scale * q[:, t].double().unsqueeze(-1) * do[:, t].double().unsqueeze(-2)
        R = R + w
        Ra = Ra + w.abs()
        kk, vv = k[:, t].double().unsqueeze(-2), v[:, t].double().unsqueeze(-1)
        dk[:, t], dv[:, t] = (R @ vv).squeeze(-1), (kk @ R).squeeze(-2)
        dka[:, t], dva[:, t] = (Ra @ vv.abs()).squeeze(-1), (kk.abs() @ Ra).squeeze(-2)
        R = g * R
        Ra = g * Ra
    return (dq, dk, dv, R), (dqa, dka, dva, Ra)


# few heads: the sequence is worked on in parallel segments, whose states are
# summed and chained by kernels of their own
@gpu
@pytest.mark.parametrize("L", [3000, 7000, 20011])
@pytest.mark.parametrize("D", [64, 128])
def test_long_sequence(D, L):
    B, H = 1, 3
    q, k, v, do = (_randn((B, L, H, D), 50 + i) for i in range(4))
    ld = torch.tensor([-1e-4, -0.01, 0.0], device="cuda")
    scale = D ** -0.5
    S, dS = (_randn((B, H, D, D), 60 + i, torch.float32) for i in range(2))
    o, s, oa, sa = _fp64_on_gpu(q, k, v, ld, scale, S.double())
    O, So = _forward(q, k, v, ld, scale, S)
    _check(O, _n(o), _n(oa), "O")
    _check(So, _n(s), _n(sa), "state", state=True)
    O2, S2 = _forward(q, k, v, ld, scale, S, inplace=True)
    assert torch.equal(O2, O) and torch.equal(S2, So)
    refs, bnds = _fp64_back_on_gpu(q, k, v, do, ld, scale, S.double(), dS.double())
    g = [_out(q.shape) for _ in range(3)]
    ws = _ws(sab.decay_attention_backward_workspace(B, L, H, D))
    d_in = _out(S.shape, torch.float32)
    d_in.copy_(dS)
    sab.decay_attention_backward(q, k, v, do, ld, scale, *g, state_in=S, d_state_out=d_in, d_state_in=d_in,
                                 workspace=ws)
    for n, got, ref, bnd in zip(("dQ", "dK", "dV", "d_state_in"), g + [d_in], refs, bnds):
        _check(got, _n(ref), _n(bnd), n, state=n == "d_state_in")


@gpu
@pytest.mark.parametrize("case", [(8, 1024, 6, 64), (3, 2300, 4, 128), (2, 9000, 2, 128), (23, 400, 8, 64)])
def test_ragged_segments(case):
    """Unequal lengths cut into segments: some end in the middle of one, some
    have none of their tokens in it.  The last case has more sequences than
    SMs, which are then taken longest first."""
    B, L, H, D = case
    lens = torch.tensor([L * (b * 37 % 100) // 100 for b in range(B)], dtype=torch.int32, device="cuda")
    lens[-1] = L
    q, k, v, do = (_randn((B, L, H, D), 160 + i) for i in range(4))
    ld = _ld(H, 1)
    S, dS = (_randn((B, H, D, D), 170 + i, torch.float32) for i in range(2))
    for b, n in enumerate(lens.tolist()):
        for x in (q, k, v, do):
            x[b, n:] = float("nan")
    O, So = _forward(q, k, v, ld, 0.1, S, lens)
    g = [_out(q.shape) for _ in range(3)]
    d_in = _out(S.shape, torch.float32)
    sab.decay_attention_backward(q, k, v, do, ld, 0.1, *g, state_in=S, d_state_out=dS, d_state_in=d_in, seq_len=lens,
                                 workspace=_ws(sab.decay_attention_backward_workspace(B, L, H, D)))
    for b, n in enumerate(lens.tolist()):
        for x in [O] + g:
            assert not bool(x[b, n:].any())
        if n == 0:
            assert torch.equal(So[b], S[b]) and torch.equal(d_in[b], dS[b])
            continue
        # each sequence by itself: the same numbers, cut otherwise
        one = [x[b:b + 1, :n].contiguous() for x in (q, k, v, do)]
        o, s, oa, sa = _fp64_on_gpu(one[0], one[1], one[2], ld, 0.1, S[b:b + 1].double())
        _check(O[b:b + 1, :n], _n(o), _n(oa), f"O {b}")
        _check(So[b:b + 1], _n(s), _n(sa), f"state {b}", state=True)
        refs, bnds = _fp64_back_on_gpu(*one, ld, 0.1, S[b:b + 1].double(), dS[b:b + 1].double())
        for name, got, ref, bnd in zip(("dQ", "dK", "dV"), g, refs, bnds):
            _check(got[b:b + 1, :n], _n(ref), _n(bnd), f"{name} {b}")
        _check(d_in[b:b + 1], _n(refs[3]), _n(bnds[3]), f"d_state_in {b}", state=True)


@gpu
@pytest.mark.parametrize("states", [False, True], ids=["no_states", "states"])
@pytest.mark.parametrize("case", [(2, 1300, 12, 64), (1, 4000, 24, 128), (1, 4000, 24, 64), (1, 1500, 12, 128),
                                  (60, 200, 3, 128), (60, 200, 3, 64), (5, 700, 30, 128)])
def test_gradients_in_several_waves(case, states):
    """The three runs of a gradient share launches of up to four times as many
    blocks as SMs, in segments and as whole sequences of equal or unequal
    lengths, with and without states."""
    B, L, H, D = case
    q, k, v, do = (_randn((B, L, H, D), 210 + i) for i in range(4))
    ld = _ld(H, 1)
    S, dS = (_randn((B, H, D, D), 220 + i, torch.float32) if states else None for i in range(2))
    lens = torch.tensor([L - 11 * b for b in range(B)], dtype=torch.int32).clamp(min=0).cuda() if B > 2 else None
    if lens is not None:
        for b, n in enumerate(lens.tolist()):
            for x in (q, k, v, do):
                x[b, n:] = float("nan")
    g = [_out(q.shape) for _ in range(3)]
    d_in = _out((B, H, D, D), torch.float32) if states else None
    sab.decay_attention_backward(q, k, v, do, ld, 0.1, *g, state_in=S, d_state_out=dS, d_state_in=d_in, seq_len=lens,
                                 workspace=_ws(sab.decay_attention_backward_workspace(B, L, H, D)))
    zero = torch.zeros((B, H, D, D), dtype=torch.float64, device="cuda")
    for b, n in enumerate([L] * B if lens is None else lens.tolist()):
        for x in g:
            assert not bool(x[b, n:].any())
        if n == 0:
            assert d_in is None or torch.equal(d_in[b], dS[b])
            continue
        one = [x[b:b + 1, :n].contiguous() for x in (q, k, v, do)]
        s0, r0 = ((S[b:b + 1].double(), dS[b:b + 1].double()) if states else (zero[b:b + 1], zero[b:b + 1]))
        refs, bnds = _fp64_back_on_gpu(*one, ld, 0.1, s0, r0)
        for name, got, ref, bnd in zip(("dQ", "dK", "dV"), g, refs, bnds):
            _check(got[b:b + 1, :n], _n(ref), _n(bnd), f"{name} {b}")
        if states:
            _check(d_in[b:b + 1], _n(refs[3]), _n(bnds[3]), f"d_state_in {b}", state=True)


@gpu
def test_pieces_and_single_tokens_equal_the_whole():
    """A stream fed as chunks and then token by token, through DecayState."""
    B, L, H, D = 2, 300, 3, 128
    q, k, v = (_randn((B, L, H, D), 70 + i) for i in range(3))
    ld = torch.tensor([-0.3, -1e-3, 0.0], device="cuda")
    o, s, oa, sa = OD.decay_attention(_n(q), _n(k), _n(v), _n(ld), D ** -0.5)
    st = sab.DecayState(ld, B, D)
    parts, t = [], 0
    for n in (128, 1, 100, 40, 20):
        parts.append(st.attention(*(x[:, t:t + n].contiguous() for x in (q, k, v))))
        t += n
    while t < L:
        parts.append(st.step(*(x[:, t].contiguous() for x in (q, k, v)))[:, None])
        t += 1
    _check(torch.cat(parts, 1), o, oa, "stream")
    _check(st.state, s, sa, "state", state=True)
    st.reset()
    assert not bool(st.state.any())


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 12), (5, 3), (64, 8), (300, 8)])
def test_step(B, H, D):
    q, k, v = (_randn((B, H, D), B + i) for i in range(3))
    ld = _ld(H, B)
    S = _randn((B, H, D, D), 3, torch.float32)
    active = (torch.arange(B, device="cuda") % 3 != 1).to(torch.int32) * 5
    O, So = _out(q.shape), _out(S.shape, torch.float32)
    args = [_n(x)[:, None] for x in (q, k, v)]
    for act in (None, active):
        lens = None if act is None else (act != 0).int().cpu().numpy()
        o, s, oa, sa = OD.decay_attention(*args, _n(ld), 0.3, _n(S), lens)
        sab.decay_attention_step(q, k, v, ld, 0.3, S, So, O, active=act)
        # fp32 throughout: D products, 2^-24 each and the running sums
        err = np.abs(_n(O)[:, None] - o)
        assert np.all(err <= 2.0 ** -8 * np.abs(o) + 2.0 ** -16 * oa)
        assert np.all(np.abs(_n(So) - s) <= 2.0 ** -20 * sa + 1e-30)
        if act is not None:
            off = act == 0
            assert torch.equal(So[off], S[off]) and not bool(O[off].any())
        S2, O2 = S.clone(), _out(q.shape)
        sab.decay_attention_step(q, k, v, ld, 0.3, S2, S2, O2, active=act)
        assert torch.equal(S2, So) and torch.equal(O2, O)
        sab.decay_attention_step(q, k, v, ld, 0.3, None, So, O, active=act)
        sab.decay_attention_step(q, k, v, ld, 0.3, torch.zeros_like(S), S2, O2, active=act)
        assert torch.equal(S2, So) and torch.equal(O2, O)
    off = active == 0  # an inactive sequence's token may hold anything
    if bool(off.any()):
        q2, k2, v2 = (x.clone() for x in (q, k, v))
        for x in (q2, k2, v2):
            x[off] = float("nan")
        sab.decay_attention_step(q, k, v, ld, 0.3, S, So, O, active=active)
        sab.decay_attention_step(q2, k2, v2, ld, 0.3, S, S2, O2, active=active)
        assert torch.equal(S2, So) and torch.equal(O2, O)


@gpu
def test_nonfinite_tokens_reach_later_tokens_only():
    """A NaN in live k or v: tokens before it are untouched."""
    B, L, H, D = 1, 300, 2, 64
    q, k, v = (_randn((B, L, H, D), 80 + i) for i in range(3))
    ld = torch.tensor([-0.1, 0.0], device="cuda")
    O, _ = _forward(q, k, v, ld, 0.1)
    for t in (5, 140, 299):
        k2, v2 = k.clone(), v.clone()
        k2[0, t, 0, 3] = float("nan")
        v2[0, t, 1, 9] = float("inf")
        O2, _ = _forward(q, k2, v2, ld, 0.1)
        start = t // 128 * 128  # tokens of earlier blocks: the same bits
        assert torch.equal(O2[:, :start], O[:, :start])
        assert bool(torch.isnan(O2[0, t:, 0]).all())
        assert not bool(torch.isfinite(O2[0, t:, 1, 9]).any())


@gpu
def test_gradient_against_differences():
    """Central differences of sum(O dO) + sum(S dS) through the forward call,
    along random directions of q, k, v and the state."""
    B, L, H, D = 1, 200, 2, 64
    scale = D ** -0.5
    q, k, v, do = (_randn((B, L, H, D), 90 + i) for i in range(4))
    ld = torch.tensor([-0.05, -2e-3], device="cuda")
    S, dS = (_randn((B, H, D, D), 95 + i, torch.float32) for i in range(2))
    g = [torch.empty_like(q) for _ in range(3)]
    dSi = torch.empty_like(S)
    sab.decay_attention_backward(q, k, v, do, ld, scale, *g, state_in=S, d_state_out=dS, d_state_in=dSi)
    refs = OD.decay_attention_backward(_n(q), _n(k), _n(v), _n(do), _n(ld), scale, _n(S), _n(dS))[0]

    def loss(x):
        O, So = _forward(*x[:3], ld, scale, x[3])
        return (O.double() * do.double()).sum() + (So.double() * dS.double()).sum()

    for i in range(4):
        # a step along the gradient's own direction, in values bf16 holds exactly
        step = torch.sign(torch.tensor(refs[i])).cuda() * 0.25
        hi, lo = ([x if j != i else (x.float() + s * step.float()).to(x.dtype) for j, x in enumerate((q, k, v, S))]
                  for s in (1, -1))
        moved = hi[i].double() - lo[i].double()
        num = float(loss(hi) - loss(lo))
        got = float((moved * (g + [dSi])[i].double()).sum())
        # linear in each argument: only roundings part the two, 2^-7 of the
        # sums that do not cancel along this direction
        assert abs(num - got) <= 2.0 ** -6 * float((moved.abs() * (g + [dSi])[i].double().abs()).sum())


@gpu
def test_rotary_then_decay_attention_training():
    """Rotary, decay attention and both gradients in a row, as a layer uses
    them, against the fp64 composition."""
    B, L, H, D = 2, 260, 2, 64
    scale = D ** -0.5
    plan = sab.rotary_plan((24, 20, 20))
    f, ax = OR.frequencies((24, 20, 20))
    t = np.arange(L)
    pos = np.stack([t // 20, t // 5 % 4, t % 5])[:, None].repeat(B, 1)
    dpos, ang = torch.tensor(pos, device="cuda"), OR.angles(pos, f, ax)
    q, k, v, do = (_randn((B, L, H, D), 110 + i) for i in range(4))
    ld = torch.tensor([-0.1, -1e-3], device="cuda")
    lens = torch.tensor([L, 131], dtype=torch.int32, device="cuda")
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    sab.rotary(plan, q, k, qr, kr, positions=dpos)
    O = torch.empty_like(q)
    sab.decay_attention(qr, kr, v, ld, scale, O, seq_len=lens)
    dqr, dkr, dv = (torch.empty_like(q) for _ in range(3))
    sab.decay_attention_backward(qr, kr, v, do, ld, scale, dqr, dkr, dv, seq_len=lens)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    sab.rotary_backward(plan, dqr, dkr, dq, dk, positions=dpos)
    qn, kn = OR.rotate(_n(q), ang, False), OR.rotate(_n(k), ang, False)
    n = lens.cpu().numpy()
    o = OD.decay_attention(qn, kn, _n(v), _n(ld), scale, lens=n)[0]
    g = OD.decay_attention_backward(qn, kn, _n(v), _n(do), _n(ld), scale, lens=n)[0]
    want = [o, OR.rotate(g[0], ang, False, backward=True), OR.rotate(g[1], ang, False, backward=True), g[2]]
    for name, got, ref in zip(("O", "dQ", "dK", "dV"), (O, dq, dk, dv), want):
        # independent roundings in a row, each 2^-8 / sqrt(3) of the norm: q', k'
        # (or the gradients), the scores or state, two stored results
        assert np.linalg.norm(_n(got) - ref) <= np.sqrt(5 / 3) * 2.0 ** -8 * np.linalg.norm(ref), name


@gpu
def test_streams_and_graph():
    """A side stream, two captured graphs with their own workspaces and a
    replay on new inputs."""
    B, L, H, D = 1, 900, 2, 128
    x = [_randn((B, L, H, D), 120 + i) for i in range(4)]
    y = [_randn((B, L, H, D), 130 + i) for i in range(4)]
    ld = torch.tensor([-0.01, -0.2], device="cuda")

    def run(a, outs, stream=None):
        O, S, g, d = outs
        sab.decay_attention(a[0], a[1], a[2], ld, 0.1, O, state_out=S, stream=stream)
        sab.decay_attention_backward(a[0], a[1], a[2], a[3], ld, 0.1, *g, d_state_in=d, stream=stream)

    def fresh():
        return (torch.zeros_like(x[0]), torch.zeros((B, H, D, D), device="cuda"), [torch.zeros_like(x[0]) for _ in range(3)],
                torch.zeros((B, H, D, D), device="cuda"))

    def flat(o):
        return [o[0], o[1], *o[2], o[3]]

    wx, wy, a, b = fresh(), fresh(), fresh(), fresh()
    run(x, wx)
    run(y, wy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(x, a, s)
    torch.cuda.synchronize()
    for p, q in zip(flat(a), flat(wx)):
        assert torch.equal(p, q)
    static = [t.clone() for t in x]
    graphs = []
    for outs in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(static, outs)
        graphs.append(g)
    for src, want in ((y, wy), (x, wx)):
        for d, t in zip(static, src):
            d.copy_(t)
        for o in flat(a) + flat(b):
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for p, q, w in zip(flat(a), flat(b), flat(want)):
            assert torch.equal(p, w) and torch.equal(q, w)


@gpu
def test_two_streams_at_once():
    """Calls of two streams overlap on the GPU; each has its own workspace."""
    ld = torch.tensor([-0.02, 0.0], device="cuda")
    sides = []
    for i, (B, L, H, D) in enumerate([(1, 2000, 2, 128), (2, 900, 2, 64)]):
        x = [_randn((B, L, H, D), 180 + 10 * i + j) for j in range(4)]
        want = [torch.empty_like(x[0]) for _ in range(4)] + [torch.empty((B, H, D, D), device="cuda")]
        got = [torch.zeros_like(t) for t in want]
        ws = [torch.empty(max(256, n), dtype=torch.uint8, device="cuda") for n in
              (sab.decay_attention_workspace(B, L, H, D), sab.decay_attention_backward_workspace(B, L, H, D))]
        sides.append((x, want, got, ws, torch.cuda.Stream()))

    def run(x, out, ws, stream=None):
        sab.decay_attention(x[0], x[1], x[2], ld, 0.1, out[0], state_out=out[4], workspace=ws[0], stream=stream)
        sab.decay_attention_backward(*x, ld, 0.1, *out[1:4], workspace=ws[1], stream=stream)

    for x, want, _, ws, _ in sides:
        run(x, want, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for x, _, got, ws, s in sides:
            run(x, got, ws, s)
    torch.cuda.synchronize()
    for _, want, got, _, _ in sides:
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@gpu
def test_memory_for_a_side_stream_is_its_own():
    """Scratch and outputs made for a call on another stream are not blocks that
    the current stream freed, whose earlier work may still be writing them."""
    from streaming_attention_block_gb300 import _abi

    s, n = torch.cuda.Stream(), 5 << 20
    like = torch.empty((1, 4096, 5, 128), dtype=torch.bfloat16, device="cuda")  # n bytes
    for make in (lambda st: _abi._scratch(n, like, st), lambda st: _abi._output(like, st)):
        for stream in (s, s.cuda_stream):
            mem = torch.empty(n, dtype=torch.uint8, device="cuda")
            freed = mem.data_ptr()
            del mem
            assert make(None).data_ptr() == freed  # the current stream's calls may reuse it at once
            assert make(stream).data_ptr() != freed
    mem = torch.empty(n, dtype=torch.uint8, device="cuda")
    freed = mem.data_ptr()
    del mem
    with torch.cuda.stream(s):  # handle 0 is the default stream
        assert torch.cuda.default_stream().cuda_stream == 0 and _abi._scratch(n, like, 0).data_ptr() == freed
        assert _abi._scratch(n, like, None).data_ptr() != freed
    state = sab.DecayState(torch.tensor([-0.1, -0.2], device="cuda"), 1, 128)
    other = sab.DecayState(state.log_decay, 1, 128)
    q, k, v = (_randn((1, 700, 2, 128), 200 + i) for i in range(3))
    s.wait_stream(torch.cuda.current_stream())
    a, b = state.attention(q, k, v), other.attention(q, k, v, stream=s)
    c, d = state.step(q[:, 0], k[:, 0], v[:, 0]), other.step(q[:, 0], k[:, 0], v[:, 0], stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(c, d) and torch.equal(state.state, other.state)


@gpu
@pytest.mark.skipif("SAB_LIBRARY" in os.environ, reason="the library is chosen by the caller")
def test_debug_build_agrees():
    """Small cases with the debug library (its index checks on) in a child process."""
    from streaming_attention_block_gb300.build import DEBUG_LIB, build

    build(debug_bounds=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k",
                        "test_forward or test_backward or test_strided_rows or 1-12 or test_special_values",
                        os.path.join(here, "test_gpu_decay.py"), os.path.join(here, "test_gpu_rotary.py")],
                       cwd=os.path.dirname(here), env=dict(os.environ, SAB_LIBRARY=DEBUG_LIB), capture_output=True,
                       text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-15:])
    assert r.returncode == 0 and " passed" in tail, tail


@gpu
def test_same_bits_every_time():
    B, L, H, D = 3, 1100, 2, 64
    x = [_randn((B, L, H, D), 140 + i) for i in range(4)]
    ld = torch.tensor([-0.01, 0.0], device="cuda")
    first = None
    for _ in range(4):
        O, S = _forward(x[0], x[1], x[2], ld, 0.1)
        g = [torch.empty_like(O) for _ in range(3)]
        sab.decay_attention_backward(*x, ld, 0.1, *g)
        now = [O, S, *g]
        if first is None:
            first = [t.clone() for t in now]
        for p, q in zip(now, first):
            assert torch.equal(p, q)


@gpu
def test_more_than_2_to_31_elements():
    """The tail of a sequence whose tensors pass 2^31 elements: with this decay
    nothing older than 64 tokens reaches the last ones (e^-64 ~ 2^-92)."""
    B, L, H, D = 1, 360000, 48, 128
    x = torch.empty((B, L, H, D), dtype=torch.bfloat16, device="cuda")
    x.view(-1)[: 1 << 20] = _randn((1 << 20,), 1)
    n = 1 << 20
    flat = x.view(-1)
    while n < flat.numel():  # repeat the block (its length is no multiple of a token)
        m = min(n, flat.numel() - n)
        flat[n:n + m] = flat[:m]
        n += m
    k, v = x.roll(7, 3), x
    ld = torch.full((H,), -1.0, device="cuda")
    O = torch.empty_like(x)
    sab.decay_attention(x, k, v, ld, 0.1, O)
    t = slice(L - 130, L)
    o, _, oa, _ = OD.decay_attention(_n(x[:, t]), _n(k[:, t]), _n(v[:, t]), _n(ld), 0.1)
    _check(O[:, L - 60:], o[:, 70:], oa[:, 70:], "tail")


def test_refusals_before_any_cuda_call():
    lib = sab.library()
    p = [ctypes.c_void_p(4096 * (i + 1)) for i in range(12)]
    odd16, odd4 = ctypes.c_void_p(4104), ctypes.c_void_p(4098)

    def fwd(Q=p[0], K=p[1], V=p[2], ld=p[3], n=None, S=None, B=1, L=64, H=1, D=64, sc=0.1, O=p[4], So=None):
        return lib.sab_decay_attention(Q, K, V, ld, n, S, B, L, H, D, sc, O, So, None, 0, None)

    def step(Q=p[0], K=p[1], V=p[2], ld=p[3], n=None, S=p[5], B=1, H=1, D=64, sc=0.1, O=p[4], So=p[6]):
        return lib.sab_decay_attention_step(Q, K, V, ld, n, S, B, H, D, sc, O, So, None)

    def bwd(Q=p[0], K=p[1], V=p[2], dO=p[3], ld=p[4], n=None, S=None, dS=None, B=1, L=64, H=1, D=64, sc=0.1, dQ=p[5],
            dK=p[6], dV=p[7], dSi=None):
        return lib.sab_decay_attention_backward(Q, K, V, dO, ld, n, S, dS, B, L, H, D, sc, dQ, dK, dV, dSi, None, 0, None)

    shapes = [dict(B=0), dict(H=0), dict(D=96), dict(D=0), dict(B=1 << 20, H=1 << 20), dict(sc=0.0), dict(sc=-1.0),
              dict(sc=float("nan")), dict(sc=float("inf"))]
    ptrs = [dict(Q=None), dict(K=None), dict(V=odd16), dict(ld=None), dict(ld=odd4), dict(n=odd4), dict(S=odd16)]
    for kw in shapes + ptrs + [dict(L=0), dict(L=(1 << 30) + 1), dict(O=None), dict(O=odd16), dict(So=odd16),
                               dict(O=p[0]), dict(O=p[1]), dict(O=p[2])]:
        assert fwd(**kw) == 1, kw
    for kw in shapes + ptrs + [dict(O=None), dict(So=None), dict(So=odd16), dict(O=p[0])]:
        assert step(**kw) == 1, kw
    for kw in shapes + ptrs + [dict(dO=None), dict(dQ=None), dict(dK=odd16), dict(dV=p[0]), dict(dQ=p[3]), dict(dK=p[5]),
                               dict(dS=odd16), dict(dSi=odd16), dict(S=p[8], dSi=p[8])]:
        assert bwd(**kw) == 1, kw


def test_python_refusals():
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sab.decay_attention(x, x, x, torch.zeros(2), 0.1, x, workspace=torch.empty(0))
    with pytest.raises(ValueError):
        sab.DecayState(torch.zeros((2, 2)), 1, 64)
