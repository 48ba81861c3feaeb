"""Cross attention over batches of unequal lengths on the GPU: the order of the
sequences (up to 64 of them are sorted), rows that no item covers, and query tiles
that have to be done again.

Tolerances are those of the tests of the two directions; where the oracle would
take too long the formula is written out in 64 bits beside the case."""

import os
import subprocess
import sys

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests.test_gpu_cross import BF, _case, _check_forward, _forward, _lens, _spoil
from tests.test_gpu_cross_backward import _backward, _check

gpu = pytest.mark.gpu


def _lengths(B, L, step, none=()):
    """Lengths spread over [0, L], with empty sequences at `none`."""
    return [0 if b in none else 1 + (step * b + 3) % L for b in range(B)]


MANY = [
    # B, Lq, Lk, H, Hk, D, states shared
    (2, 2600, 300, 6, 2, 64, False),
    (9, 300, 400, 10, 10, 128, False),
    (64, 130, 200, 4, 4, 64, False),
    (64, 40, 150, 12, 4, 128, True),
    (65, 130, 200, 3, 3, 64, False),
    (70, 33, 90, 8, 2, 128, False),
]


@gpu
@pytest.mark.parametrize("which", ["queries", "keys", "both"])
@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D, shared", MANY)
def test_many_items_of_unequal_lengths(B, Lq, Lk, H, Hk, D, shared, which):
    ql = _lengths(B, Lq, 37, (1, B - 1)) if which != "keys" else None
    kl = None if which == "queries" else [Lk - 5] if shared else _lengths(B, Lk, 53, (0, B // 2))
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D, 1 if shared else None)
    for t, n in ((q, ql), (do, ql), (k, kl), (v, kl)):
        _spoil(t, n, float("nan"))
    o, lse = _forward(q, k, v, D ** -0.5, ql, kl)
    grads = _backward(q, k, v, do, D ** -0.5, ql, kl)
    for t in (q, k, v, do):  # the oracle may not read it either
        t.nan_to_num_(0.0)
    _check_forward(q, k, v, D ** -0.5, o, lse, ql, kl, "forward")
    _check(q, k, v, do, D ** -0.5, grads, ql, kl, "backward")


@gpu
def test_no_sequence_has_anything():
    q, k, v, do = _case(4, 6000, 100, 2, 2, 64)
    for ql, kl in (([0] * 4, None), (None, [0] * 4), ([0, 5, 0, 7], [3, 0, 4, 0])):
        o, lse = _forward(q, k, v, 0.1, ql, kl)
        assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
        for g in _backward(q, k, v, do, 0.1, ql, kl):
            assert bool((g == 0).all())


@gpu
@pytest.mark.parametrize("lens", ["all", "some"])
@pytest.mark.parametrize("low", ["every row", "few rows"])
def test_more_tiles_to_be_done_again_than_a_block_remembers(lens, low):
    """Rows whose scores all lie near -120: their sums without a maximum are 0.
    16 keys in 64 sequences of 188 query tiles: some 80 tiles a block."""
    B, Lq, Lk, D = 64, 24000, 16, 64
    g = torch.Generator().manual_seed(5)
    q = (torch.rand((1, Lq, 1, D), generator=g) + 0.5).bfloat16().cuda().repeat(B, 1, 1, 1)
    k = -(torch.rand((B, Lk, 1, D), generator=g) + 0.5).bfloat16().cuda()
    v = torch.randn((B, Lk, 1, D), generator=g).bfloat16().cuda()
    if low == "few rows":
        keep = torch.zeros(Lq, dtype=torch.bool, device="cuda")
        keep[::1000] = True
        q = torch.where(keep.view(1, -1, 1, 1), q, (q * 2.0 ** -8).bfloat16())
    ql = None if lens == "all" else [Lq - 300 * (b % 7) for b in range(B)]
    kl = None if lens == "all" else [16 - b % 3 for b in range(B)]
    scale = 1.9
    o, lse = _forward(q, k, v, scale, ql, kl)
    for b in range(0, B, 9):
        n, m = Lq if ql is None else ql[b], Lk if kl is None else kl[b]
        s = scale * q[b, :n, 0].double() @ k[b, :m, 0].double().T
        size = scale * q[b, :n, 0].double().abs() @ k[b, :m, 0].double().abs().T
        p = torch.softmax(s, 1)
        ref, w = p @ v[b, :m, 0].double(), p @ v[b, :m, 0].double().abs()
        es = D * 2.0 ** -23 * size.amax(1, keepdim=True) + 2.0 ** -20  # a score, its sum in fp32
        err = (o[b, :n, 0].double() - ref).abs()
        assert bool((err <= (BF + 2 * es + 2.0 ** -16) * w + BF * ref.abs()).all()), b
        ref = torch.logsumexp(s, 1)
        tol = es[:, 0] + (Lk / 2 + 16) * 2.0 ** -24 + 2.0 ** -20 * ref.abs()
        assert bool(((lse[b, 0, :n].double() - ref).abs() <= tol).all()), b
        assert bool((o[b, n:] == 0).all()) and bool((lse[b, :, n:] == -float("inf")).all())


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_one_key_has_no_gradient_but_its_value(D, shared):
    """The softmax over one key is 1: dQ and dK are 0, not a rounding."""
    q, k, v, do = _case(3, 200, 1, 6, 2, D, 1 if shared else None)
    dq, dk, dv = _backward(q, k, v, do, 0.3)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    _check(q, k, v, do, 0.3, (dq, dk, dv), None, None, "one key")
    q, k, v, do = _case(3, 200, 140, 6, 2, D, 1 if shared else None)
    lens = [1] if shared else [1, 140, 1]
    dq, dk, dv = _backward(q, k, v, do, 0.3, None, lens)
    for b in ([0, 1, 2] if shared else [0, 2]):
        assert bool((dq[b] == 0).all()) and bool((dk[0 if shared else b] == 0).all())
    _check(q, k, v, do, 0.3, (dq, dk, dv), None, lens, "a length of one")


@gpu
@pytest.mark.parametrize("Lk", [2, 3, 6, 20, 128])
def test_few_keys_and_scores_of_all_sizes(Lk):
    """delta from P and dP; sharp and flat softmaxes, query tiles of several items."""
    for q_scale in (0.0, 1.0, 30.0):
        q, k, v, do = _case(4, 1100, Lk, 10, 2, 64, q_scale=q_scale)
        grads = _backward(q, k, v, do, 0.125, [1100, 3, 0, 700], None)
        for t in (q, do):
            t.nan_to_num_(0.0)
        _check(q, k, v, do, 0.125, grads, [1100, 3, 0, 700], None, f"{Lk} keys, {q_scale}")


@gpu
@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D", [(6, 3100, 809, 4, 4, 64), (3, 2500, 1100, 6, 2, 128),
                                                 (6, 3100, 300, 4, 4, 64), (4, 3000, 100, 4, 4, 128)])
def test_equal_bits_while_copies_hold_up_the_loads(B, Lq, Lk, H, Hk, D):
    """Each wait is for its own copy, however late that one is: calls of a cold
    cache beside copies of another stream give the bits of calls left alone."""
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D)
    o, lse = _forward(q, k, v, 0.1)
    ref = [o, lse, *_backward(q, k, v, do, 0.1)]
    _check_forward(q[:1], k[:1], v[:1], 0.1, o[:1], lse[:1], None, None, "alone")
    _check(q[:1], k[:1], v[:1], do[:1], 0.1, [g[:1] for g in ref[2:]], None, None, "alone")
    out = [torch.empty_like(t) for t in ref]
    ws = torch.empty(sab.cross_attention_backward_workspace(B, Lq, Lk, H, Hk, D), dtype=torch.uint8, device="cuda")
    big = torch.empty((2, 1 << 28), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for i in range(12):
        big[1].fill_(i)  # nothing of the call is left in L2
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(1 + i % 3):
                big[0].copy_(big[1])
        sab.cross_attention(q, k, v, 0.1, *out[:2])
        sab.cross_attention_backward(q, k, v, out[0], do, out[1], 0.1, *out[2:], workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), i


@gpu
def test_lengths_change_between_replays():
    """A captured call reads the lengths of each replay."""
    B, Lq, Lk, H, D = 6, 400, 260, 8, 64
    q, k, v, do = _case(B, Lq, Lk, H, H, D)
    runs = [(_lengths(B, Lq, 61), _lengths(B, Lk, 97, (2,))), (_lengths(B, Lq, 173, (0, 4)), _lengths(B, Lk, 31))]
    ref = [(*_forward(q, k, v, 0.1, *n), *_backward(q, k, v, do, 0.1, *n)) for n in runs]
    ql, kl = _lens([Lq] * B), _lens([Lk] * B)
    out = [torch.empty_like(t) for t in ref[0]]
    ws = torch.empty(sab.cross_attention_backward_workspace(B, Lq, Lk, H, H, D), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sab.cross_attention(q, k, v, 0.1, *out[:2], q_len=ql, kv_len=kl)
        sab.cross_attention_backward(q, k, v, out[0], do, out[1], 0.1, *out[2:], q_len=ql, kv_len=kl, workspace=ws)
    for i in (0, 1, 0):
        ql.copy_(_lens(runs[i][0]))
        kl.copy_(_lens(runs[i][1]))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref[i]))


@gpu
@pytest.mark.skipif("SAB_LIBRARY" in os.environ, reason="the library is chosen by the caller")
def test_debug_build_agrees():
    """Small cases with the debug library (its index checks on) in a child process."""
    from streaming_attention_block_gb300.build import DEBUG_LIB, build

    build(debug_bounds=True)
    here = os.path.dirname(os.path.abspath(__file__))
    names = "unequal or past_them or anything or heads_before or strides"
    files = [os.path.join(here, f) for f in ("test_gpu_cross.py", "test_gpu_cross_backward.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", names,
                        *files, os.path.abspath(__file__)],
                       cwd=os.path.dirname(here), env=dict(os.environ, SAB_LIBRARY=DEBUG_LIB), capture_output=True,
                       text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-15:])
    assert r.returncode == 0 and " passed" in tail, tail
