"""Infinite elements of a decay-attention state on the GPU: S_t = g S_{t-1} +
k v^T keeps an infinity infinite as long as g is not 0 in fp32, in every form
of the operator, and no other element of the state or output notices."""

import pytest
import torch

import streaming_attention_block_gb300 as sab

pytestmark = pytest.mark.gpu

# to g = 4e-40, which fp32 still holds; over a tile of tokens all but three are 0
LD = [0.0, -1e-4, -0.02, -0.4, -0.7, -4.0, -90.0]
INF = float("inf")
# single tokens, short runs, whole sequences (CTAs fill the SMs), segments
FORMS = [("step", 3, 1, None), ("short", 2, 9, None), ("whole", 20, 200, None), ("ragged", 20, 300, True),
         ("segments", 1, 1500, None), ("ragged_segments", 2, 1100, True)]


def _randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g).to(dtype)
    return torch.where(x == 0, torch.ones_like(x), x).cuda()  # 0 times infinity is no number


def _lens(B, L, ragged):
    if not ragged:
        return None, [L] * B
    n = [(L * (37 * b % 100 + 1)) // 100 for b in range(B)]
    n[-1] = L - 3
    return torch.tensor(n, dtype=torch.int32, device="cuda"), n


def _both(shape, seed):
    """A state with an infinity of each sign in every head, and with 0 there."""
    S = _randn(shape, seed, torch.float32)
    S[..., 3, 5] = S[..., 10, 20] = 0.0
    T = S.clone()
    T[..., 3, 5], T[..., 10, 20] = INF, -INF
    return S, T


def _state_as(got, plain, what):
    assert bool((got[..., 3, 5] == INF).all()) and bool((got[..., 10, 20] == -INF).all()), what
    got = got.clone()
    got[..., 3, 5], got[..., 10, 20] = plain[..., 3, 5], plain[..., 10, 20]
    assert torch.equal(got, plain), what


def _rows_as(got, plain, lens, places, what):
    """Columns c of the live rows are infinite with the sign of x (times s)."""
    want = plain.float()
    for c, x, s in places:
        want[..., c] = torch.sign(x.float()) * s * INF
    for b, n in enumerate(lens):
        assert torch.equal(got[b, :n].float(), want[b, :n]), (what, b)
        assert not bool(got[b, n:].any()), (what, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=[f[0] for f in FORMS])
def test_infinities_stay(form, D):
    name, B, L, ragged = form
    H = len(LD)
    ld = torch.tensor(LD, device="cuda")
    q, k, v = (_randn((B, L, H, D), 10 + i) for i in range(3))
    dl, lens = _lens(B, L, ragged)
    S, T = _both((B, H, D, D), 20)
    res = []
    for state in (S, T):
        O, out = torch.empty_like(q), torch.empty_like(S)
        if name == "step":
            sab.decay_attention_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), ld, 0.1, state,
                                     out, O[:, 0])
        else:
            sab.decay_attention(q, k, v, ld, 0.1, O, state_in=state, state_out=out, seq_len=dl)
        res.append((O, out))
    (O, out), (O2, out2) = res
    _state_as(out2, out, "state")
    _rows_as(O2, O, lens, [(5, q[..., 3], 1), (20, q[..., 10], -1)], "O")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", FORMS[1:], ids=[f[0] for f in FORMS[1:]])
def test_infinities_stay_in_the_gradients(form, D):
    _, B, L, ragged = form
    H = len(LD)
    ld = torch.tensor(LD, device="cuda")
    q, k, v, do = (_randn((B, L, H, D), 30 + i) for i in range(4))
    dl, lens = _lens(B, L, ragged)
    S, T = _both((B, H, D, D), 40)
    R, U = _both((B, H, D, D), 41)
    res = []
    for state, dstate in ((S, R), (T, U)):
        g, d_in = [torch.empty_like(q) for _ in range(3)], torch.empty_like(S)
        sab.decay_attention_backward(q, k, v, do, ld, 0.1, *g, state_in=state, d_state_out=dstate, d_state_in=d_in,
                                     seq_len=dl)
        res.append(g + [d_in])
    (dq, dk, dv, d_in), (dq2, dk2, dv2, d_in2) = res
    _state_as(d_in2, d_in, "d_state_in")
    _rows_as(dq2, dq, lens, [(3, do[..., 5], 1), (10, do[..., 20], -1)], "dQ")
    _rows_as(dk2, dk, lens, [(3, v[..., 5], 1), (10, v[..., 20], -1)], "dK")
    _rows_as(dv2, dv, lens, [(5, k[..., 3], 1), (20, k[..., 10], -1)], "dV")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [9, 300])
def test_huge_finite_elements_still_decay(D, L):
    """A huge finite element is gone once its decay is below fp32's range:
    at most 2^-148 of it is left (1e-6)."""
    ld = torch.tensor([-90.0, -20.0], device="cuda")
    q, k, v = (_randn((1, L, 2, D), 50 + i) for i in range(3))
    S = torch.zeros((1, 2, D, D), device="cuda")
    T = S.clone()
    T[..., 3, 5], T[..., 10, 20] = 5e37, -5e37
    res = []
    for state in (S, T):
        O, out = torch.empty_like(q), torch.empty_like(S)
        sab.decay_attention(q, k, v, ld, 0.1, O, state_in=state, state_out=out)
        res.append((O[:, 8:].float(), out))  # e^-180 after nine tokens
    (O, out), (O2, out2) = res
    assert bool(((out - out2).abs() <= 1e-6).all())
    # scores of up to 100 times this, one rounding of the bf16 outputs
    assert bool(((O - O2).abs() <= 1e-5 + 2.0 ** -7 * O.abs()).all())
