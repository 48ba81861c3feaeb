"""Returned states of decay attention held to what the library documents: k
enters them with 24 bits, in whole sequences, in segments and reversed in time.

Bounds, from the arithmetic of a state S = g^n S0 + sum_t w_t k_t v_t^T.  w is
an approximate power of two (2^-22 of it) of an fp32 exponent x (2^-23 |x|,
which the power weighs down to 2^-23 in the sum); the fp32 product k w and its
third bf16 part round by 2^-24 each.  A tensor-core accumulator is cut towards
zero at each addition by at most 2^-23 of what it holds, eight times at full
size per 128 tokens; what comes out of it is summed in fp32 registers.
* element: 2^-19 of the same sum over absolute values (2^-22 + 2^-23 + 2^-23 of
  the powers and parts, 8 * 2^-23 of the cuts), and 2^-23 of it for every fp32
  addition and decay (at most one of each per tile and segment);
* norm, of random inputs: 2^-22 of the power, 2^-23 of the parts, 2^-22 of the
  cuts (eight of half an ulp on average, the sum growing to its full size) and
  2^-23 of the fp32 sums' independent roundings: 2^-20 together.
k in two bf16 parts (16 bits) errs by 2^-18.5 of the norm and more."""

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab

gpu = pytest.mark.gpu
LD = [-0.5, -0.02, 0.0, -1e-3, -4.0, -1e-5]
NORM = 2.0 ** -20


def _randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _exact(k, v, ld, S0, n, mul, reverse):
    """(S, the same over absolute values) of one sequence's first n tokens, fp64."""
    t = torch.arange(n, device=k.device, dtype=torch.float64)
    w = mul * torch.exp(ld.double()[:, None] * (t + 1 if reverse else n - 1 - t))  # [H, n]
    kw, vv = (k[:n].double().permute(1, 2, 0) * w[:, None], v[:n].double().transpose(0, 1))
    g = torch.exp(ld.double() * n)[:, None, None]
    return g * S0.double() + kw @ vv, g * S0.double().abs() + kw.abs() @ vv.abs()


def _check(got, ref, A, adds, what):
    err = (got.double() - ref).abs()
    tol = (2.0 ** -19 + adds * 2.0 ** -23) * A + 1e-30
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.2f} of the bound"
    ratio = err.flatten(1).norm(dim=1) / (NORM * ref.flatten(1).norm(dim=1) + 1e-30)
    assert bool((ratio <= 1).all()), f"{what}: norms {[round(x, 3) for x in ratio.tolist()]} of the limit, by head"


CASES = [
    # B, L, H, D, lengths (None: all)
    (2, 128, 6, 128, None),
    (3, 300, 6, 64, (300, 131, 45)),
    (14, 700, 6, 128, None),    # whole sequences
    (14, 700, 6, 64, None),
    (30, 1300, 6, 64, True),    # whole, of unequal lengths
    (1, 1536, 12, 128, None),   # segments of one tile or two
    (2, 2300, 6, 128, (2300, 777)),
    (1, 20011, 3, 64, None),    # many segments
    (1, 30720, 36, 128, None),  # long segments
    (1, 30720, 36, 64, None),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[f"{b}x{l}_h{h}_d{d}{'_ragged' if n else ''}" for b, l, h, d, n in CASES])
def test_states_have_the_documented_accuracy(case):
    B, L, H, D, n = case
    lens = [L] * B if n is None else [max(1, L * (37 * b % 100) // 100) for b in range(B)] if n is True else list(n)
    dl = None if n is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ld = torch.tensor([LD[h % len(LD)] for h in range(H)], device="cuda")
    q, k, v, do = (_randn((B, L, H, D), 300 + i) for i in range(4))
    S, dS = (_randn((B, H, D, D), 310 + i, torch.float32) * 4 for i in range(2))
    O, So, g, d_in = torch.empty_like(q), torch.empty_like(S), [torch.empty_like(q) for _ in range(3)], torch.empty_like(S)
    sab.decay_attention(q, k, v, ld, 0.1, O, state_in=S, state_out=So, seq_len=dl)
    sab.decay_attention_backward(q, k, v, do, ld, 0.1, *g, state_in=S, d_state_out=dS, d_state_in=d_in, seq_len=dl)
    scale = float(np.float32(0.1))
    for b, m in enumerate(lens):
        adds = 2 * ((m + 127) // 128 + 1)
        _check(So[b], *_exact(k[b], v[b], ld, S[b], m, 1.0, False), adds, f"state {b}")
        _check(d_in[b], *_exact(q[b], do[b], ld, dS[b], m, scale, True), adds, f"d_state_in {b}")


def _bf16(x):
    return torch.tensor(x, dtype=torch.float32).bfloat16().double().numpy()


def test_two_parts_of_k_would_not_pass():
    """The limit tells 24 bits of k from 16 (a model in numpy): with two parts
    every head that decays is above it, with three none comes near."""
    rng = np.random.default_rng(1)
    n, D = 700, 64
    k, v = (_bf16(rng.standard_normal((n, D))) for _ in range(2))
    for ld in (-0.5, -0.02, -1e-3, -1e-5):
        kw = (k * np.exp(ld * (n - 1 - np.arange(n)))[:, None]).astype(np.float32).astype(np.float64)
        ref = kw.T @ v
        parts, rest = np.zeros_like(kw), kw
        for terms in (1, 2, 3):
            part = _bf16(rest)
            parts, rest = parts + part, rest - part
            err = np.linalg.norm(parts.T @ v - ref) / np.linalg.norm(ref)
            assert (err > NORM) if terms < 3 else (err < NORM / 16), (ld, terms, err)


# a decay whose rounding to fp32 is off by nearly half a step, in both directions
def _uneven(near):
    xs = (np.float32(near) * (1 + np.arange(256) / 1024)).astype(np.float32)
    off = np.exp(xs.astype(np.float64)).astype(np.float32).astype(np.float64) / np.exp(xs.astype(np.float64)) - 1
    return [float(xs[np.argmax(off)]), float(xs[np.argmin(off)])]


STEPS = 4096
# Each token rounds the state twice, by at most 2^-24 of it; independent, so
# 2^-24 / sqrt(3) in the norm and sqrt(2 * 4096) times that after all: 2^-18.3.
# (What came later is less decayed, and less rounded.)
DRIFT = 2.0 ** -17


@gpu
def test_thousands_of_steps_do_not_drift():
    ld = torch.tensor(_uneven(-1e-4) + _uneven(-2e-4), device="cuda")
    H, D = 4, 64
    q, k, v = (_randn((STEPS, 1, H, D), 320 + i) for i in range(3))
    S0 = _randn((1, H, D, D), 330, torch.float32) * 64
    S, O = S0.clone(), torch.empty_like(q[0])
    for t in range(STEPS):
        sab.decay_attention_step(q[t], k[t], v[t], ld, 0.1, S, S, O)
    ref = _exact(k[:, 0], v[:, 0], ld, S0[0], STEPS, 1.0, False)[0]
    ratio = (S[0].double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert bool((ratio <= DRIFT).all()), ratio.tolist()


def test_plain_products_would_drift():
    """The limit tells a decay held in two numbers from its fp32 value alone."""
    rng = np.random.default_rng(2)
    for ld in _uneven(-1e-4) + _uneven(-2e-4):
        g = np.exp(np.float64(np.float32(ld)))
        hi = np.float32(g)
        lo = np.float32(g - np.float64(hi))
        exact = rng.standard_normal(64) * 64
        plain = both = exact.astype(np.float32)
        exact = plain.astype(np.float64)
        for kv in _bf16(rng.standard_normal((STEPS, 64))) * _bf16(rng.standard_normal((STEPS, 1))):
            exact = g * exact + kv
            plain = (plain.astype(np.float64) * hi + 0.0).astype(np.float32)
            plain = (plain.astype(np.float64) + kv).astype(np.float32)
            rest = (both * lo).astype(np.float64)
            both = (both.astype(np.float64) * hi + rest).astype(np.float32)
            both = (both.astype(np.float64) + kv).astype(np.float32)
        off = [np.linalg.norm(x - exact) / np.linalg.norm(exact) for x in (plain, both)]
        assert off[0] > 2 * DRIFT and off[1] < DRIFT, (ld, off)
