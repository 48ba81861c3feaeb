"""Cross attention and its gradients on the GPU: the error of each tile of 128 tokens
of a head, as a share of that tile's norm.

The bounds of single elements are sums of absolute terms, some times larger than
an error is, so that a few stale rows or a delta slightly off can hide below them.
For inputs of independent signs the errors of roundings add up as squares.  A
rounding to bf16 is spread evenly over its step, at most 2^-7 of the value: a root
mean square of 2^-8 / sqrt(3) of it at most.  O and dV have two, of P and their own;
dQ and dK a third at most, of O in delta, which is part of dP - delta.  So a tile is
off by at most 2^-8 sqrt(2 / 3) and 2^-8 of its norm; with 16 keys or tokens of 64
columns at least, a share of 1 / sqrt(2 x 1024) of that is chance, and six times as
much is allowed."""

import math

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests.test_gpu_cross import BF, _case, _lens

pytestmark = pytest.mark.gpu

CASES = [
    # B, Lq, Lk, H, Hk, D, Bk, q_len, kv_len
    (1, 1536, 512, 4, 4, 128, 1, None, None),
    (6, 3100, 809, 4, 4, 64, 6, None, None),
    (3, 2500, 1100, 6, 2, 128, 3, None, None),
    (1, 9000, 130, 3, 3, 128, 1, None, None),
    (2, 5000, 77, 4, 4, 128, 2, None, None),
    (4, 2047, 333, 12, 4, 64, 1, [2047, 1024, 16, 1500], None),
    (8, 1023, 777, 12, 2, 64, 8, [1023, 900, 16, 128, 129, 500, 0, 1000], [777, 16, 640, 641, 300, 128, 50, 0]),
    (64, 40, 700, 8, 2, 128, 64, None, [16 + 10 * (7 * b % 64) for b in range(64)]),
    (13, 16, 2816, 10, 10, 64, 13, None, None),
]


def _reference(q, k, v, do, scale, q_len, kv_len):
    """(O, dQ, dK, dV) in 64 bits, head by head."""
    B, Lq, H, D = q.shape
    Bk, Lk, Hk, _ = k.shape
    out = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (q, q, k, k)]
    for b in range(B):
        e = b if Bk == B else 0
        m, n = Lq if q_len is None else q_len[b], Lk if kv_len is None else kv_len[e]
        if m == 0 or n == 0:
            continue
        for h in range(H):
            j = h // (H // Hk)
            Q, K, V, G = q[b, :m, h].double(), k[e, :n, j].double(), v[e, :n, j].double(), do[b, :m, h].double()
            p = torch.softmax(scale * Q @ K.T, 1)
            dp = G @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
            out[0][b, :m, h], out[1][b, :m, h] = p @ V, ds @ K
            out[2][e, :n, j] += ds.T @ Q
            out[3][e, :n, j] += p.T @ G
    return out


def _tiles(t, lens):
    """Sums of squares over tiles of 128 tokens of a head, [B, tiles, H], and which have 16 tokens or more."""
    B, L, H, D = t.shape
    n = -(-L // 128)
    x = torch.nn.functional.pad(t.square().sum(3), (0, 0, 0, n * 128 - L)).view(B, n, 128, H).sum(2)
    left = torch.tensor([L] * B if lens is None else lens, device=t.device)[:, None] - 128 * torch.arange(n, device=t.device)
    return x, (left >= 16)[..., None].expand(x.shape)


@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D, Bk, q_len, kv_len", CASES)
def test_errors_of_tiles(B, Lq, Lk, H, Hk, D, Bk, q_len, kv_len):
    q, k, v, do = _case(B, Lq, Lk, H, Hk, D, Bk)
    scale = D ** -0.5
    ref = _reference(q, k, v, do, scale, q_len, kv_len)
    ql, kl = _lens(q_len), _lens(kv_len)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o, dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, q, k, v))
        lse = torch.empty((B, H, Lq), device="cuda")
        flush.fill_(1)  # nothing of the call is left in L2
        sab.cross_attention(q, k, v, scale, o, lse, q_len=ql, kv_len=kl)
        flush.fill_(2)
        sab.cross_attention_backward(q, k, v, o, do, lse, scale, dq, dk, dv, q_len=ql, kv_len=kl)
        for name, got, want, lens in zip(("O", "dQ", "dK", "dV"), (o, dq, dk, dv), ref, (q_len, q_len, kv_len, kv_len)):
            size, full = _tiles(want, lens)
            off, _ = _tiles(got.double() - want, lens)
            assert bool(full.any()) and not bool(off.isnan().any())
            share = torch.where(full & (size > 0), off / size.clamp(min=1e-300), torch.zeros_like(off)).sqrt()
            bound = BF * (math.sqrt(2 / 3) if name in ("O", "dV") else 1.0) * (1 + 6 / math.sqrt(2 * 1024))
            assert share.max().item() <= bound, (name, share.max().item(), bound, share.argmax().item())
    assert sab.get_last_device_error() == 0
