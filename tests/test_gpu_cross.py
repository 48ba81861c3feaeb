"""Cross attention and its gradients on the GPU against the fp64 oracle
(``oracle/cross.py``), through the C ABI.

Bounds per element, derived from the arithmetic.  A score is a sum of D exact
products in fp32, cut towards zero at worst: e_s = D 2^-23 scale sum |q| |k| +
2^-20 (the exponent's product and exponential, for exponents up to 2^6).
Forward: P is rounded to bf16 (2^-8) before its product, so O is off by at most
(2^-8 + 2 e_s + 2^-16) sum p |v|, and one rounding of |O|.  LSE: e_s and the
additions of the row's sum."""

import ctypes

import numpy as np
import pytest
import torch

import streaming_attention_block_gb300 as sab
from oracle import cross as OC

gpu = pytest.mark.gpu
BF = 2.0 ** -8


def _np(t):
    return t.double().cpu().numpy()


def _rand(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def _case(B, Lq, Lk, H, Hk, D, Bk=None, seed=0, fused=False, q_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    q, do = _rand((B, Lq, H, D), g, q_scale), _rand((B, Lq, H, D), g)
    Bk = Bk or B
    if fused:
        k, v = _rand((Bk, Lk, 2, Hk, D), g).unbind(2)
    else:
        k, v = _rand((Bk, Lk, Hk, D), g), _rand((Bk, Lk, Hk, D), g)
    return q, k, v, do


def _lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def _spoil(t, lens, value):
    """Fill what lies past the lengths."""
    if lens is not None:
        for b, n in enumerate(lens):
            t[b, max(n, 0):] = value


def _check_forward(q, k, v, scale, o, lse, q_len, kv_len, what):
    ref, lse_ref, w, score = OC.forward(_np(q), _np(k), _np(v), scale, q_len, kv_len)
    D, Lk = q.shape[3], k.shape[1]
    es = np.transpose(D * 2.0 ** -23 * score + 2.0 ** -20, (0, 2, 1))[..., None]
    tol = (BF + 2 * es + 2.0 ** -16) * w + BF * np.abs(ref)
    err = np.abs(_np(o) - ref)
    assert np.all(err <= tol), f"{what}: O off by {np.max(err - tol):.3e} at {np.argwhere(~(err <= tol))[:3]}"
    if lse is None:
        return
    got = _np(lse)
    live = np.isfinite(lse_ref)
    assert np.array_equal(live, np.isfinite(got)) and np.all(got[~live] == -np.inf), what
    tol = es[..., 0].transpose(0, 2, 1) + (Lk / 2 + 16) * 2.0 ** -24 + 2.0 ** -20 * np.abs(np.where(live, lse_ref, 0))
    err = np.abs(got[live] - lse_ref[live])
    assert np.all(err <= tol[live]), f"{what}: LSE off by {np.max(err):.3e}"


def _forward(q, k, v, scale, q_len=None, kv_len=None, what="", **kw):
    o = torch.full_like(q, float("nan"))
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), float("nan"), device="cuda")
    sab.cross_attention(q, k, v, scale, o, lse, q_len=_lens(q_len), kv_len=_lens(kv_len), **kw)
    torch.cuda.synchronize()
    assert sab.get_last_device_error() == 0
    return o, lse


SHAPES = [
    # B, Lq, Lk, H, Hk, D, Bk
    (1, 1, 1, 1, 1, 64, 1),
    (1, 1, 1, 1, 1, 128, 1),
    (1, 1, 77, 12, 12, 128, 1),
    (2, 1, 300, 8, 1, 64, 2),
    (3, 1, 1000, 24, 8, 128, 3),
    (1, 1, 8200, 2, 1, 128, 1),
    (2, 3, 64, 6, 2, 128, 2),
    (2, 5, 65, 7, 1, 64, 1),
    (1, 127, 128, 2, 2, 128, 1),
    (1, 128, 129, 2, 2, 64, 1),
    (2, 129, 16, 3, 3, 128, 2),
    (1, 200, 17, 10, 2, 64, 1),
    (2, 333, 257, 12, 3, 128, 1),
    (1, 1000, 512, 4, 2, 128, 1),
    (5, 260, 400, 9, 9, 64, 5),
    (4, 700, 77, 12, 12, 128, 4),
    (3, 2000, 130, 6, 6, 64, 1),
]


@gpu
@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D, Bk", SHAPES)
def test_shapes(B, Lq, Lk, H, Hk, D, Bk):
    q, k, v, _ = _case(B, Lq, Lk, H, Hk, D, Bk, fused=Lk % 2 == 1)
    o, lse = _forward(q, k, v, D ** -0.5)
    _check_forward(q, k, v, D ** -0.5, o, lse, None, None, f"{B} {Lq} {Lk} {H}/{Hk} {D}")


RAGGED = [
    # Lq, Lk, H, Hk, D, q_len, kv_len (None: all; past the ends: clamped)
    (1, 300, 6, 2, 128, None, [0, 1, 16, 129, 300]),
    (1, 2000, 2, 2, 64, [1, 0, 1], [1999, 5, 1024]),
    (40, 80, 3, 1, 128, [40, 0, 1, 39], [80, 80, 0, 63]),
    (300, 260, 4, 4, 64, [300, 129, 128, 1], [65, 260, 64, 200]),
    (500, 140, 24, 8, 64, [7, 500, 400], None),
    (260, 400, 2, 1, 128, None, [-3, 1000, 255]),
    (130, 1000, 1, 1, 128, [130], [897]),
]


@gpu
@pytest.mark.parametrize("Lq, Lk, H, Hk, D, q_len, kv_len", RAGGED)
@pytest.mark.parametrize("junk", [0.0, float("nan"), float("inf")])
def test_lengths_and_what_lies_past_them(Lq, Lk, H, Hk, D, q_len, kv_len, junk):
    B = len(q_len or kv_len)
    q, k, v, _ = _case(B, Lq, Lk, H, Hk, D, fused=Hk == 2)
    _spoil(q, q_len, junk)
    _spoil(k, kv_len, junk)
    _spoil(v, kv_len, junk)
    o, lse = _forward(q, k, v, D ** -0.5, q_len, kv_len)
    for t in (q, k, v):  # the oracle may not read it either
        t.nan_to_num_(0.0, 0.0, 0.0)
    _check_forward(q, k, v, D ** -0.5, o, lse, q_len, kv_len, "ragged")


@gpu
@pytest.mark.parametrize("Lq, H, Hk, D", [(1, 24, 8, 128), (1, 6, 6, 64), (5, 16, 16, 128), (129, 4, 4, 64)])
def test_many_sequences_of_unequal_lengths(Lq, H, Hk, D):
    """Several query tiles a block, of odd and even numbers of key tiles, and none."""
    B, Lk = 64, 900
    lens = [(97 * b) % (Lk + 1) for b in range(B)]
    lens[5] = lens[40] = 0
    lens[7], lens[8], lens[9] = 128, 129, 1
    q, k, v, _ = _case(B, Lq, Lk, H, Hk, D)
    o, lse = _forward(q, k, v, D ** -0.5, None, lens)
    _check_forward(q, k, v, D ** -0.5, o, lse, None, lens, "many")


@gpu
def test_one_length_for_states_that_all_share():
    q, k, v, _ = _case(4, 70, 200, 4, 2, 128, 1)
    o, lse = _forward(q, k, v, 0.1, [70, 3, 0, 50], [150])
    _check_forward(q, k, v, 0.1, o, lse, [70, 3, 0, 50], [150], "shared")


@gpu
@pytest.mark.parametrize("q_scale", [0.0, 20.0, 150.0])
@pytest.mark.parametrize("Lq, Lk", [(130, 500), (1, 3000)])
def test_scores_far_from_the_reference(q_scale, Lq, Lk):
    """Maxima in the hundreds, far below zero, and rising from tile to tile."""
    D = 64
    q, k, v, _ = _case(1, Lq, Lk, 2, 2, D, q_scale=q_scale)
    o, lse = _forward(q, k, v, D ** -0.5)
    _check_forward(q, k, v, D ** -0.5, o, lse, None, None, "random")
    q = q.abs()
    k = (k.abs() * torch.linspace(-2.0, 2.0, Lk, device="cuda").view(1, -1, 1, 1)).bfloat16()
    for kk in (k, k.flip(1).contiguous(), -k.abs()):
        o, lse = _forward(q, kk, v, D ** -0.5)
        _check_forward(q, kk, v, D ** -0.5, o, lse, None, None, "rising, falling, all low")


@gpu
def test_scores_out_of_range_in_more_tiles_than_a_block_remembers():
    """Every third stretch of queries has scores in the hundreds: 0, 1 or all
    tiles of many blocks are done again."""
    H, D, Lk = 1, 64, 40
    Lq = 152 * 2 * 128 * 75 + 77
    q, k, v, _ = _case(1, Lq, Lk, H, H, D)
    for first, last in ((0, Lq // 3), (Lq // 2, Lq // 2 + 1)):
        q[:, first:last] *= 100.0
    o, lse = _forward(q, k, v, 0.5)
    for at in (0, 128 * 64, Lq // 3 - 300, Lq // 2 - 64, Lq - 300):
        part = slice(at, at + 300)
        _check_forward(q[:, part], k, v, 0.5, o[:, part], lse[:, :, part].contiguous(), None, None, f"rows {at}")


@gpu
def test_strides_slices_and_rows_in_between():
    B, Lq, Lk, H, Hk, D = 2, 200, 150, 4, 2, 128
    q, k, v, _ = _case(B, Lq, Lk, H, Hk, D)
    ref, lse = _forward(q, k, v, 0.1)
    wide = torch.full((B, Lq + 3, 3, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :Lq, 1] = q
    kv = torch.full((Lk, B, 2, Hk + 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # tokens outermost
    kv[:, :, 0, :Hk] = k.transpose(0, 1)
    kv[:, :, 1, 1:] = v.transpose(0, 1)
    out = torch.full((B, Lq + 5, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for lq in (Lq, 1):
        sab.cross_attention(wide[:, :lq, 1], kv[:, :, 0, :Hk].transpose(0, 1), kv[:, :, 1, 1:].transpose(0, 1), 0.1,
                            out[:, 2:2 + lq, 1:])
        if lq == Lq:
            assert torch.equal(out[:, 2:2 + Lq, 1:], ref)
            rest = out.clone()
            rest[:, 2:2 + Lq, 1:] = 7.0
            assert bool((rest == 7).all())
        else:
            _check_forward(q[:, :1], k, v, 0.1, out[:, 2:3, 1:], None, None, None, "one token")


def _heads_first(t, fill=None):
    """The same [B, L, H, D] values (or `fill`) with heads before tokens in memory."""
    B, L, H, D = t.shape
    out = torch.empty((B, H, L, D), dtype=t.dtype, device=t.device)
    return (out.copy_(t.transpose(1, 2)) if fill is None else out.fill_(fill)).transpose(1, 2)


@gpu
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [(2, 200, 150, 4, 2, 128), (3, 65, 300, 6, 2, 64), (1, 1, 1000, 4, 4, 128)])
def test_heads_before_tokens(B, Lq, Lk, H, Hk, D):
    q, k, v, _ = _case(B, Lq, Lk, H, Hk, D)
    ref, lse_ref = _forward(q, k, v, 0.1)
    o, lse = _heads_first(q, 7.0), torch.empty_like(lse_ref)
    lens = [Lk] * (B - 1) + [0]
    sab.cross_attention(_heads_first(q), _heads_first(k), _heads_first(v), 0.1, o, lse)
    assert torch.equal(o, ref) and torch.equal(lse, lse_ref)
    ref, lse_ref = _forward(q, k, v, 0.1, None, lens)
    sab.cross_attention(_heads_first(q), k, _heads_first(v), 0.1, o, lse, kv_len=_lens(lens))
    assert torch.equal(o, ref) and torch.equal(lse, lse_ref)


@gpu
def test_a_bad_value_stays_in_its_rows():
    q, k, v, _ = _case(1, 300, 200, 4, 4, 64)
    ref, lse_ref = _forward(q, k, v, 0.125)
    q[0, 7, 2, 3] = float("nan")
    q[0, 200, 0, 0] = float("inf")
    o, lse = _forward(q, k, v, 0.125)
    same = torch.ones((300, 4), dtype=torch.bool, device="cuda")
    same[7, 2] = same[200, 0] = False
    assert torch.equal(o[0][same], ref[0][same]) and torch.equal(lse[0].T[same], lse_ref[0].T[same])
    assert bool(o[0, 7, 2].isnan().all()) and bool(o[0, 200, 0].isnan().any())


@gpu
def test_other_stream_two_at_once_and_graph():
    a = _case(2, 1536, 512, 12, 12, 128)[:3]
    b = _case(3, 1, 900, 8, 2, 64, seed=1)[:3]
    ref = [_forward(*t, 0.1) for t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [(torch.empty_like(t[0]), torch.empty((t[0].shape[0], t[0].shape[2], t[0].shape[1]), device="cuda"))
           for t in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, (o, l), s in zip((a, b), out, streams):
            sab.cross_attention(*t, 0.1, o, l, stream=s)
    torch.cuda.synchronize()
    for (o, l), (ro, rl) in zip(out, ref):
        assert torch.equal(o, ro) and torch.equal(l, rl)
    lens = _lens([900, 900, 900])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sab.cross_attention(*a, 0.1, *out[0])
        sab.cross_attention(*b, 0.1, *out[1], kv_len=lens)
    for n in ([900, 900, 900], [0, 3, 500]):  # lengths are read when it runs
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for o, l in out:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], ref[0][0])
        _check_forward(*b, 0.1, *out[1], None, n, "replayed")


@gpu
def test_rows_past_2_31_elements():
    B, Lq, H, D = 2, (1 << 31) // (8 * 128) // 2 + 100, 8, 128
    k, v = _case(1, 1, 50, 8, 8, 128)[1:3]
    q = torch.zeros((B, Lq, H, D), dtype=torch.bfloat16, device="cuda")
    tail = _rand((1, 64, H, D), torch.Generator().manual_seed(3))
    q[-1:, -64:] = tail
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Lq), device="cuda")
    sab.cross_attention(q, k, v, 0.1, o, lse)
    _check_forward(tail, k, v, 0.1, o[-1:, -64:], lse[-1:, :, -64:].contiguous(), None, None, "far rows")
    _check_forward(q[:1, :64], k, v, 0.1, o[:1, :64], lse[:1, :, :64].contiguous(), None, None, "first rows")


def _desc(**kw):
    d = dict(batch=2, q_tokens=4, kv_batch=2, kv_tokens=8, heads=4, kv_heads=2, head_dim=64)
    d.update(kw)
    return sab.CrossDesc(*(d[n] for n, _ in sab.CrossDesc._fields_))


def _rows(data=4096, batch=1 << 20, token=256, head=0):
    return sab.TokenRows(data, batch, token, head)


SHAPE_REFUSALS = [dict(batch=0), dict(q_tokens=0), dict(kv_tokens=0), dict(heads=0), dict(kv_heads=0), dict(heads=5),
                  dict(kv_batch=3), dict(kv_batch=0), dict(head_dim=32), dict(head_dim=96), dict(head_dim=256),
                  dict(heads=258, kv_heads=2), dict(q_tokens=(1 << 30) + 1), dict(kv_tokens=(1 << 26) + 1),
                  dict(batch=-1, kv_batch=-1), dict(batch=1 << 30, kv_batch=1, heads=2, kv_heads=1)]
ROW_REFUSALS = [dict(data=None), dict(data=4104), dict(token=260), dict(token=120), dict(batch=-8), dict(batch=100),
                dict(token=1 << 39), dict(batch=1 << 39), dict(token=-256), dict(head=-64), dict(head=68),
                dict(head=56), dict(head=1 << 39), dict(head=256), dict(head=320, token=128)]


def test_refusals_before_any_cuda_call():
    lib = sab.library()

    def call(d=_desc(), q=None, k=None, v=None, o=None, ql=None, kl=None, scale=0.1, lse=None):
        r = [_rows(a) if x is None else x for a, x in ((4096, q), (8192, k), (12288, v), (16384, o))]
        p = [ctypes.byref(x) if x != 0 else None for x in r]
        return lib.sab_cross_attention(ctypes.byref(d) if d else None, *p[:3], ql, kl, scale, p[3], lse, None)

    P = ctypes.c_void_p
    assert call(d=None) == 1
    for kw in SHAPE_REFUSALS:
        assert call(d=_desc(**kw)) == 1, kw
    for name in ("q", "k", "v", "o"):
        assert call(**{name: 0}) == 1
        for kw in ROW_REFUSALS:
            assert call(**{name: _rows(**kw)}) == 1, (name, kw)
    bad = [dict(o=_rows(4096)), dict(o=_rows(8192)), dict(o=_rows(12288)), dict(ql=P(4098)), dict(kl=P(4097)),
           dict(lse=P(4104)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
           dict(o=_rows(16384, 512, 256))]  # its sequences on top of each other
    for kw in bad:
        assert call(**kw) == 1, kw


def test_python_refusals():
    q = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sab.cross_attention(q, q, q, 0.1, q)  # not on the GPU
    with pytest.raises(TypeError):
        sab.cross_attention(q[0], q, q, 0.1, q)
    with pytest.raises(ValueError):
        sab.cross_attention(q, torch.zeros((1, 2, 2, 128), dtype=torch.bfloat16), q, 0.1, q)
