"""Norm and cross attention, each call right behind the one that writes what it
reads: every kernel of the library starts ahead of the end of the one before it."""

import glob
import os
import re

import pytest
import torch

import streaming_attention_block_gb300 as sab

CSRC = os.path.join(os.path.dirname(sab.__file__), "csrc")


def test_nothing_is_read_on_the_read_only_path():
    """That path is for data that no kernel writes while the reader runs, which
    a reader that starts early cannot promise."""
    files = glob.glob(os.path.join(CSRC, "cross_*")) + [os.path.join(CSRC, "layer_norm.cu")]
    assert len(files) == 4
    for f in files:
        with open(f) as src:
            assert not re.findall(r"__ldg\b|\.global\.nc\b|__restrict__", src.read()), f


@pytest.mark.gpu
def test_a_chain_without_pauses_gives_the_bits_of_one_with_them():
    """Moments, LSE, delta, partial sums and weights all change from turn to turn and
    are read by the next kernel; one workspace for all turns."""
    B, Lq, Lk, H, Hk, D = 3, 500, 300, 8, 4, 64
    C, turns = H * D, 12
    g = torch.Generator().manual_seed(8)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g).to(dtype).cuda()

    x = [rand(B * Lq, C) * (1 + i) + i for i in range(turns)]
    kv = [[rand(B, Lk, Hk, D) for _ in range(2)] for _ in range(turns)]
    do = [rand(B, Lq, H, D) for _ in range(turns)]
    ql = [torch.randint(Lq + 1, (B,), generator=g).int().cuda() for _ in range(turns)]
    kl = [torch.randint(Lk + 1, (B,), generator=g).int().cuda() for _ in range(turns)]
    w0, b0 = rand(C, dtype=torch.float32), rand(C, dtype=torch.float32)
    ws = torch.empty(sab.cross_attention_backward_workspace(B, Lq, Lk, H, Hk, D), dtype=torch.uint8, device="cuda")
    ws_n = torch.empty(sab.layer_norm_backward_workspace(B * Lq, C, B * Lq), dtype=torch.uint8, device="cuda")

    def chain(pause):
        def done():
            if pause:
                torch.cuda.synchronize()

        kept = []
        # the places that every turn writes and the next kernel reads
        q, o, dq, dx, dx2 = (torch.zeros((B * Lq, C), dtype=torch.bfloat16, device="cuda") for _ in range(5))
        mean, rstd = (torch.zeros(B * Lq, device="cuda") for _ in range(2))
        w, b, dw, db = w0.clone(), b0.clone(), torch.zeros(C, device="cuda"), torch.zeros(C, device="cuda")
        lse = torch.zeros((B, H, Lq), device="cuda")
        dk, dv = (torch.zeros((B, Lk, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for i in range(turns):
            k, v = kv[i]
            q4, o4, dq4 = (t.view(B, Lq, H, D) for t in (q, o, dq))
            sab.layer_norm(x[i], w, b, 1e-6, q, mean, rstd)
            done()
            sab.cross_attention(q4, k, v, 0.125, o4, lse, q_len=ql[i], kv_len=kl[i])
            done()
            sab.cross_attention_backward(q4, k, v, o4, do[i], lse, 0.125, dq4, dk, dv, q_len=ql[i], kv_len=kl[i],
                                         workspace=ws)
            done()
            # dw and db are the next norm's weight and bias
            sab.layer_norm_backward(x[i], dq, w, mean, rstd, dx, dw, db, workspace=ws_n)
            done()
            sab.layer_norm(x[i], dw, db, 1e-6, dx2, mean, rstd, weight_offset=1.0)
            done()
            kept.append([t.clone() for t in (q, o, lse, dq, dk, dv, dx, dx2, mean, rstd, dw, db)])
            done()
            w, dw, b, db = dw, w, db, b
        torch.cuda.synchronize()
        return kept

    ref = chain(True)
    for _ in range(5):
        for i, (a, b) in enumerate(zip(ref, chain(False))):
            assert all(torch.equal(s, t) for s, t in zip(a, b)), i
    assert sab.get_last_device_error() == 0
