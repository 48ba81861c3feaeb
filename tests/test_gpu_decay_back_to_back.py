"""Decay attention calls of every tile count, one behind the other without a
wait: blocks follow others on the same SM and in the same shared memory, and
each has to give what it gives alone."""

import pytest
import torch

import streaming_attention_block_gb300 as sab

pytestmark = pytest.mark.gpu


def _randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("B,H", [(1, 2), (20, 8)], ids=["segments", "whole"])
def test_calls_back_to_back(B, H):
    ld = torch.tensor([-0.01 * h for h in range(H)], device="cuda")
    jobs = []
    for tiles in range(1, 9):
        for D in (64, 128):
            L = 128 * tiles - (17 if tiles % 2 else 0)
            x = [_randn((B, L, H, D), 400 + 10 * tiles + i) for i in range(4)]
            S = _randn((B, H, D, D), 390, torch.float32)
            outs = [[torch.zeros_like(x[0]) for _ in range(5)] + [torch.zeros_like(S) for _ in range(2)] for _ in range(2)]
            ws = [torch.empty(max(256, n), dtype=torch.uint8, device="cuda") for n in
                  (sab.decay_attention_workspace(B, L, H, D), sab.decay_attention_backward_workspace(B, L, H, D))]
            jobs.append((x, S, outs, ws))

    def run(x, S, out, ws):
        sab.decay_attention(*x[:3], ld, 0.1, out[0], state_in=S, state_out=out[5], workspace=ws[0])
        sab.decay_attention(*x[:3], ld, 0.1, out[4], state_in=S, workspace=ws[0])
        sab.decay_attention_backward(*x, ld, 0.1, *out[1:4], state_in=S, d_state_out=S, d_state_in=out[6], workspace=ws[1])

    for x, S, outs, ws in jobs:
        run(x, S, outs[0], ws)
        torch.cuda.synchronize()
    for _ in range(3):
        for x, S, outs, ws in jobs:
            run(x, S, outs[1], ws)
    torch.cuda.synchronize()
    for i, (x, S, outs, ws) in enumerate(jobs):
        for a, b in zip(*outs):
            assert torch.equal(a, b), i
