"""The operators of a block that reads a text, together as they are used: layer norm
with weights, queries of it over an encoder's states, and a layer norm whose scale
and shift are each chunk's own; forward and backward.

Every operator is held to its own oracle on the inputs that it got from the ones
before, with the tolerances of its own tests."""

import pytest
import torch

import streaming_attention_block_gb300 as sab
from tests import test_gpu_cross, test_gpu_cross_backward, test_gpu_layer_norm

gpu = pytest.mark.gpu
EPS = 1e-6


class Block:
    """x + Wo cross(Wq norm(x), Wkv text), then norm with a scale and shift for
    each `chunk` rows; buffers made once, so that a run can be captured."""

    def __init__(self, B, L, Lk, C, H, Hk, D, chunk, lens):
        g = torch.Generator().manual_seed(B * L + C)

        def rand(*shape, scale=1.0, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()

        f4 = torch.float32
        self.shape, self.scale, self.chunk = (B, L, Lk, C, H, Hk, D), D ** -0.5, chunk
        rows, groups = B * L, -(-B * L // chunk)
        self.w, self.b = 1 + rand(C, scale=0.1, dtype=f4), rand(C, scale=0.1, dtype=f4)
        self.scale2, self.shift2 = rand(groups, C, scale=0.3, dtype=f4), rand(groups, C, scale=0.3, dtype=f4)
        self.wq, self.wo = rand(C, H * D, scale=C ** -0.5), rand(H * D, C, scale=C ** -0.5)
        self.wkv = rand(C, 2 * Hk * D, scale=C ** -0.5)
        self.x, self.text, self.dout = rand(B, L, C), rand(B, Lk, C), rand(B, L, C)
        self.lens = test_gpu_cross._lens(lens)
        e = torch.empty
        self.y, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.mean, self.rstd, self.mean2, self.rstd2 = (e(rows, device="cuda") for _ in range(4))
        self.o, self.lse = e((B, L, H, D), dtype=torch.bfloat16, device="cuda"), e((B, H, L), device="cuda")
        self.dh, self.dx, self.do = torch.empty_like(self.x), torch.empty_like(self.x), torch.empty_like(self.o)
        self.dq, self.dkv = torch.empty_like(self.o), e((B, Lk, 2, Hk, D), dtype=torch.bfloat16, device="cuda")
        self.dw, self.db = torch.empty_like(self.w), torch.empty_like(self.b)
        self.dscale2, self.dshift2 = torch.empty_like(self.scale2), torch.empty_like(self.shift2)
        n = max(sab.cross_attention_backward_workspace(B, L, Lk, H, Hk, D),
                sab.layer_norm_backward_workspace(rows, C, chunk), sab.layer_norm_backward_workspace(rows, C, rows), 256)
        self.ws = e(n, dtype=torch.uint8, device="cuda")

    def forward(self):
        B, L, Lk, C, H, Hk, D = self.shape
        sab.layer_norm(self.x, self.w, self.b, EPS, self.y, self.mean, self.rstd)
        self.q = (self.y @ self.wq).view(B, L, H, D)
        self.kv = (self.text @ self.wkv).view(B, Lk, 2, Hk, D)
        sab.cross_attention(self.q, *self.kv.unbind(2), self.scale, self.o, self.lse, kv_len=self.lens)
        self.h = self.x + self.o.view(B, L, H * D) @ self.wo
        sab.layer_norm(self.h, self.scale2, self.shift2, EPS, self.out, self.mean2, self.rstd2, group_rows=self.chunk,
                       weight_offset=1.0)

    def backward(self):
        B, L, Lk, C, H, Hk, D = self.shape
        sab.layer_norm_backward(self.h, self.dout, self.scale2, self.mean2, self.rstd2, self.dh, self.dscale2,
                                self.dshift2, group_rows=self.chunk, weight_offset=1.0, workspace=self.ws)
        torch.matmul(self.dh.view(-1, C), self.wo.T, out=self.do.view(-1, H * D))
        sab.cross_attention_backward(self.q, *self.kv.unbind(2), self.o, self.do, self.lse, self.scale, self.dq,
                                     *self.dkv.unbind(2), kv_len=self.lens, workspace=self.ws)
        self.dy = self.dq.view(B, L, H * D) @ self.wq.T
        sab.layer_norm_backward(self.x, self.dy, self.w, self.mean, self.rstd, self.dx, self.dw, self.db,
                                workspace=self.ws)

    def results(self):
        return [self.out, self.dh, self.dscale2, self.dshift2, self.dq, self.dkv, self.dx, self.dw, self.db]


CASES = [
    # B, L, Lk, C, H, Hk, D, rows of a chunk, text lengths
    (1, 384, 77, 256, 2, 2, 128, 128, None),
    (2, 300, 130, 192, 6, 2, 64, 100, [130, 45]),
    (3, 65, 512, 512, 4, 4, 128, 65, [1, 0, 512]),
]


@gpu
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case):
    t = Block(*case)
    B, L, Lk, C, H, Hk, D = t.shape
    t.forward()
    t.backward()
    torch.cuda.synchronize()
    assert sab.get_last_device_error() == 0
    norm, rows = test_gpu_layer_norm, B * L
    norm._check_forward(t.x.view(-1, C), t.w[None], t.b[None], t.y.view(-1, C), t.mean, t.rstd, rows, 0.0, "first norm")
    lens = case[-1]
    k, v = t.kv.unbind(2)
    test_gpu_cross._check_forward(t.q, k, v, t.scale, t.o, t.lse, None, lens, "cross attention")
    norm._check_forward(t.h.view(-1, C), t.scale2, t.shift2, t.out.view(-1, C), t.mean2, t.rstd2, t.chunk, 1.0,
                        "second norm")
    norm._check_backward(t.h.view(-1, C), t.dout.view(-1, C), t.scale2, t.mean2, t.rstd2, t.dh.view(-1, C), t.dscale2,
                         t.dshift2, t.chunk, 1.0, "second norm's gradients")
    test_gpu_cross_backward._check(t.q, k, v, t.do, t.scale, (t.dq, *t.dkv.unbind(2)), None, lens, "cross gradients")
    norm._check_backward(t.x.view(-1, C), t.dy.view(-1, C), t.w[None], t.mean, t.rstd, t.dx.view(-1, C), t.dw[None],
                         t.db[None], rows, 0.0, "first norm's gradients")


@gpu
def test_a_captured_step_on_new_inputs():
    """A step captured into a graph beside the eager one; new inputs, equal bits."""
    eager, held = Block(*CASES[1]), Block(*CASES[1])
    for t in (eager, held):
        t.forward()
        t.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.forward()
        held.backward()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for name in ("x", "text", "dout"):
            a = getattr(eager, name)
            a.copy_(torch.randn(a.shape, generator=g, device="cuda"))
            getattr(held, name).copy_(a)
        for r in held.results():
            r.fill_(float("nan"))
        eager.forward()
        eager.backward()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager.results(), held.results()))
