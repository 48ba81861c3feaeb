"""Index checks of the debug build in cross attention and its gradients: the items
of one sequence too many, and one block of the key gradients too many, are left out.

Forged from the host, in a child process with the debug library.  What the forged
indices point at is the test's own (one sequence more in every tensor, a workspace
that is larger than asked for), so nothing could fault without the checks either."""

import os
import subprocess
import sys

import pytest
import torch

import streaming_attention_block_gb300 as sab

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = os.environ.get("SAB_CROSS_BOUNDS_CHILD") == "1"
needs_debug = pytest.mark.skipif(not CHILD, reason="runs in the debug-build child process")
gpu = pytest.mark.gpu

SHAPES = [
    # B, Lq, Lk, H, Hk, D, lengths
    (2, 1, 900, 2, 1, 64, False),      # keys cut among a cluster
    (2, 200, 300, 8, 8, 128, False),   # so too, full tiles
    (2, 130, 100, 40, 40, 64, False),  # a tile an item
    (2, 130, 100, 40, 40, 64, True),
    (2, 20000, 140, 1, 1, 128, False),  # two tiles an item, several items a block
    (3, 20000, 140, 1, 1, 64, True),   # sequences in order: their items are counted from the lengths
]


@gpu
@pytest.mark.skipif(CHILD or "SAB_LIBRARY" in os.environ, reason="runs in the parent process only")
def test_forged_indices_under_debug_build():
    from streaming_attention_block_gb300.build import DEBUG_LIB, build

    build(debug_bounds=True)
    env = dict(os.environ, SAB_LIBRARY=DEBUG_LIB, SAB_CROSS_BOUNDS_CHILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-rs", "-m", "gpu", "-p", "no:cacheprovider",
                        "-k", "left_out", os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-25:])
    assert r.returncode == 0 and " passed" in tail and "skipped" not in tail, tail


@gpu
@needs_debug
@pytest.mark.parametrize("B, Lq, Lk, H, Hk, D, lengths", SHAPES)
@pytest.mark.parametrize("shared", [False, True])
def test_what_is_past_the_last_is_left_out(B, Lq, Lk, H, Hk, D, lengths, shared):
    assert sab.debug_bounds_enabled()
    g = torch.Generator().manual_seed(2)

    def rand(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()

    Bk = 1 if shared else B
    q, do, k, v = rand(B + 1, Lq, H, D), rand(B + 1, Lq, H, D), rand(B + 1, Lk, Hk, D), rand(B + 1, Lk, Hk, D)
    ql = torch.tensor([Lq // 2, Lq, 0, 7], dtype=torch.int32, device="cuda") if lengths else None
    kl = torch.tensor([Lk, Lk // 2, 3, 7], dtype=torch.int32, device="cuda") if lengths else None
    n = sab.cross_attention_backward_workspace(B, Lq, Lk, H, Hk, D, Bk)
    ws = torch.empty(2 * n + (1 << 22), dtype=torch.uint8, device="cuda")

    def call(forge):
        o, dq = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
        dk, dv = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
        lse = torch.full((B + 1, H, Lq), 7.0, device="cuda")
        kw = dict(q_len=None if ql is None else ql[:B], kv_len=None if kl is None else kl[:Bk])
        status = []
        if forge:
            sab.debug_inject_bounds_error(sab.DEBUG_INJECT_CROSS_ITEM)
        sab.cross_attention(q[:B], k[:Bk], v[:Bk], 0.125, o[:B], lse[:B], **kw)
        status.append(sab.get_last_device_error())
        if forge:
            sab.debug_inject_bounds_error(sab.DEBUG_INJECT_CROSS_ITEM)
        sab.cross_attention_backward(q[:B], k[:Bk], v[:Bk], o[:B], do[:B], lse[:B], 0.125, dq[:B], dk[:Bk], dv[:Bk],
                                     workspace=ws, **kw)
        status.append(sab.get_last_device_error())
        return status, (o, lse, dq, dk, dv)

    status, ref = call(False)
    assert status == [0, 0]
    status, out = call(True)
    assert status == [sab.ERR_BOUNDS] * 2
    for a, b, e in zip(out, ref, (B, B, B, Bk, Bk)):
        assert torch.equal(a, b) and bool((a[e:] == 7.0).all())
    assert call(False)[0] == [0, 0]
