"""The norm's scratch decides where its statistics are gathered, not how many workgroups run: with any workspace the
results are the same bits, and the call takes about as long as without one.  The bound on the time is loose (a grid cut
to the slots of a 16-byte workspace, one workgroup for the whole tensor, takes over a hundred times as long)."""

import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device

pytestmark = pytest.mark.gpu


def time_us(call):
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 3 * 1e3)
    return best


@pytest.mark.parametrize("stats", [False, True])
@pytest.mark.parametrize("rows,cols", [(8192, 4096), (8192, 512), (512, 20000)])
def test_a_small_workspace_neither_slows_nor_changes_the_norm(rows, cols, stats):
    announce(f"norm workspace {rows}x{cols} stats={stats}")
    g = torch.Generator(device=device()).manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device=device()).bfloat16()
    w = torch.ones(cols, dtype=torch.bfloat16, device=device())
    scale = torch.full((1,), 150.0, device=device())                       # some values saturate
    ref = None
    for size in (0, 16, 64, 4096, 1 << 20):
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=device()) if size else None
        q = torch.empty((rows, cols), dtype=torch.uint8, device=device())
        amax = torch.full((1,), -1.0, device=device()) if stats else None
        sat = torch.full((1,), 99, dtype=torch.int64, device=device()) if stats else None

        def call():
            fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", scale, q, amax=amax, sat=sat, workspace=ws)

        call()
        torch.cuda.synchronize()
        got = [q] + ([amax, sat] if stats else [])
        us = time_us(call)
        if ref is None:
            ref, base = got, us
            continue
        assert all(torch.equal(a, b) for a, b in zip(ref, got)), size
        assert us < 4 * base + 20, (size, us, base)
