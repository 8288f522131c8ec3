"""Marshalling of tensors into the entry points: what it takes, what it refuses, and where the call goes."""

import threading

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from fp8_precision_numerics_amd import _binding as binding


def module():
    return binding._MODULE or binding._load_module()


@pytest.mark.parametrize("name", ["gemm", "gated", "fused", "norm", "norm_blocks", "norm_back", "act_back", "gated_back"])
def test_a_wrong_number_of_arguments_is_a_type_error(name):
    with pytest.raises(TypeError):
        getattr(module(), name)(0, 0)
    with pytest.raises(TypeError):
        getattr(module(), name)(*[None] * 40)


@pytest.mark.parametrize("x,error", [(None, ValueError), (3, TypeError), ("x", TypeError), (np.zeros((2, 2)), TypeError),
                                     (torch.zeros(2, 2), ValueError)])
def test_a_first_operand_that_is_no_gpu_tensor(x, error):
    with pytest.raises(error):
        fm.fp8_rmsnorm_quantize(x, None, 1e-5, "e4m3", None, None)
    with pytest.raises(error):
        fm.fp8_gemm(x, "e4m3", x, "e4m3", None, None, None)


def operands(M=24, N=40, K=64):
    g = torch.Generator().manual_seed(3)
    a = torch.randint(0, 0x70, (M, K), dtype=torch.uint8, generator=g).cuda()
    b = torch.randint(0, 0x70, (N, K), dtype=torch.uint8, generator=g).cuda()
    s = torch.tensor([0.5], device="cuda")
    return a, b, s, torch.full((M, N), -1.0, device="cuda")


@pytest.mark.gpu
def test_codes_as_names_as_ints_and_as_numpy_ints():
    a, b, s, c = operands()
    fm.fp8_gemm(a, "e4m3", b, "e5m2", s, s, c, accum="mfma_fp8")
    for e4, e5, acc in ((0, 1, 1), (np.int64(0), np.int32(1), np.int64(1)), (False, True, True)):
        d = torch.empty_like(c)
        fm.fp8_gemm(a, e4, b, e5, s, s, d, accum=acc)
        assert torch.equal(c, d)
    for bad in (2, -1, "E4M3", 1.5, None, [0], torch.tensor(0)):
        with pytest.raises(ValueError):
            fm.fp8_gemm(a, bad, b, "e4m3", s, s, c)
        with pytest.raises(ValueError):
            fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, c, accum=bad)


@pytest.mark.gpu
def test_refusals_name_the_operand_and_its_shape():
    a, b, s, c = operands()
    with pytest.raises(ValueError, match=r"c must have shape \[24, 40\], got \[40, 24\]"):
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, c.view(40, 24))
    with pytest.raises(TypeError, match="b must be Byte, got Float"):
        fm.fp8_gemm(a, "e4m3", b.float(), "e4m3", s, s, c)
    with pytest.raises(ValueError, match="b must be contiguous"):
        fm.fp8_gemm(a, "e4m3", b.t().contiguous().t(), "e4m3", s, s, c)
    with pytest.raises(ValueError, match="sinv_b is not on the device"):
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s.cpu(), c)
    with pytest.raises(ValueError, match="sinv_a must have 1 element"):
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s.expand(2).contiguous(), s, c)
    with pytest.raises(TypeError):
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, c.half())
    assert (c == -1).all()


@pytest.mark.gpu
def test_streams_as_objects_and_as_handles():
    a, b, s, c = operands()
    fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        d = torch.full_like(c, -1.0)
        side.wait_stream(torch.cuda.current_stream())
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, d, stream=stream)
        side.synchronize()
        assert torch.equal(c, d)
    with torch.cuda.stream(side):
        d = torch.full_like(c, -1.0)
        fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, d)
    side.synchronize()
    assert torch.equal(c, d)


@pytest.mark.gpu
def test_calls_of_several_threads():
    a, b, s, c = operands()
    fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, c)
    out = [torch.full_like(c, -1.0) for _ in range(4)]
    torch.cuda.synchronize()

    def work(d):
        for _ in range(50):
            fm.fp8_gemm(a, "e4m3", b, "e4m3", s, s, d)

    threads = [threading.Thread(target=work, args=(d,)) for d in out]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(c, d) for d in out)
