"""The cut of a product into whole rounds of compute units and a rest (csrc/gemm_rounds.hpp), asked of the code itself
(plain C++, compiled here for the host): the losses that the GPU tests run select the kernels they are there for."""

import ctypes
import os
import shutil
import subprocess

import pytest

import vocab_cases

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_numerics_amd", "csrc")
SHIM = """#include "gemm_rounds.hpp"
extern "C" int64_t plan(int64_t fixed, int64_t free_, int64_t k, int fp8_cores, size_t bytes, int64_t cus, double* us) {
  const fp8mi::Rounds r = fp8mi::plan_rounds(fixed, free_, k, fp8_cores != 0, bytes, cus);
  *us = r.us;
  return r.first;
}
extern "C" int shape(int64_t m, int64_t brows, int64_t k, int fp8_cores, int64_t cus, double* us) {
  const fp8mi::TileChoice c = fp8mi::choose_tile(m, brows, k, fp8_cores != 0, 0, cus);
  *us = c.us;
  return c.shape;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("rounds")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"), "-o", str(d / "shim.so")],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_size_t, ctypes.c_int64, ctypes.c_void_p]
    lib.plan.restype = ctypes.c_int64
    lib.shape.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]
    return lib


def plan(lib, fixed, free, k, fp8, workspace=0, cus=256):
    us = ctypes.c_double()
    return lib.plan(fixed, free, k, fp8, workspace, cus, ctypes.byref(us)), us.value


def shape(lib, m, n, k, fp8, cus=256):
    us = ctypes.c_double()
    return lib.shape(m, n, k, fp8, cus, ctypes.byref(us)), us.value


@pytest.mark.parametrize("case", vocab_cases.LOGITS)
@pytest.mark.parametrize("fp8", [0, 1])
def test_the_tested_losses_select_their_kernels(lib, case, fp8):
    m, v, k = case
    first, head, rest = vocab_cases.LOGITS[case][fp8]
    assert plan(lib, m, v, k, fp8)[0] == first and shape(lib, m, first, k, fp8)[0] == head
    assert (first == v) == (rest is None)
    if rest is not None:
        assert shape(lib, m, v - first, k, fp8)[0] == rest


def test_every_kernel_of_the_loss_is_tested():
    for fp8 in (0, 1):
        used = {min(s, 2) for c in vocab_cases.LOGITS.values() for s in c[fp8][1:] if s is not None}
        assert used == {0, 1, 2}


@pytest.mark.parametrize("fp8", [0, 1])
def test_a_cut_is_whole_tiles_and_pays(lib, fp8):
    """Over many sizes: the first launch is whole tiles that fit whole rounds, and what is chosen is never estimated slower than one launch."""
    for m in (17, 300, 1003, 2048, 5000, 8192):
        for v in (1000, 5003, 20000, 50021, 131072):
            for k in (64, 1040, 4096):
                for cus in (256, 64):
                    first, us = plan(lib, m, v, k, fp8, 0, cus)
                    whole = shape(lib, m, v, k, fp8, cus)[1]
                    assert 0 < first <= v and us <= whole
                    if first < v:
                        assert first % 256 == 0 and ((m + 255) // 256) * (first // 256) <= ((m + 255) // 256) * ((v + 255) // 256) // cus * cus
                        assert us < 0.97 * whole
                    else:
                        assert us == whole
