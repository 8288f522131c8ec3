"""The cuts of the vocabulary's gradient products (csrc/vocab_pieces.hpp, csrc/gemm_rounds.hpp), asked of the code itself (plain
C++, compiled here for the host): the cases that the GPU tests run take the paths they are there for."""

import ctypes
import os
import shutil
import subprocess

import pytest

import fp8_precision_numerics_amd as fm
import vocab_product_cases

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_numerics_amd", "csrc")
SHIM = """#include "vocab_pieces.hpp"
using namespace fp8mi;
// columns of a piece, rows of dx's first launch, columns of dw's, parts of dx's K
extern "C" void plan(int64_t m, int64_t v, int64_t k, size_t bytes, int fp8, int64_t* out) {
  const int64_t p = grad_piece(m, v, k, bytes, fp8 != 0, fp8 != 0, 256);
  const size_t left = bytes - (size_t)grad_bytes(m, v, k, p);
  out[0] = p;
  out[1] = plan_rounds(k, m, p, fp8 != 0, left, 256).first;
  out[2] = plan_rounds(k, p, m, fp8 != 0, left, 256).first;
  out[3] = choose_tile(out[1], k, p, fp8 != 0, left, 256).split;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("products")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"), "-o", str(d / "shim.so")],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("case", vocab_product_cases.CUT)
@pytest.mark.parametrize("fp8", [0, 1])
def test_the_tested_products_are_cut(lib, case, fp8):
    pieces, *want = vocab_product_cases.CUT[case]
    out = (ctypes.c_int64 * 4)()
    lib.plan(*case, fm.vocab_workspace_bytes(*case, pieces), fp8, out)
    assert list(out)[:3] == want


@pytest.mark.parametrize("case", vocab_product_cases.SPLIT)
@pytest.mark.parametrize("fp8", [0, 1])
def test_the_tested_pieces_are_split(lib, case, fp8):
    size, P, parts = vocab_product_cases.SPLIT[case]
    out = (ctypes.c_int64 * 4)()
    lib.plan(*case, size, fp8, out)
    assert out[0] == P < case[1] and out[1] == case[0] and out[3] == parts, list(out)


def test_either_gradient_is_cut_in_some_case():
    """dx with pieces before it to add to, and dw."""
    assert any(dx < M and P < V and -(-V // P) > 1 for (M, V, K), (_, P, dx, dw) in vocab_product_cases.CUT.items())
    assert any(dw < P for _, P, dx, dw in vocab_product_cases.CUT.values())
