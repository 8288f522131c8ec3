"""The tile shape and split of K that csrc/gemm_shape.hpp chooses, asked of the code itself (plain C++, compiled here
for the host): the products that the GPU tests run do select the kernels they are there for."""

import ctypes
import os
import shutil
import subprocess

import pytest

import tile_cases

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_numerics_amd", "csrc")
SHIM = """#include "gemm_shape.hpp"
extern "C" void choose(int64_t m, int64_t brows, int64_t k, int fp8_cores, size_t bytes, int64_t cus, int* out) {
  const fp8mi::TileChoice c = fp8mi::choose_tile(m, brows, k, fp8_cores != 0, bytes, cus);
  out[0] = c.shape;
  out[1] = c.split;
}
extern "C" int step(void) { return fp8mi::kShapeStep; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("shape")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.choose.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_size_t, ctypes.c_int64, ctypes.c_void_p]
    return lib


def choice(lib, m, brows, k, fp8_cores, workspace=0, cus=256):
    out = (ctypes.c_int * 2)()
    lib.choose(m, brows, k, fp8_cores, workspace, cus, out)
    return tuple(out)


PLAIN = {**tile_cases.PLAIN, **tile_cases.PLAIN_BT, **tile_cases.LARGEST_K, **tile_cases.LARGEST_KN_BT}


@pytest.mark.parametrize("case", PLAIN)
@pytest.mark.parametrize("fp8_cores", [0, 1])
def test_plain_products_select_their_tiles(lib, case, fp8_cores):
    assert choice(lib, *case, fp8_cores) == (PLAIN[case][fp8_cores], 1)


def test_every_shape_is_tested_in_every_layout():
    for cases in (tile_cases.PLAIN, tile_cases.PLAIN_BT):
        for fp8_cores in (0, 1):
            assert {s[fp8_cores] for s in cases.values()} == {0, 1, 2, 3}
    assert all(n % 16 == 0 for _, n, _ in {**tile_cases.PLAIN_BT, **tile_cases.LARGEST_KN_BT})


def test_the_step_is_the_kernels(lib):
    with open(os.path.join(CSRC, "gemm_tile.hpp")) as f:
        assert f"constexpr int kBK = {lib.step()};" in f.read()


@pytest.mark.parametrize("case", tile_cases.EPILOGUE)
@pytest.mark.parametrize("fp8_cores", [0, 1])
def test_products_with_an_epilogue_select_their_tiles(lib, case, fp8_cores):
    assert choice(lib, *case, fp8_cores, tile_cases.WORKSPACE) == tile_cases.EPILOGUE[case][fp8_cores]


def test_every_shape_is_tested_whole_and_split():
    for fp8_cores in (0, 1):
        seen = {(shape, split > 1) for shape, split in (v[fp8_cores] for v in tile_cases.EPILOGUE.values())}
        assert {(0, False), (0, True), (1, False), (1, True), (2, True), (3, True)} <= seen


@pytest.mark.parametrize("fp8_cores", [0, 1])
def test_a_split_fits_its_workspace_and_leaves_no_part_empty(lib, fp8_cores):
    for m, brows, k in list(tile_cases.EPILOGUE) + [(17, 16, 16), (64, 4096, 16384), (24, 4096, 16384), (500, 4096, 16384)]:
        for workspace in (0, 15, m * brows * 4, 2 * m * brows * 4 - 1, 2 * m * brows * 4, 5 * m * brows * 4, 1 << 30):
            shape, split = choice(lib, m, brows, k, fp8_cores, workspace)
            assert 0 <= shape <= 3 and 1 <= split <= max(1, -(-k // 128))
            assert split == 1 or split * m * brows * 4 <= workspace
