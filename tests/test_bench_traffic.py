"""bench.py reports counter-measured HBM traffic of the FC1 GEMM only for the code that was measured: the guard covers
every file that the GEMM is compiled from, comments aside, and the committed figures belong to the present code."""

import os
import re
import shutil
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_precision_numerics_amd", "csrc")
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def included(name, seen):
    if name not in seen:
        seen.add(name)
        with open(os.path.join(CSRC, name)) as f:
            for inner in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                included(inner, seen)
    return seen


def test_every_source_of_the_gemm_is_hashed():
    assert included("gemm.hip", set()) == set(bench.GEMM_SOURCES)


def test_the_figures_belong_to_the_present_code():
    """A change of the GEMM's code asks for new counter runs (profiles/gemm_fc1_8192x16384x4096_hbm_traffic.md says which)."""
    for accum in ("exact", "mfma_fp8"):
        assert bench.gemm_traffic(accum) == sum(bench.GEMM_TRAFFIC[accum].values())


def test_code_counts_and_comments_do_not(tmp_path):
    for name in bench.GEMM_SOURCES:
        shutil.copy(os.path.join(CSRC, name), tmp_path / name)
    assert bench.gemm_sources_sha256(str(tmp_path)) == bench.GEMM_TRAFFIC_SHA256
    path = tmp_path / "stats.hpp"
    text = path.read_text()
    path.write_text("// another comment\n\n" + text + "// and one more\n")
    assert bench.gemm_sources_sha256(str(tmp_path)) == bench.GEMM_TRAFFIC_SHA256
    path.write_text(text + "constexpr int kOther = 1;\n")
    assert bench.gemm_sources_sha256(str(tmp_path)) != bench.GEMM_TRAFFIC_SHA256
