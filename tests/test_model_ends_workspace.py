"""What the workspace queries of the operators at both ends of a model promise, against what the calls use.  Host only: the
sizes' arithmetic is asked of the code itself (plain C++, compiled here), and a call is made only where it is refused."""

import ctypes
import os
import shutil
import subprocess

import pytest

import fp8_precision_numerics_amd as fm

EWS = -10
P = ctypes.c_void_p(0x10000)  # never dereferenced
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_numerics_amd", "csrc")
SHIM = """#include "token_chunks.hpp"
#include "vocab_pieces.hpp"
#include "few_rows_shape.hpp"
extern "C" size_t need(int64_t rows, int64_t cols) { return fp8mi::embedding_need(rows, cols); }
extern "C" int64_t chunks(int64_t rows) { return fp8mi::chunk_count(rows); }
extern "C" int64_t most(int64_t m, int64_t k) { return fp8mi::most_columns(m, k); }
extern "C" int64_t launch_columns(int64_t m) { return fp8mi::launch_columns(m); }
extern "C" int64_t few_columns() { return fp8mi::kFewColumns; }
extern "C" int whole(int64_t m, int64_t v, int64_t k, size_t bytes) { return fp8mi::grad_whole(m, v, k, bytes); }
extern "C" int64_t longest(int64_t m, int64_t k, size_t bytes) { return fp8mi::grad_longest(m, k, bytes); }
extern "C" int64_t piece(int64_t m, int64_t v, int64_t k, size_t bytes, int fp8) { return fp8mi::grad_piece(m, v, k, bytes, fp8 != 0, fp8 != 0, 256); }
extern "C" size_t loss_bytes(int64_t m, int64_t p) { return fp8mi::vocab_loss_bytes(m, p); }
extern "C" int64_t few_split(int64_t n, int64_t waves, int64_t most) { return fp8mi::few_split(n, waves, most); }
extern "C" int64_t few_groups(int64_t n, int split) { return fp8mi::few_groups(n, split); }
extern "C" int64_t grad_bytes(int64_t m, int64_t v, int64_t k, int64_t p) { return fp8mi::grad_bytes(m, v, k, p); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("sizes")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"), "-o", str(d / "shim.so")],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.need.argtypes, lib.need.restype = [ctypes.c_int64] * 2, ctypes.c_size_t
    lib.chunks.argtypes, lib.chunks.restype = [ctypes.c_int64], ctypes.c_int64
    for name, args in (("most", "ii"), ("launch_columns", "i"), ("few_columns", ""), ("whole", "iiis"), ("longest", "iis"), ("piece", "iiisc"), ("grad_bytes", "iiii"), ("loss_bytes", "ii"), ("few_split", "iii"),
                       ("few_groups", "ic")):
        f = getattr(lib, name)
        f.argtypes = [dict(i=ctypes.c_int64, s=ctypes.c_size_t, c=ctypes.c_int)[a] for a in args]
        f.restype = dict(whole=ctypes.c_int, loss_bytes=ctypes.c_size_t).get(name, ctypes.c_int64)
    return lib


# around the block of the sort, the last number of tokens in chunks of 16, and each later length of a chunk (24, 32, ..)
ROWS = sorted({1, 15, 16, 17, 31, 8191, 8192, 8193, 40000, 65535, 65536, 65537, 70000, 1 << 20}
              | {4096 * c + d for c in range(16, 257, 8) for d in (-1, 0, 1) if 4096 * c + d <= 1 << 20})


@pytest.mark.parametrize("cols", [16, 64, 4096])
def test_embedding_workspace_holds_any_fewer_tokens(host, cols):
    """The size never falls as the tokens grow, so a scratch that is sized for the largest batch serves every smaller one."""
    sizes = [fm.embedding_workspace_bytes(rows, cols) for rows in ROWS]
    assert sizes == sorted(sizes)
    for rows, size in zip(ROWS, sizes):
        assert host.need(rows, cols) <= size and host.chunks(rows) <= 4096
        if host.need(rows, cols) > 16:
            assert fm.load_library().fp8_embedding_backward(P, 1, rows, P, 1, 256, cols, 1.0, None, P, 1, P, host.need(rows, cols) - 1, None) == EWS


def test_a_head_has_room_for_the_lookups_of_fewer_tokens(host):
    """70000 tokens and a vocabulary of bytes, whose loss asks for less than the lookup's gradient of 65536 tokens."""
    T, H, V = 70000, 4096, 256
    space = fm.Fp8VocabHead(T, H, V, pieces=1, device="cpu").workspace.numel()
    for n in (1, 8193, 65536, 65537, T):
        assert host.need(n, H) <= space


# (rows, vocabulary, hidden): small and large, odd, and hidden sizes at which the longest piece of the gradient, 2^31 codes of the weight, is shorter than the vocabulary
VOCABS = [(1, 1, 16), (1, 131072, 4096), (3, 255, 48), (16, 300, 1024), (17, 257, 128), (63, 50021, 2048), (219, 50021, 2048), (1000, 3000, 64), (1003, 50021, 4096), (2047, 8201, 2048),
          (2048, 32000, 4096), (8191, 65537, 4096), (8192, 65536, 4096), (1000, 40000, 65536), (16, 300, 1 << 22), (500, 600, 1 << 22), (17, 1800, 1 << 20), (7, 1 << 23, 16)]
PIECES = (1, 2, 3, 4, 5, 8, 33, 1000, (1 << 63) - 1)


@pytest.mark.parametrize("M,V,K", VOCABS)
def test_vocab_workspace_is_never_below_its_least(M, V, K):
    """A size for any number of pieces is one that both calls accept."""
    least = fm.vocab_workspace_bytes(M, V, K, 0)
    assert all(fm.vocab_workspace_bytes(M, V, K, pieces) >= least for pieces in PIECES)
    assert fm.load_library().fp8_vocab_cross_entropy_backward(P, 0, P, 0, M, V, K, P, P, P, 1, P, P, 1, P, P, P, 1, P, 1, None, None, 0, P, least - 1, None) == EWS


@pytest.mark.parametrize("M,V,K", VOCABS)
def test_vocab_workspace_holds_the_pieces_it_was_asked_for(host, M, V, K):
    """A workspace for so many pieces serves the gradient in no more, but where the longest piece asks for it; what the estimate
    then takes is at most four more of them, and always fits."""
    for pieces in PIECES:
        size = fm.vocab_workspace_bytes(M, V, K, pieces)
        least = 1 if host.whole(M, V, K, size) else -(-V // host.longest(M, K, size))
        assert least <= max(pieces, -(-V // host.most(M, K))), pieces
        for fp8 in (0, 1):
            P = host.piece(M, V, K, size, fp8)
            assert host.grad_bytes(M, V, K, P) <= size and P <= host.most(M, K) and -(-V // P) <= least + 4 and (P == V or P % 256 == 0)


def test_pieces_of_a_training_step(host):
    """8192 x 65536 x 4096: 2, 4 and 8 pieces asked for are 2, 4 and 8 that fit."""
    for pieces in (1, 2, 4, 8):
        size = fm.vocab_workspace_bytes(8192, 65536, 4096, pieces)
        assert (1 if host.whole(8192, 65536, 4096, size) else -(-65536 // host.longest(8192, 4096, size))) == pieces


def test_few_rows_fit_where_a_pair_for_every_128_columns_does(host):
    """The streaming kernel leaves a pair a workgroup: with the documented bytes for the whole vocabulary its workgroups are no more than
    the pairs, and with room for more they are as many as without a limit."""
    for V in (1, 16, 100, 128, 129, 1000, 16384, 32000, 50021, 65536, 131072, 1 << 20):
        for M in (1, 3, 8, 16):
            slots = (host.loss_bytes(M, V) - host.loss_bytes(M, 0)) // (8 * M)
            assert slots == -(-V // 128)
            for waves in (512, 2048, 2432):
                free = host.few_split(V, waves, 1 << 62)
                split = host.few_split(V, waves, slots)
                assert split in (1, 2, 4, 8) and host.few_groups(V, split) <= slots
                assert split == free or host.few_groups(V, 2 * split) > slots
                assert host.few_split(V, waves, host.few_groups(V, free)) == free
    assert host.few_split(32000, 2048, 1 << 62) == 2 and host.few_groups(32000, 2) == 500 and host.few_split(32000, 2048, 250) == 1


def test_a_launch_has_fewer_than_2_32_threads(host):
    """Whatever the workspace holds: a launch of the logits' product on the smallest tiles, and of the streaming kernel."""
    for M in (1, 16, 17, 64, 65, 8192, 1 << 20, (1 << 23) - 16):
        n = host.launch_columns(M)
        assert n >= 256 and n % 256 == 0 and -(-M // 64) * -(-n // 128) * 256 < 1 << 32
        assert host.most(M, 16) <= n
    assert host.few_columns() % 256 == 0 and host.few_groups(host.few_columns(), 1) * 512 < 1 << 32


@pytest.mark.parametrize("M,V,K", [(1 << 20, 100, 2048), (32, 1000, 72), (1 << 23, 100, 16), ((1 << 23) - 16, 1 << 30, 16), (32, 1 << 31, 16), (32, 1000, (1 << 22) + 16), (-1, 10, 16), (4, 0, 16)])
def test_no_workspace_for_a_loss_that_is_refused(M, V, K):
    """0 where the calls answer an error about their sizes."""
    for call in (lambda: fm.load_library().fp8_vocab_cross_entropy(P, 0, P, 0, M, V, K, P, P, P, 1, P, P, 1, P, 16, None),
                 lambda: fm.load_library().fp8_vocab_cross_entropy_backward(P, 0, P, 0, M, V, K, P, P, P, 1, P, P, 1, P, P, P, 1, P, 1, None, None, 0, P, 16, None)):
        assert call() in (-2, -3)
    assert all(fm.vocab_workspace_bytes(M, V, K, pieces) == 0 for pieces in (0, 1, 4))


@pytest.mark.parametrize("rows,cols", [(100, 24), (100, 8), (100, -16), (-1, 64), ((1 << 20) + 1, 64), (100, (1 << 20) + 16)])
def test_no_workspace_for_a_lookup_that_is_refused(rows, cols):
    assert fm.load_library().fp8_embedding_backward(P, 1, rows, P, 1, 256, cols, 1.0, None, P, 1, P, 16, None) in (-2, -3)
    assert fm.embedding_workspace_bytes(rows, cols) == 0
