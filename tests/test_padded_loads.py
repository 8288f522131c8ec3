"""Host-only replay of the vocabulary products' loads (csrc/gemm_kernel.hpp, SlabLoader with PADDED) and of the code tiles
that feed them (csrc/vocab_epilogue.hpp).

The hardware checks a load's per-lane VGPR offset against the resource's size and adds the scalar offset afterwards.
A's rows are padded to whole steps, so its loads are the plain ones with lda in the place of K; B [K x N] carries its row in the
VGPR offset in every step, so that a row at or past K reads as zero whatever K is."""

import numpy as np
import pytest

from test_load_bounds import KBK, U32_MAX, bt_lds_offset, lds_swz

SHAPES = [(256, 256, 8), (128, 128, 4), (64, 128, 4)]
OUT_OF_RANGE = 0x80000000


@pytest.mark.parametrize("BM,BN,NW", SHAPES)
@pytest.mark.parametrize("lda,rows_left", [(128, 1), (128, 300), (384, 37), (1 << 20, 255), (1 << 23, 256)])
def test_a_loads_stay_inside_the_padded_rows(BM, BN, NW, lda, rows_left):
    nrec = min(rows_left * lda, U32_MAX)
    for kt in sorted({0, 1, lda // KBK - 1}):
        if kt * KBK >= lda:
            continue
        seen = set()
        for w in range(NW):
            for lane in range(64):
                lrow = w * 8 + (lane >> 3)
                for q in range(BM // 8 // NW):
                    v = lrow * lda + (((lane & 7) ^ lds_swz(lrow)) & 7) * 16 + q * NW * 8 * lda
                    assert v < 2 ** 31
                    row = lrow + q * NW * 8
                    if v + 16 <= nrec:                    # fetched: inside the row that passed the check
                        start = v + kt * KBK
                        assert start // lda == row and start + 16 <= rows_left * lda and row < rows_left
                        seen.add((row, start % lda - kt * KBK))
                    else:
                        assert row >= rows_left
        assert seen == {(r, g * 16) for r in range(min(BM, rows_left)) for g in range(8)}


@pytest.mark.parametrize("BN,NW", [(256, 8), (128, 4)])
@pytest.mark.parametrize("N,K", [(16, 1), (16, 127), (144, 128), (272, 129), (4096, 219), (2048, (1 << 20) - 3), (256, (1 << 23) - 1), (1 << 22, 511)])
def test_b_loads_read_rows_below_k_and_nothing_else(BN, NW, N, K):
    """Offsets are 32-bit: one that wraps has to come from a column past N, which feeds no stored output."""
    assert N * K < 2 ** 31
    RPB = 1024 // BN
    steps = (K + KBK - 1) // KBK
    for n0 in sorted({0, (N - 1) // BN * BN}):
        for kt in sorted({0, steps - 1}):
            got = {}
            for w in range(NW):
                for lane in range(64):
                    r = w * RPB + lane // (BN // 16)
                    g = (lane % (BN // 16)) ^ (r & 7)
                    col = n0 + 16 * g
                    base = r * N + col if col < N else OUT_OF_RANGE
                    for d in range(BN // 8 // NW):
                        off = (base + (d * NW * RPB + kt * KBK) * N) & U32_MAX
                        krow = kt * KBK + d * NW * RPB + r
                        inside = off + 16 <= N * K
                        if col < N:
                            assert inside == (krow < K)
                            if inside:
                                assert (off // N, off % N) == (krow, col)
                                lds = (w + d * NW) * 1024 + lane * 16
                                assert lds == bt_lds_offset(BN, krow - kt * KBK, col - n0)
                                got[krow, col] = True
            want = {(k, c) for k in range(kt * KBK, min(K, kt * KBK + KBK)) for c in range(n0, min(N, n0 + BN), 16)}
            assert set(got) == want


@pytest.mark.parametrize("BM,BN", [(256, 256), (128, 128), (64, 128)])
@pytest.mark.parametrize("BLK", [32, 16])
def test_code_tiles_hold_every_code_once_both_ways(BM, BN, BLK):
    """The lanes' dwords and their quad transposes fill both LDS tiles, which lie one behind the other in the stages' space."""
    assert 2 * BM * BN <= 2 * (BM + BN) * KBK

    def at(cols, r, byte):
        return r * cols + ((((byte >> 4) ^ r) & (cols // 16 - 1)) << 4) + (byte & 15)

    rows, cols = -np.ones(BM * BN, dtype=np.int64), -np.ones(BN * BM, dtype=np.int64)
    groups = 4 if BLK == 32 else 1
    for i in range(BM // BLK):
        for j in range(BN // BLK):
            for g in range(groups):
                words = {}
                for lane in range(64):
                    r = i * BLK + (lane & (BLK - 1))
                    c = j * BLK + (8 * g + 4 * (lane >> 5) if BLK == 32 else 4 * (lane >> 4))
                    words[lane] = [(r, c + e) for e in range(4)]
                    for e in range(4):
                        p = at(BN, r, c) + e
                        assert rows[p] == -1
                        rows[p] = r * BN + c + e
                for lane in range(64):
                    r, c = words[lane][0]
                    quad = [words[(lane & ~3) + k][lane & 3] for k in range(4)]     # byte k: lane k's code of column lane & 3
                    for k in range(4):
                        p = at(BM, c + (lane & 3), r & ~3) + k
                        assert cols[p] == -1
                        cols[p] = quad[k][0] * BN + quad[k][1]
    for r in range(BM):
        for b in range(0, BN, 16):
            p = at(BN, r, b)
            assert np.array_equal(rows[p:p + 16], r * BN + b + np.arange(16))
    for c in range(BN):
        for b in range(0, BM, 16):
            p = at(BM, c, b)
            assert np.array_equal(cols[p:p + 16], (b + np.arange(16)) * BN + c)


@pytest.mark.parametrize("M", [1, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 200, 256, 300])
@pytest.mark.parametrize("BM", [64, 128, 256])
def test_the_transposed_rows_are_written_up_to_their_padding(M, BM):
    """Rows of the transposed codes are up128(M) long; the tiles and, with 64-row tiles, the last one's extra half fill each exactly once."""
    ldt = (M + 127) // 128 * 128
    written = np.zeros(ldt, dtype=int)
    for m_base in range(0, M, BM):
        for byte in range(0, BM, 16):
            if m_base + byte < ldt:
                written[m_base + byte:m_base + byte + 16] += 1
        if BM < 128 and m_base + 2 * BM == ldt and m_base + BM >= M:
            written[m_base + BM:m_base + 2 * BM] += 1
    assert (written == 1).all()
