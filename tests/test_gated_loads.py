"""Host-only replay of the gated product's B loads (fp8_precision_numerics_amd/csrc/gemm_kernel.hpp
`SlabLoader` with PAIR): every byte of a tile's slab comes from the gate or up row that the tile's
column needs, inside the operand, at the position the fragment reads expect; and of the epilogue's
map from a thread's staged columns to output columns (epilogue.hpp `EpiPass`)."""

import pytest

BK = 128


def lds_swz(row):
    return (row & 6) | ((row >> 3) & 1)


def pair_row(e, P):
    return (8 * e // (2 * P)) * P + 8 * e % P


def pair_up(e, P):
    return (8 * e // P) & 1


@pytest.mark.parametrize("BN,NW,PAIR", [(256, 8, 32), (256, 8, 16), (128, 4, 32), (128, 4, 16)])
@pytest.mark.parametrize("F,n0,K", [(256, 0, 256), (300, 256, 272), (16, 0, 128), (129, 128, 144), (1000, 896, 400)])
def test_pair_slab(BN, NW, PAIR, F, n0, K):
    seen = {}
    for w in range(NW):
        for lane in range(64):
            lrow = w * 8 + (lane >> 3)
            voff = lrow * K + (((lane & 7) ^ lds_swz(lrow)) & 7) * 16
            lane_off = voff - w * 8 * K
            for q in range(BN // 8 // NW):
                e = w + q * NW
                off = lane_off + pair_row(e, PAIR) * K      # the 32-bit offset that the range check sees
                assert 0 <= off < 1 << 31
                lds = w * 1024 + q * NW * 1024 + lane * 16
                seen[lds] = (pair_up(e, PAIR), off)
    assert len(seen) == BN * 8
    rows_left = F - n0
    for row in range(BN):
        col = (row // (2 * PAIR)) * PAIR + row % PAIR       # output column inside the tile
        up = (row // PAIR) & 1
        for g in range(8):
            is_up, off = seen[row * BK + (((g ^ lds_swz(row)) & 7) << 4)]
            assert is_up == up and off == col * K + g * 16
            if col < rows_left:                              # inside: the row exists in its projection
                assert off + 16 <= rows_left * K or g * 16 >= K
            else:                                            # past F: the range check fails, the load reads zero
                assert off >= rows_left * K


@pytest.mark.parametrize("BN,PAIR", [(256, 32), (256, 16), (128, 32), (128, 16)])
def test_epilogue_columns(BN, PAIR):
    """Thread chunk c's staged columns hold output columns 8c .. 8c + 7, and PAIR further their up projection."""
    for c in range(BN // 2 // 8):
        col = (c * 8 // PAIR) * 2 * PAIR + c * 8 % PAIR
        for e in range(8):
            for half in (0, 1):
                row = col + e + half * PAIR
                assert (row // PAIR) & 1 == half
                assert (row // (2 * PAIR)) * PAIR + row % PAIR == 8 * c + e


@pytest.mark.parametrize("steps,split", [(1, 1), (32, 3), (128, 12), (5, 4), (7, 6), (33, 32), (9, 8)])
def test_split_parts_cover_k_once(steps, split):
    """epi_run's part size and the kernel's step ranges: no part is empty, every step has one part."""
    per = -(-steps // split)
    parts = -(-steps // per)
    taken = []
    for part in range(parts):
        kernel_per = -(-steps // parts)
        kt0 = part * kernel_per
        nk = kernel_per if kt0 + kernel_per < steps else steps - kt0
        assert nk >= 1
        taken += range(kt0, kt0 + nk)
    assert taken == list(range(steps))


@pytest.mark.parametrize("chunks,split", [(16, 8), (16, 2), (1, 8), (7, 4), (0, 8)])
def test_few_row_chunks_cover_k_once(chunks, split):
    for tile in (0, 1, 5, 1000):
        first = tile % chunks if chunks else 0
        taken = []
        for part in range(split):
            for c in range(part, chunks, split):
                k = c + first
                taken.append(k if k < chunks else k - chunks)
        assert sorted(taken) == list(range(chunks))


@pytest.mark.parametrize("nfull", [1, 2, 7, 8, 32, 127])
def test_turned_k_steps_are_each_taken_once(nfull):
    for xcd in range(8):
        turn = (xcd * nfull) >> 3
        steps = [kt + turn - (nfull if kt + turn >= nfull else 0) for kt in range(nfull)]
        assert sorted(steps) == list(range(nfull))


@pytest.mark.parametrize("groups", [1, 7, 8, 9, 24, 1972, 2047])
def test_strips_by_xcd_is_a_bijection(groups):
    """The gradients' workgroup order where rows are no multiple of 128 bytes (act_backward.hip)."""
    each, more = groups >> 3, groups & 7
    places = [(b & 7) * each + min(b & 7, more) + (b >> 3) for b in range(groups)]
    assert sorted(places) == list(range(groups))
