"""Host-only replay of the 64 x 128 tiles of the dense GEMMs (csrc/gemm_kernel.hpp): the offsets of their slab loads
(SlabLoader, four wavefronts), and the rotation of the three stages of loads (run_main_loop_deep)."""

import pytest

from test_load_bounds import KBK, U32_MAX, bt_accesses, bt_lds_offset, slab_accesses

BM, BN, NW = 64, 128, 4


@pytest.mark.parametrize("K", [128, 400, 4096, 1 << 23])          # the largest K that the entry points accept
@pytest.mark.parametrize("rows_a,rows_b", [(1, BN), (BM, 1), (BM - 1, BN - 7), (9, 17), (35, 59), (BM, BN), (31, 33), (200, 300)])
def test_slab_loads_stay_inside_the_operand(rows_a, rows_b, K):
    for kt in sorted({0, K // KBK - 1}):
        fetched = {"A": set(), "B": set()}
        for op, row, start, size, chk, nrec in slab_accesses(BM, BN, NW, rows_a, rows_b, K, kt):
            rows_left = rows_a if op == "A" else rows_b
            if chk + size > nrec:                                 # fails the range check: reads zero, touches nothing
                assert row >= rows_left, (op, row)
                continue
            assert row < rows_left and start + size <= rows_left * K
            assert start // K == row and kt * KBK <= start % K and start % K + size <= (kt + 1) * KBK
            fetched[op].add((row, start % K))
        for op, rows in (("A", min(rows_a, BM)), ("B", min(rows_b, BN))):
            assert fetched[op] == {(r, kt * KBK + g * 16) for r in range(rows) for g in range(8)}, op


@pytest.mark.parametrize("N,K", [(4112, 400), (272, 272), (4096, (1 << 19) - 16)])
def test_b_stored_k_by_n(N, K):
    """As for the 128 x 128 tiles, whose B slab this is, for the last tile of a row of tiles and the ragged step."""
    nrec, nfull = min(K * N, U32_MAX), K // KBK
    for n0 in (0, (N - 1) // BN * BN):
        for kt, ragged in ((0, False), (nfull - 1, False), (nfull, True)):
            fetched = set()
            for krow, col, start, chk, lds, _ in bt_accesses(BN, NW, N, K, n0, kt, ragged):
                k = kt * KBK + krow
                if chk + 16 > nrec:
                    assert col >= N or k >= K
                    continue
                assert start == k * N + col and start + 16 <= K * N and lds == bt_lds_offset(BN, krow, col - n0)
                fetched.add((krow, col))
            assert fetched == {(r, c) for r in range(min(KBK, K - kt * KBK)) for c in range(n0, min(n0 + BN, N), 16)}


class Stages:
    """Three LDS stages and each wave's loads in flight, oldest first (they arrive in order).  Every wave is assumed to be
    anywhere between the barriers of the present step, so a stage that is read in a step may not be written in it."""

    LOADS = BM // 8 // NW + BN // 8 // NW                          # one wave's loads of a step (LQA + LQB)

    def __init__(self):
        self.holds = [None] * 3
        self.flight = []                                           # (stage, step), LOADS of them a step, of every wave alike
        self.read, self.written = set(), set()

    def issue(self, stage, step):
        assert stage not in self.read, "a stage is refilled while it is read"
        self.flight += [(stage, step)] * self.LOADS
        self.holds[stage] = None
        self.written.add(stage)

    def put(self, stage, step):                                    # the ragged step, through registers (and direct loads)
        assert stage not in self.read
        self.holds[stage] = step
        self.written.add(stage)

    def wait(self, left):
        done, self.flight = self.flight[:max(0, len(self.flight) - left)], self.flight[max(0, len(self.flight) - left):]
        for stage, step in done:
            self.holds[stage] = step
        for stage, _ in self.flight:
            self.holds[stage] = None

    def barrier(self):
        self.read, self.written = set(), set()

    def frags(self, stage, step):
        assert self.holds[stage] == step, (stage, step, self.holds)
        assert stage not in self.written, "a stage is read in the step that fills it"
        self.read.add(stage)


def run_deep(nfull, ragged):
    """run_main_loop_deep, line by line; returns the steps that were contracted."""
    s, cur, nxt, pre, done = Stages(), 0, 1, 2, []

    def compute(step, into=None):
        s.frags(cur, step)
        if into is not None:
            s.issue(pre, into)
        done.append(step)

    nk = nfull + ragged
    if nfull > 0:
        s.issue(cur, 0)
        if nfull > 1:
            s.issue(nxt, 1)
            s.wait(s.LOADS)
        else:
            s.wait(0)
        s.barrier()
        s.frags(cur, 0)
    kt = 0
    while kt + 2 < nfull:
        compute(kt, kt + 2)
        s.wait(s.LOADS)
        s.barrier()
        s.frags(nxt, kt + 1)
        cur, nxt, pre = nxt, pre, cur
        kt += 1
    while kt < nfull:
        last = kt + 1 == nfull
        if last and ragged:
            s.put(nxt, nfull)
        compute(kt)
        s.wait(0)
        s.barrier()
        if not last:
            s.frags(nxt, kt + 1)
        cur, nxt, pre = nxt, pre, cur
        kt += 1
    if kt < nk:
        if nfull == 0:
            s.put(0, 0)
            s.wait(0)
        s.barrier()
        s.frags(cur, kt)
        compute(kt)
    s.wait(0)
    assert not s.flight
    return done


@pytest.mark.parametrize("ragged", [0, 1])
@pytest.mark.parametrize("nfull", [0, 1, 2, 3, 4, 5, 6, 7, 32])
def test_three_stages_rotate_without_a_clash(nfull, ragged):
    assert run_deep(nfull, ragged) == list(range(nfull + ragged))


def test_the_replay_sees_a_missing_wait():
    """The model itself: reading the next stage with its loads still in flight fails."""
    s = Stages()
    s.issue(0, 0)
    s.issue(1, 1)
    s.wait(s.LOADS + 1)                                            # one load of step 0 is still under way
    s.barrier()
    with pytest.raises(AssertionError):
        s.frags(0, 0)
