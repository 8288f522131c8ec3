"""Pins of the oracle of the operators at both ends of a model: the generator's published
answers, closed forms, and every gradient against central differences of the value it belongs to."""

import numpy as np
import pytest

from oracle import model_ends as me


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_known_answers(counter, key, want):
    """The three known-answer vectors that the generator's authors publish for 10 rounds."""
    assert tuple(me.philox4x32(counter, key)) == want


def test_dropout_factors_take_the_half_words_in_order():
    seed, offset, first = (7 << 40) + 11, (3 << 33) + 5, (1 << 32) - 1   # the octets' numbers pass 2^32
    f = me.dropout_factors((4, 16), 0.25, seed, offset, first).reshape(-1)
    want = []
    for g in range(first, first + 8):
        words = me.philox4x32((g & me.MASK, g >> 32, offset & me.MASK, offset >> 32), (seed & me.MASK, seed >> 32))
        for w in words:
            want += [w & 0xFFFF, w >> 16]
    assert np.array_equal(f, np.where(np.array(want) < 16384, 0.0, 4.0 / 3.0))


def test_dropout_keeps_the_expectation():
    for p in (0.1, 0.5, 0.9):
        f = me.dropout_factors((1000, 1000), p, 1, 2)
        cut = me.dropout_cut(p) / 65536
        assert abs(cut - p) < 2.0 ** -16
        # a million draws: five deviations of their mean
        assert abs(f.mean() - 1.0) < 5 * np.sqrt(cut / (1 - cut) / 1e6)
    assert np.all(me.dropout_factors((3, 8), 0.0, 1, 2) == 1.0)
    assert me.dropout_cut(0.1) == 6554 and me.dropout_cut(1.0 - 2.0 ** -16) == 65535


def test_norm_closed_forms():
    w, b = np.array([1.0, -2.0, 0.5, 3.0]), np.array([0.0, 1.0, 0.0, -1.0])
    y, m, r = me.layer_norm([[1.0, 3.0, 1.0, 3.0], [7.0, 7.0, 7.0, 7.0], [0.0, 0.0, 8.0, 0.0]], w, b, 1e-30)
    assert np.allclose(m, [2.0, 7.0, 2.0]) and np.allclose(r[[0, 2]], [1.0, 1.0 / np.sqrt(12.0)], rtol=1e-14)
    assert np.allclose(y[0], [-1.0, -1.0, -0.5, 2.0], rtol=1e-14) and np.allclose(y[1], b)
    assert np.isclose(me.layer_norm([[1.0, -1.0]], [1.0, 1.0], None, 8.0)[2][0], 1 / 3.0, rtol=1e-15)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    h, w, b, dy = rng.normal(size=(3, 7)) + 2, rng.normal(size=7), rng.normal(size=7), rng.normal(size=(3, 7))
    dh, dw, db = me.layer_norm_grad(dy, h, w, 0.1)
    e = 1e-6

    def value(h_, w_, b_):
        return np.sum(dy * me.layer_norm(h_, w_, b_, 0.1)[0])

    for i in range(3):
        for j in range(7):
            d = np.zeros_like(h)
            d[i, j] = e
            assert dh[i, j] == pytest.approx((value(h + d, w, b) - value(h - d, w, b)) / (2 * e), abs=1e-8)
    for j in range(7):
        d = np.zeros(7)
        d[j] = e
        assert dw[j] == pytest.approx((value(h, w + d, b) - value(h, w - d, b)) / (2 * e), abs=1e-8)
        assert db[j] == pytest.approx((value(h, w, b + d) - value(h, w, b - d)) / (2 * e), abs=1e-8)


def test_cross_entropy_closed_forms():
    z = np.array([[0.0, 0.0, 0.0, 0.0], [np.log(1.0), np.log(2.0), np.log(3.0), np.log(10.0)], [1000.0, 0.0, 0.0, 0.0], [5.0, 1.0, 2.0, 3.0]])
    loss, lse = me.cross_entropy(z, [2, 1, 0, -100])
    assert np.allclose(lse[:3], [np.log(4.0), np.log(16.0), 1000.0], rtol=1e-15)
    assert np.allclose(loss, [np.log(4.0), np.log(8.0), 0.0, 0.0], atol=1e-12)
    d = me.cross_entropy_grad(z, [2, 1, 0, 4], [1.0, 2.0, 1.0, 1.0])
    assert np.allclose(d[0], [0.25, 0.25, -0.75, 0.25]) and np.allclose(d[1], np.array([1, 2 - 16, 3, 10]) / 8.0) and np.all(d[3] == 0)


def test_cross_entropy_gradient_against_differences():
    rng = np.random.default_rng(5)
    z, t, g = rng.normal(size=(4, 9)) * 3, np.array([0, 8, -1, 3]), rng.normal(size=4)
    d = me.cross_entropy_grad(z, t, g)
    e = 1e-6
    for i in range(4):
        for j in range(9):
            s = np.zeros_like(z)
            s[i, j] = e
            num = np.sum(g * (me.cross_entropy(z + s, t)[0] - me.cross_entropy(z - s, t)[0])) / (2 * e)
            assert d[i, j] == pytest.approx(num, abs=1e-8)


def test_embedding_and_its_gradient():
    rng = np.random.default_rng(7)
    table, ids = rng.normal(size=(6, 4)), np.array([2, 5, 2, -1, 0, 6, 2])
    out = me.embedding(ids, table, 3.0)
    assert np.allclose(out[0], 3 * table[2]) and np.all(out[3] == 0) and np.all(out[5] == 0)
    dy, base = rng.normal(size=(7, 4)), rng.normal(size=(6, 4))
    grad = me.embedding_grad(ids, dy, 6, 3.0, base) - base
    e = 1e-6
    for i in range(6):
        for j in range(4):
            s = np.zeros_like(table)
            s[i, j] = e
            num = np.sum(dy * (me.embedding(ids, table + s, 3.0) - me.embedding(ids, table - s, 3.0))) / (2 * e)
            assert grad[i, j] == pytest.approx(num, abs=1e-8)
    assert np.all(grad[[1, 3, 4]] == 0)
