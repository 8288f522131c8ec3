"""GPU parity of the vocabulary's cross entropy against the fp64 definition.

Tolerances, derived before the first run:
* logits z: the library's GEMM bound B = 1e-5 * sum|ab| * sinv_x * sinv_w (exact mode), or the FP8 matrix
  cores' error model (gpu_helpers.mfma8_bound).
* lse: it moves by at most the largest move of a logit, max B; its sum of exponentials passes through
  less than 128 roundings (at most 64 values a lane, then lanes, waves, tiles), and each exponential is good to 4
  roundings on average: SUMS = 1e-5; then EW of lse itself.  loss = lse - z[target]: max B + B of the target, SUMS,
  EW |lse| and EW |z[target]|.
* d = dloss (exp(z - lse) - [target]): |dloss| (p (exp(B) - 1) + EW (p (1 + |z - lse|) + [target])); the codes lie in the
  oracle's bracket of round_to_fp8 over that interval.
* dx, dw: the products of the oracle's codes, with what the bracket leaves open times the other operand, the GEMM
  bound on those codes, and half a step of the output's type."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
import vocab_cases
from gpu_helpers import announce, device, mfma8_bound
from oracle import codec, gemm, model_ends as me, scaling
from test_gpu_feed_forward import EW, HALF, check_close, d64, rand_codes, scalar, u8

pytestmark = pytest.mark.gpu
SUMS = 1e-5


def decoded(q, fmt):
    """fp64 values of codes, on the GPU."""
    return q.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double()


def normal_codes(seed, shape, fmt, std):
    """Codes of a normal tensor and the inverse scale that makes its deviation `std`."""
    g = torch.Generator(device=device()).manual_seed(seed)
    to, top = (torch.float8_e4m3fn, 448.0) if fmt == "e4m3" else (torch.float8_e5m2, 57344.0)
    v = torch.randn(shape, generator=g, device=device()) * (top / 6)
    return v.clamp(-top, top).to(to).view(torch.uint8), scalar(6 * std / top)


class Problem:
    def __init__(self, M, V, K, fx="e4m3", fw="e4m3", seed=0, spread=3.0, index=torch.int64, ignored=0.1):
        self.M, self.V, self.K, self.fx, self.fw = M, V, K, fx, fw
        self.x, self.sx = normal_codes(seed + 1, (M, K), fx, 1.0)
        self.w, self.sw = normal_codes(seed + 2, (V, K), fw, spread / np.sqrt(K))
        gen = np.random.default_rng(seed + 3)
        t = gen.integers(0, V, size=M)
        if M > 3:
            t[gen.random(M) < ignored] = -100
            t[1], t[2] = V, V - 1                     # one past the end, and the last column
        self.t = t.astype(np.int64)
        self.targets = torch.from_numpy(self.t).to(index).to(device())
        self.dloss = torch.from_numpy(gen.normal(size=M).astype(np.float32)).to(device())

    def logits(self, accum, rows=None, cols=None):
        """z and its bound B for some rows and columns, fp64 numpy."""
        x = self.x if rows is None else self.x[rows]
        w = self.w if cols is None else self.w[cols]
        a, b, s = decoded(x, self.fx), decoded(w, self.fw), self.sx.double() * self.sw.double()
        z = (a @ b.t() * s).cpu().numpy()
        if accum == "mfma_fp8" and self.M > 16:
            return z, mfma8_bound(u8(x), self.fx, u8(w), self.fw, self.sx.item(), self.sw.item())
        return z, (1e-5 * (a.abs() @ b.abs().t()) * s).cpu().numpy()

    def forward(self, accum="exact", pieces=1, workspace=None, **kw):
        loss, lse = (torch.full((self.M,), -7.0, device=device()) for _ in range(2))
        if workspace is None:
            workspace = torch.full((max(16, fm.vocab_workspace_bytes(self.M, self.V, self.K, pieces)),), 0xA5, dtype=torch.uint8, device=device())
        fm.fp8_vocab_cross_entropy(self.x, self.fx, self.w, self.fw, self.sx, self.sw, self.targets, loss, lse, accum=accum, workspace=workspace, **kw)
        return loss, lse

    def backward(self, lse, accum="exact", pieces=1, fmt="e5m2", scale=64.0, types=(torch.float32, torch.float32), stats=True, workspace=None, **kw):
        dx = None if types[0] is None else torch.full((self.M, self.K), -7.0, dtype=types[0], device=device())
        dw = None if types[1] is None else torch.full((self.V, self.K), -7.0, dtype=types[1], device=device())
        amax, sat = (scalar(-1.0), scalar(12345, torch.int64)) if stats else (None, None)
        if workspace is None:
            workspace = torch.full((max(16, fm.vocab_workspace_bytes(self.M, self.V, self.K, pieces)),), 0xA5, dtype=torch.uint8, device=device())
        fm.fp8_vocab_cross_entropy_backward(self.x, self.fx, self.w, self.fw, self.sx, self.sw, self.targets, lse, self.dloss, fmt, scalar(scale), scalar(1 / scale),
                                            dx=dx, dw=dw, amax=amax, sat=sat, accum=accum, workspace=workspace, **kw)
        return dx, dw, amax, sat


def check_forward(p, accum, loss, lse, rows):
    z, B = p.logits(accum, rows)
    want, want_lse = me.cross_entropy(z, p.t[rows])
    inside = (p.t[rows] >= 0) & (p.t[rows] < p.V)
    at = np.where(inside, p.t[rows], 0)
    zt, Bt = z[np.arange(len(rows)), at], B[np.arange(len(rows)), at]
    tol = B.max(axis=1) + SUMS + EW * np.abs(want_lse)
    check_close(d64(lse)[rows], want_lse, tol, "lse")
    check_close(d64(loss)[rows], want, np.where(inside, tol + Bt + EW * np.abs(zt), 0.0), "loss")


def gradient(p, accum, lse, rows, cols, fmt, scale):
    """(d, error bound) of rows x cols."""
    z, B = p.logits(accum, rows, cols)
    r, c = np.arange(p.M) if rows is None else rows, np.arange(p.V) if cols is None else cols
    l = d64(lse)[r][:, None]
    t, g = p.t[r][:, None], d64(p.dloss)[r][:, None]
    live, hit = (t >= 0) & (t < p.V), t == c[None, :]
    prob = np.exp(z - l)
    d = np.where(live, g * (prob - hit), 0.0)
    return d, np.where(live, np.abs(g) * (prob * np.expm1(B) + EW * (prob * (1 + np.abs(z - l)) + hit)), 0.0)


def check_product(got, d, err, other, fo, so, scale, inv, fmt, accum, what):
    """got = codes(d) · other / scale, d [R x N], other: codes [N x K] as a GPU tensor."""
    r = gemm.requant_bracket(d, err, np.float32(scale), fmt)
    q = scaling.quantize(d.astype(np.float32), np.float32(scale), fmt)[0]
    v = codec.decode(q, fmt)
    open_ = np.maximum(r["hi"] - v, v - r["lo"])
    b = decoded(other, fo).cpu().numpy()
    inv32, inv = np.float32(inv), np.float64(np.float32(inv)) * so.item()
    want = v @ b * inv
    mag = np.abs(v) @ np.abs(b) * inv
    if accum == "exact":
        bound = 1e-5 * mag
    else:  # any n: the run of 8 is completed with zeros
        n = (-v.shape[1]) % 8
        bound = mfma8_bound(np.pad(q, ((0, 0), (0, n))), fmt, np.pad(u8(other).T, ((0, 0), (0, n))), fo, inv32, so.item())
    got = d64(got)
    half = HALF[what[1]]
    # The type's rounding is of the value that was computed, not of `want`: that one is at most |want| + `off` large, so half
    # a step is at most half * (|want| + off).  (bf16, a code at the other end of its bracket: 2.452e-5 wanted, 6.390e-5 got, off by
    # 3.9373e-5; without half * off, 3.84e-5 / 256 = 1.5e-7, the bound was 3.9338e-5.)
    off = bound + open_ @ np.abs(b) * inv + 2.0 ** -24 * mag
    check_close(got, want, off + half * 1.001 * (np.abs(want) + off), what[0])


def check_backward(p, accum, lse, out, fmt, scale, rows=None, cols=None, types=(torch.float32, torch.float32), inv=None):
    dx, dw, amax, sat = out
    inv = 1 / scale if inv is None else inv.item()
    if dx is not None:
        d, err = gradient(p, accum, lse, rows, None, fmt, scale)
        check_product(dx if rows is None else dx[rows], d, err, p.w, p.fw, p.sw, scale, inv, fmt, accum, ("dx", types[0]))
        if rows is None and amax is not None:
            top = np.abs(d)
            assert (top - err).max() <= amax.item() * (1 + 1e-6) and amax.item() <= (top + err).max() * (1 + 1e-6)
            limit = codec.FORMATS[fmt].max_value
            lo, hi = np.sum((top - err) * scale * (1 - 1e-6) > limit), np.sum((top + err) * scale * (1 + 1e-6) > limit)
            assert sat is None or lo <= sat.item() <= hi
    if dw is not None:
        d, err = gradient(p, accum, lse, None, cols, fmt, scale)
        check_product(dw if cols is None else dw[cols], d.T, err.T, p.x, p.fx, p.sx, scale, inv, fmt, accum, ("dw", types[1]))


SMALL = [(1, 1, 16), (1, 1000, 16), (3, 17, 48), (5, 2, 4096), (16, 300, 64), (17, 257, 128), (33, 2500, 80), (100, 1000, 1040), (130, 515, 256), (250, 127, 144), (8, 33001, 16), (9, 33001, 16), (16, 33001, 48)]


@pytest.mark.parametrize("M,V,K", SMALL)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("fx,fw,index", [("e4m3", "e4m3", torch.int64), ("e5m2", "e4m3", torch.int32), ("e4m3", "e5m2", torch.int64), ("e5m2", "e5m2", torch.int32)])
def test_forward(M, V, K, accum, fx, fw, index):
    announce(f"cross entropy {M}x{V}x{K} {accum} {fx} {fw}")
    p = Problem(M, V, K, fx, fw, index=index)
    for pieces in (1, 3, 0):
        loss, lse = p.forward(accum, pieces)
        check_forward(p, accum, loss, lse, np.arange(M))
    only = torch.full((M,), -7.0, device=device())
    ws = torch.empty(fm.vocab_workspace_bytes(M, V, K), dtype=torch.uint8, device=device())
    loss, lse = p.forward(accum)
    fm.fp8_vocab_cross_entropy(p.x, fx, p.w, fw, p.sx, p.sw, p.targets, only, None, accum=accum, workspace=ws)
    assert torch.equal(only, loss)
    fm.fp8_vocab_cross_entropy(p.x, fx, p.w, fw, p.sx, p.sw, p.targets, None, only, accum=accum, workspace=ws)
    assert torch.equal(only, lse)


@pytest.mark.parametrize("M,V,K", SMALL)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("fx,fw,fmt,types,pieces", [("e4m3", "e4m3", "e5m2", (torch.bfloat16, torch.bfloat16), 1), ("e4m3", "e5m2", "e5m2", (torch.bfloat16, torch.float32), 3),
                                                    ("e5m2", "e4m3", "e4m3", (torch.float32, torch.bfloat16), 2), ("e5m2", "e5m2", "e4m3", (torch.bfloat16, torch.bfloat16), 0)])
def test_backward(M, V, K, accum, fx, fw, fmt, types, pieces):
    announce(f"cross entropy backward {M}x{V}x{K} {accum} {fx} {fw} {fmt} {types} pieces={pieces}")
    p = Problem(M, V, K, fx, fw)
    lse = p.forward(accum)[1]
    scale = 64.0 if fmt == "e4m3" else 40000.0            # some of the targets' values saturate
    out = p.backward(lse, accum, pieces, fmt, scale, types)
    check_backward(p, accum, lse, out, fmt, scale, types=types)
    # either gradient by itself, without statistics: the same bits
    dx = p.backward(lse, accum, pieces, fmt, scale, (types[0], None), stats=False)[0]
    dw = p.backward(lse, accum, pieces, fmt, scale, (None, types[1]), stats=False)[1]
    assert torch.equal(dw, out[1])
    if pieces == 1:                                       # the pieces depend on the space, and that on what is asked for
        assert torch.equal(dx, out[0])


@pytest.mark.parametrize("M,V,K", vocab_cases.LOGITS)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_large(M, V, K, accum):
    announce(f"cross entropy large {M}x{V}x{K} {accum}")
    p = Problem(M, V, K, seed=5)
    rows, cols = np.array([0, 1, 2, M // 2, M - 1]), np.array([0, 5, V // 2, V - 1])
    for pieces in (1, 2):
        loss, lse = p.forward(accum, pieces)
        check_forward(p, accum, loss, lse, rows)
        assert torch.isfinite(lse).all()
        out = p.backward(lse, accum, pieces, "e5m2", 20000.0, (torch.bfloat16, torch.bfloat16))
        check_backward(p, accum, lse, out, "e5m2", 20000.0, rows, cols, (torch.bfloat16, torch.bfloat16))
        dx, dw = out[:2]
        assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()
        assert (dx[torch.from_numpy((p.t < 0) | (p.t >= V)).to(device())] == 0).all()
    # the same call again gives the same bits
    again = p.backward(lse, accum, 2, "e5m2", 20000.0, (torch.bfloat16, torch.bfloat16))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], out[2])


def test_the_gradient_is_the_slope_of_the_loss():
    """All logits 0: d = 1/4 and -3/4 are codes, so dx is the loss's slope at x = 0; it is compared with the loss of
    x = +-2^-6 along each coordinate (E4M3's smallest normal number).  Error of the difference: the third derivative's e^2 / 6 < 4.1e-5 times |w|^3 / 10 < 1, and
    two fp32 losses of 1.4 rounded a few times, 4 * 1.2e-7 / (2 e) = 1.6e-5; under 1e-4 in all."""
    announce("cross entropy against differences")
    K, V = 16, 4
    w = rand_codes(3, (V, K), "e4m3")
    w = torch.where((w & 0x7F) > 0x38, (w & 0x80) | 0x38, w)                       # |w| <= 1
    one, t = scalar(1.0), torch.tensor([2] * 17, device=device())
    ws = torch.empty(fm.vocab_workspace_bytes(17, V, K), dtype=torch.uint8, device=device())
    loss, lse = torch.zeros(17, device=device()), torch.zeros(17, device=device())

    def values(x):
        fm.fp8_vocab_cross_entropy(x, "e4m3", w, "e4m3", one, one, t, loss, lse, workspace=ws)
        return d64(loss).copy()

    x = torch.zeros((17, K), dtype=torch.uint8, device=device())
    for i in range(K):
        x[i, i] = 0x08                                                               # 2^-6
    up = values(x)
    x[x != 0] = 0x88
    down = values(x)
    x.zero_()
    assert np.allclose(values(x), np.log(4.0), atol=1e-6)
    dx, dw = torch.zeros((17, K), device=device()), torch.zeros((V, K), device=device())
    fm.fp8_vocab_cross_entropy_backward(x, "e4m3", w, "e4m3", one, one, t, lse, torch.ones(17, device=device()), "e5m2", one, one, dx=dx, dw=dw, workspace=ws)
    assert np.abs(d64(dx)[0] - ((up - down) * 2.0 ** 5)[:K]).max() < 1e-4 and (dw == 0).all()


def test_extreme_logits():
    """Logits of +-20000: the loss keeps its error relative to them; columns far below the largest add nothing."""
    announce("cross entropy extreme logits")
    for M in (3, 40):
        p = Problem(M, 700, 64, spread=5000.0, ignored=0.0)
        loss, lse = p.forward()
        check_forward(p, "exact", loss, lse, np.arange(M))
        out = p.backward(lse, scale=8.0)
        # an error of B in a logit of this size is more than a unit of its exponent: only the bits' sanity is left
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[1]).all()


def test_special_values():
    """A NaN and an infinite logit make their row NaN and no other; a row without a target has no gradient even then; a logit of -Inf adds 0."""
    announce("cross entropy special values")
    for M in (6, 60):
        p = Problem(M, 300, 64, fx="e5m2", ignored=0.0)
        p.t[:] = np.arange(M) % 300
        p.t[4] = -1
        p.targets.copy_(torch.from_numpy(p.t).to(device()))
        clean, clean_lse = p.forward()
        x = p.x.clone()
        x[0, 3], x[4, 0] = 0x7F, 0x7F                                                # NaN
        x[2, 5] = 0x7C                                                               # +Inf, times weights of both signs
        p.x, keep = x, p.x
        loss, lse = p.forward()
        bad = torch.zeros(M, dtype=torch.bool, device=device())
        bad[[0, 2]] = True
        assert torch.isnan(loss[bad]).all() and torch.isnan(lse[[0, 2, 4]]).all() and loss[4] == 0
        good = ~bad
        good[4] = False
        assert torch.equal(loss[good], clean[good]) and torch.equal(lse[good], clean_lse[good])
        dx, dw, amax, _ = p.backward(lse)
        assert torch.isnan(dx[bad]).all() and (dx[4] == 0).all() and torch.isfinite(dx[good]).all() and torch.isnan(amax).all()
        assert torch.isnan(dw).all()                                                 # every column's gradient has the two rows in it
        p.x = keep
        # no target at all: the logits may be anything
        p.x = torch.full_like(keep, 0x7F)
        p.targets.fill_(-100)
        loss, lse = p.forward()
        dx, dw, amax, sat = p.backward(lse)
        assert (loss == 0).all() and (dx == 0).all() and amax.item() == 0 and sat.item() == 0
        # 0 * NaN of dw's other operand: dw = codes (all 0) · x
        assert torch.isnan(dw).all()
        p.x = keep
        dx, dw, amax, sat = p.backward(clean_lse)
        assert (dx == 0).all() and (dw == 0).all()
    # weights of one sign: a row of -Inf in x gives logits of -Inf in all but the columns of zeros
    w = torch.full((5, 16), 0x38, dtype=torch.uint8, device=device())
    w[[1, 3]] = 0
    x = torch.zeros((2, 16), dtype=torch.uint8, device=device())
    x[0, 0] = 0xC8                                                                   # -8 in E5M2
    one, ws = scalar(100.0), torch.empty(4096, dtype=torch.uint8, device=device())
    loss, lse = torch.zeros(2, device=device()), torch.zeros(2, device=device())
    fm.fp8_vocab_cross_entropy(x, "e5m2", w, "e4m3", one, one, torch.tensor([1, 0], device=device()), loss, lse, workspace=ws)
    assert np.allclose(loss.cpu(), [np.log(2.0), np.log(5.0)], atol=1e-6)


@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_infinite_dloss(M, accum):
    """A row's infinite dloss saturates its codes, and the columns that pad the vocabulary stay zeros; where a probability is 0
    the gradient is NaN, and so is amax."""
    announce(f"cross entropy infinite dloss {M} {accum}")
    V, K, scale = 130, 64, 8.0
    p = Problem(M, V, K, spread=1.0, ignored=0.0)
    p.t[2] = V - 1
    p.dloss[2] = float("inf")
    _, lse = p.forward(accum)
    dx, dw, amax, sat = p.backward(lse, accum, scale=scale)
    v = np.full(V, 57344.0)
    v[p.t[2]] = -57344.0
    w = decoded(p.w, p.fw).cpu().numpy()
    inv = p.sw.item() / scale
    # the codes are known; all other rows' are too small to saturate, so the count is the row's
    mag = np.abs(v) @ np.abs(w) * inv
    bound = 1e-5 * mag if accum == "exact" else mfma8_bound(np.pad(np.where(v > 0, 0x7B, 0xFB).astype(np.uint8)[None], ((0, 0), (0, (-V) % 8))), "e5m2", np.pad(u8(p.w).T, ((0, 0), (0, (-V) % 8))), p.fw, np.float32(1 / scale), p.sw.item())[0]
    check_close(d64(dx)[2], v @ w * inv, bound + 2.0 ** -23 * mag, "dx of the infinite row")
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert amax.item() == float("inf") and sat.item() == V
    p = Problem(M, V, K, spread=5000.0, ignored=0.0)
    p.t[2] = V - 1
    p.dloss[2] = float("inf")
    _, lse = p.forward(accum)
    dx, dw, amax, _ = p.backward(lse, accum, scale=scale)
    assert torch.isnan(dx[2]).all() and torch.isnan(amax).all()
    rest = torch.arange(M, device=device()) != 2
    assert torch.isfinite(dx[rest]).all()


def test_rows_of_infinite_logits():
    """-Inf in all columns but one, in all but none, and a +Inf among them; int32 and int64 targets."""
    announce("cross entropy infinite logits")
    w = torch.full((70, 16), 0x38, dtype=torch.uint8, device=device())               # 1 in E4M3
    w[5] = 0xB8                                                                      # -1
    for M in (3, 35):
        x = torch.zeros((M, 16), dtype=torch.uint8, device=device())
        x[0, 0] = 0xFC                                                               # -Inf in E5M2: column 5 is +Inf, the others -Inf
        x[1, 2] = 0xFC
        for index in (torch.int32, torch.int64):
            t = torch.zeros(M, dtype=index, device=device())
            one, ws = scalar(1.0), torch.empty(1 << 16, dtype=torch.uint8, device=device())
            loss, lse = torch.zeros(M, device=device()), torch.zeros(M, device=device())
            fm.fp8_vocab_cross_entropy(x, "e5m2", w, "e4m3", one, one, t, loss, lse, workspace=ws)
            assert torch.isnan(loss[:2]).all() and torch.isnan(lse[:2]).all() and np.allclose(lse[2:].cpu(), np.log(70.0), atol=1e-6)
            down = torch.cat([w[:5], w[6:]])
            fm.fp8_vocab_cross_entropy(x, "e5m2", down, "e4m3", one, one, t, loss, lse, workspace=ws)
            assert (lse[:2] == -float("inf")).all() and torch.isnan(loss[:2]).all() and np.allclose(lse[2:].cpu(), np.log(69.0), atol=1e-6)


@pytest.mark.parametrize("M,V,K", [(36001, 60033, 32), (20, 131201, 16384)])
def test_operands_of_more_than_2_31_codes(M, V, K):
    """Codes of the logits' gradient beyond 2^31 in one piece, and a weight of more than 2^31 codes: the last rows and columns are right."""
    announce(f"cross entropy {M}x{V}x{K}")
    p = Problem(M, V, K)
    rows, cols = np.array([0, M - 2, M - 1]), np.array([0, V // 2, V - 1])
    loss, lse = p.forward()
    check_forward(p, "exact", loss, lse, rows)
    assert torch.isfinite(lse).all()
    types = (torch.bfloat16, torch.bfloat16)
    out = p.backward(lse, "exact", 1, "e5m2", 20000.0, types)
    check_backward(p, "exact", lse, out, "e5m2", 20000.0, rows, cols, types)


def test_no_rows():
    announce("cross entropy no rows")
    p = Problem(0, 300, 64)
    loss, lse = p.forward()
    dx, dw, amax, sat = p.backward(lse)
    assert (dw == 0).all() and amax.item() == 0 and sat.item() == 0
    dw = p.backward(lse, types=(None, torch.bfloat16))[1]
    assert (dw == 0).all()


def test_workspace_is_not_passed():
    """The least workspace, with a guard behind it, forward and backward."""
    announce("cross entropy workspace")
    for M, V, K in ((1, 70000, 32), (16, 5000, 64), (17, 300, 32), (300, 1000, 128), (1000, 3000, 64)):
        p = Problem(M, V, K)
        ws = fm.vocab_workspace_bytes(M, V, K, 0)
        space = torch.full((ws + 4096,), 0xA5, dtype=torch.uint8, device=device())
        loss, lse = p.forward(workspace=space[:ws])
        full, full_lse = p.forward()
        assert (space[ws:] == 0xA5).all()
        tol = SUMS + EW * 50
        assert (loss - full).abs().max() < tol and (lse - full_lse).abs().max() < tol
        dx, dw, _, _ = p.backward(lse, types=(torch.bfloat16, torch.bfloat16), workspace=space[:ws])
        assert (space[ws:] == 0xA5).all()
        check_backward(p, "exact", lse, (dx, dw, None, None), "e5m2", 64.0, np.array([0, M - 1]), np.array([0, V - 1]), (torch.bfloat16, torch.bfloat16))
        for call in (lambda s: p.forward(workspace=s), lambda s: p.backward(lse, workspace=s)):
            with pytest.raises(fm.Fp8Error, match="workspace"):
                call(space[:16])


def test_captured():
    """A captured forward and backward replayed with new hidden states and targets: each replay equals the eager calls."""
    announce("cross entropy captured")
    for M in (9, 150):
        p = Problem(M, 1500, 128)
        ws = torch.empty(fm.vocab_workspace_bytes(M, 1500, 128, 2), dtype=torch.uint8, device=device())
        one, inv = scalar(64.0), scalar(1 / 64.0)
        dev = device()

        def outputs():
            return [torch.full((M,), -3.0, device=dev), torch.full((M,), -3.0, device=dev), torch.full((M, 128), -3.0, dtype=torch.bfloat16, device=dev),
                    torch.full((1500, 128), -3.0, dtype=torch.bfloat16, device=dev), scalar(5.0), scalar(5, torch.int64)]

        def step(o):
            fm.fp8_vocab_cross_entropy(p.x, "e4m3", p.w, "e4m3", p.sx, p.sw, p.targets, o[0], o[1], workspace=ws)
            fm.fp8_vocab_cross_entropy_backward(p.x, "e4m3", p.w, "e4m3", p.sx, p.sw, p.targets, o[1], p.dloss, "e5m2", one, inv, dx=o[2], dw=o[3], amax=o[4], sat=o[5],
                                                workspace=ws)

        got = outputs()
        step(got)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(got)
        for k in range(4):
            other = Problem(M, 1500, 128, seed=10 * k + 7)
            p.x.copy_(other.x)
            p.targets.copy_(other.targets)
            for o in got:
                o.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            want = outputs()
            step(want)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_two_streams_at_once():
    announce("cross entropy on two streams")
    p = Problem(200, 3000, 256)
    want = p.forward()
    want_back = p.backward(want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(fm.vocab_workspace_bytes(200, 3000, 256), dtype=torch.uint8, device=device()) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for s, ws in zip(streams, spaces):
        with torch.cuda.stream(s):
            loss, lse = p.forward(workspace=ws)
            outs.append((loss, lse) + p.backward(lse, workspace=ws))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want + want_back))
