"""GPU parity of the feed-forward operators against the fp64 oracle.

Tolerances, derived before the first run:
* GEMM results c: the library's bound, 1e-5 * sum|ab| * sinv_a * sinv_b (exact mode), or the FP8
  matrix cores' error model (gpu_helpers.mfma8_bound).
* fp32 arithmetic behind them: `EW` = 32 roundings of 2^-24 relative per elementwise chain (every chain
  here is shorter; exp and reciprocal count for a few), so 2e-6, on the magnitudes that enter it.
* norms: a sum of N terms over at least 64 lanes is rounded less than N/64 + 40 times; N <= 16400 gives
  less than 300 roundings, 2e-5 relative at worst, halved by the square root: REL = 2e-5.
* column sums (dweight, dbias): less than 1200 roundings of 2^-24 on the sum of magnitudes: 1e-4.
* the last rounding: half a step, torch.finfo(t).eps / 2 of the value (bf16 2^-8), and for FP8 codes the oracle's bracket
  of round_to_fp8(fp32(c * s)) over the interval c -+ bound.
Slopes: |silu'| < 1.1, |gelu'| < 1.13, |relu'| <= 1, |silu''|, |gelu''| < 1."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device, mfma8_bound
from oracle import codec, feed_forward as ff, gemm

pytestmark = pytest.mark.gpu
EW, REL, SUM = 2e-6, 2e-5, 1e-4
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}
LIP = 1.13


def d64(t):
    return t.detach().double().cpu().numpy()


def u8(t):
    return t.detach().cpu().numpy()


def scalar(v, dtype=torch.float32):
    return torch.tensor([v], dtype=dtype, device=device())


def randn(seed, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, std, shape).astype(np.float32)).to(dtype).to(device())


def rand_codes(seed, shape, fmt, low=0):
    """Codes of moderate magnitudes (a quarter of the exponent range below the top), both signs, some zeros."""
    rng = np.random.default_rng(seed)
    top = codec.FORMATS[fmt].max_code
    mag = rng.integers(top // 3, 2 * top // 3, size=shape)
    mag[rng.random(shape) < 0.05] = 0
    return torch.from_numpy((mag | (rng.integers(0, 2, size=shape) << 7)).astype(np.uint8)).to(device())


def workspace(n=64 << 20):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device=device())


def check_close(got, want, bound, what):
    got, want, bound = np.asarray(got), np.asarray(want), np.broadcast_to(bound, np.shape(want))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bound[bad][:4])


def check_codes(q, want, bound, scale, fmt, amax=None, sat=None):
    r = gemm.requant_bracket(want, bound, np.float32(scale), fmt)
    v = codec.decode(u8(q).reshape(want.shape), fmt)
    ok = (v >= r["lo"]) & (v <= r["hi"])
    assert ok.all(), (np.argwhere(~ok)[:4], v[~ok][:4], want[~ok][:4])
    if amax is not None:
        assert r["amax"][0] * (1 - 1e-7) <= amax.item() <= r["amax"][1] * (1 + 1e-7)
    if sat is not None:
        assert r["sat"][0] <= sat.item() <= r["sat"][1]


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORM_SHAPES = [(1, 16), (1, 4096), (5, 48), (3, 512), (7, 528), (9, 1024), (6, 1040), (257, 2048), (33, 4112), (5, 7168), (3, 16384),
               (3, 16400), (2, 40000)]


def norm_inputs(rows, cols, dtype, residual, seed=0):
    x = randn(seed + 1, rows, cols, dtype=dtype)
    res = randn(seed + 2, rows, cols, std=3.0, dtype=dtype) if residual else None
    w = (randn(seed + 3, cols, std=0.2, dtype=torch.float32) + 1).to(dtype)
    h = x if res is None else (x.float() + res.float()).to(dtype)   # one fp32 sum, one rounding
    return x, res, w, h


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual,stats,fmt", [(True, True, "e4m3"), (False, False, "e5m2"), (True, False, "e4m3"), (False, True, "e5m2")])
def test_norm(rows, cols, dtype, residual, stats, fmt):
    announce(f"norm {rows}x{cols} {dtype} residual={residual} stats={stats} {fmt}")
    x, res, w, h = norm_inputs(rows, cols, dtype, residual)
    scale = 100.0 if fmt == "e4m3" else 9000.0                   # some values saturate
    q = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device=device())
    total = torch.full_like(x, 7.0) if residual else None
    rstd = torch.full((rows,), -1.0, device=device())
    amax, sat = (scalar(-1.0), scalar(12345, torch.int64)) if stats else (None, None)
    fm.fp8_rmsnorm_quantize(x, w, 1e-5, fmt, scalar(scale), q, residual=res, sum_out=total, rstd=rstd, amax=amax, sat=sat,
                            workspace=workspace(65536) if rows % 2 else None)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(total, h)
    y, r = ff.rms_norm(d64(h), d64(w), np.float32(1e-5))
    check_close(d64(rstd), r, REL * r, "rstd")
    check_codes(q, y, REL * np.abs(y), scale, fmt, amax, sat)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_norm_blockwise(rows, cols, dtype, fmt):
    announce(f"norm blockwise {rows}x{cols} {dtype} {fmt}")
    x, res, w, h = norm_inputs(rows, cols, dtype, rows != 3)
    if cols >= 256:
        w[128:256] = 0                                           # a block of zeros has scale 1
    nb = (cols + 127) // 128
    q = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device=device())
    si = torch.full((rows, nb), -1.0, device=device())
    fm.fp8_rmsnorm_quantize_blockwise(x, w, 1e-5, fmt, q, si, residual=res, sum_out=torch.empty_like(x) if res is not None else None)
    torch.cuda.synchronize()
    y, _ = ff.rms_norm(d64(h), d64(w), np.float32(1e-5))
    top, half, tiny = codec.FORMATS[fmt].max_value, (2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3), (2.0 ** -10 if fmt == "e4m3" else 2.0 ** -17)
    inv, v = d64(si), codec.decode(u8(q), fmt)
    for b in range(nb):
        yb = y[:, b * 128:(b + 1) * 128]
        m = np.abs(yb).max(axis=1)
        want = np.where(m > 0, m / top, 1.0)
        check_close(inv[:, b], want, (REL + 4 * 2.0 ** -24) * want, "scale_inv")
        # half a step of the code, or of the smallest subnormals, at the block's scale
        check_close(v[:, b * 128:(b + 1) * 128] * inv[:, b:b + 1], yb, (half + 2 * REL) * np.abs(yb) + tiny * want[:, None], "codes")


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(2000, 1024), (2049, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_backward(rows, cols, dtype):
    announce(f"norm backward {rows}x{cols} {dtype}")
    dy, w = randn(11, rows, cols, std=0.1, dtype=dtype), (randn(12, cols, std=0.2, dtype=torch.float32) + 1).to(dtype)
    h = randn(13, rows, cols, std=2.0, dtype=dtype)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-5).float()
    dh, dw = ff.rms_norm_grad(d64(dy), d64(h), d64(w), 1e-5, d64(rstd))
    r = d64(rstd)[:, None]
    g = np.abs(d64(dy) * d64(w))
    mag = r * (g + np.abs(d64(h)) * r * r * np.mean(g * np.abs(d64(h)), axis=1, keepdims=True))
    for dres in (None, randn(14, rows, cols, std=0.1, dtype=dtype)):
        want = dh if dres is None else dh + d64(dres)
        outs = []
        for size in (64 << 20, cols * 4):                        # many partial rows, and a single one
            dx, dweight = torch.full_like(h, 7.0), torch.full((cols,), 7.0, device=device())
            fm.fp8_rmsnorm_backward(dy, h, rstd, w, dx, dweight=dweight, dresidual=dres, workspace=workspace(size))
            torch.cuda.synchronize()
            check_close(d64(dx), want, REL * mag + EW * np.abs(want) + HALF[dtype] * np.abs(want) * 1.001, "dx")
            check_close(d64(dweight), dw, SUM * np.sum(np.abs(d64(dy) * d64(h) * r), axis=0), "dweight")
            outs.append(dx)
        assert torch.equal(outs[0], outs[1])
        alone = torch.full_like(h, 7.0)
        fm.fp8_rmsnorm_backward(dy, h, rstd, w, alone, dresidual=dres)     # no dweight, no workspace
        assert torch.equal(alone, outs[0])


@pytest.mark.parametrize("cols", [512, 4096, 16400])
@pytest.mark.parametrize("alias", ["x", "residual"])
def test_norm_in_place(cols, alias):
    announce(f"norm in place {cols} {alias}")
    x, res, w, h = norm_inputs(9, cols, torch.bfloat16, True)
    q1, q2 = (torch.empty((9, cols), dtype=torch.uint8, device=device()) for _ in range(2))
    fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", scalar(50.0), q1, residual=res, sum_out=torch.empty_like(x))
    into = x if alias == "x" else res
    fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", scalar(50.0), q2, residual=res, sum_out=into)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(into, h)
    # the gradient over its own inputs
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-5).float()
    dy, dx = randn(5, 9, cols), torch.empty_like(h)
    fm.fp8_rmsnorm_backward(dy, h, rstd, w, dx, dresidual=dy)
    fm.fp8_rmsnorm_backward(dy, h, rstd, w, dy, dresidual=dy)
    torch.cuda.synchronize()
    assert torch.equal(dx, dy)


@pytest.mark.parametrize("cols", [512, 4096, 16400])
@pytest.mark.parametrize("blocks", [False, True])
def test_norm_special_rows(cols, blocks):
    """A zero row with eps, a zero row without (0 * Inf), an Inf and a NaN touch only their own rows."""
    announce(f"norm special rows {cols} blocks={blocks}")
    x = randn(21, 6, cols, dtype=torch.float32)
    x[1] = 0
    x[2, 5], x[3, 7] = float("inf"), float("nan")
    w = torch.ones(cols, device=device())

    def run(t, eps):
        q = torch.empty(t.shape, dtype=torch.uint8, device=device())
        amax = scalar(0.0)
        if blocks:
            fm.fp8_rmsnorm_quantize_blockwise(t, w, eps, "e4m3", q, torch.empty((t.shape[0], (cols + 127) // 128), device=device()))
        else:
            fm.fp8_rmsnorm_quantize(t, w, eps, "e4m3", scalar(40.0), q, amax=amax)
        torch.cuda.synchronize()
        return u8(q), amax.item()

    q, amax = run(x, 1e-5)
    clean, _ = run(torch.cat([x[:1], x[4:]]), 1e-5)
    assert np.array_equal(q[[0, 4, 5]], clean)
    assert np.all((q[1] & 0x7F) == 0)
    assert (q[2, 5] & 0x7F) == 0x7F and np.all((np.delete(q[2], 5) & 0x7F) == 0)      # Inf * 0 is NaN, finite * 0 is 0
    assert np.all((q[3] & 0x7F) == 0x7F)
    if not blocks:
        assert np.isnan(amax)
    q, _ = run(x[1:2], 0.0)
    assert np.all((q & 0x7F) == 0x7F)


# ---------------------------------------------------------------------------
# gated and fused products
# ---------------------------------------------------------------------------
# few-row kernel (<= 16), the three tile shapes, K split over the workspace (256 x 64 x 8192 and the like), ragged everything
# (beyond 16 rows these select 64 x 128 tiles, in two or three stages; test_gpu_tile_epilogues.py has the larger tiles, whole and split)
GEMM_SHAPES = [(1, 16, 16), (1, 48, 4096), (3, 40, 144), (16, 136, 1040), (16, 2064, 528), (17, 33, 272), (64, 64, 8192), (65, 200, 400),
               (130, 72, 4112), (200, 131, 144), (300, 300, 1040), (1100, 700, 272)]


def c_bound(a, fa, b, fb, sa, sb, accum):
    M, K = a.shape
    if accum == "exact" or M <= 16:
        return gemm.abs_bound(u8(a), fa, u8(b).T, fb, sa, sb)
    return mfma8_bound(u8(a), fa, u8(b), fb, sa, sb) + gemm.abs_bound(u8(a), fa, u8(b).T, fb, sa, sb)


def gemm_case(M, N, K, fa, fb, accum):
    a, b = rand_codes(M + K, (M, K), fa), rand_codes(N + 3 * K, (N, K), fb)
    one = gemm.dequant_gemm(u8(a), fa, u8(b).T, fb, 1.0, 1.0)
    sa = np.float32(2.5 / max(one.std(), 1e-30))
    sb = np.float32(0.75)
    return a, b, sa, sb, gemm.dequant_gemm(u8(a), fa, u8(b).T, fb, sa, sb), c_bound(a, fa, b, fb, sa, sb, accum)


def check_output(y, out, want, bound, scale, amax, sat):
    if out in ("e4m3", "e5m2"):
        check_codes(y, want, bound + EW * np.abs(want), scale, out, amax, sat)
    else:
        t = torch.bfloat16 if out == "bf16" else torch.float32
        check_close(d64(y), want, (bound + EW * np.abs(want)) * 1.01 + HALF[t] * np.abs(want) * 1.01, "y")


def new_output(M, N, out):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}.get(out, torch.uint8)
    y = torch.empty((M, N), dtype=t, device=device())
    y.view(torch.uint8).fill_(0xA5)
    return y


OUTS = [("bf16", "silu"), ("e4m3", "gelu"), ("f32", "relu"), ("e5m2", "none")]


@pytest.mark.parametrize("M,F,K", GEMM_SHAPES)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("out,act", OUTS)
def test_gated(M, F, K, accum, out, act):
    announce(f"gated {M}x{F}x{K} {accum} {out} {act}")
    fa, fb = ("e4m3", "e4m3") if out != "f32" else ("e5m2", "e4m3")
    a, b, sa, sb, gu, bnd = gemm_case(M, 2 * F, K, fa, fb, accum)
    g, u = gu[:, :F], gu[:, F:]
    v, _ = ff.activation(g, act)
    want = v * u
    bound = (LIP * bnd[:, :F] + EW * np.abs(g)) * np.abs(u) + np.abs(v) * bnd[:, F:] + LIP * bnd[:, :F] * bnd[:, F:]
    scale = 30.0 if out == "e4m3" else 4000.0
    fp8 = out in ("e4m3", "e5m2")
    for ws, save in ((workspace(), True), (None, False), (workspace(max(16, 2 * M * 2 * F * 4)), True)):
        h, z = new_output(M, F, out), torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device=device()) if save else None
        amax, sat = (scalar(-1.0), scalar(99, torch.int64)) if fp8 else (None, None)
        fm.fp8_gemm_gated(a, fa, b, fb, scalar(sa), scalar(sb), act, h, gu=z, out_fmt=out if fp8 else None,
                          out_scale=scalar(scale) if fp8 else None, amax=amax, sat=sat, accum=accum, workspace=ws)
        torch.cuda.synchronize()
        check_output(h, out, want, bound, scale, amax, sat)
        if save:
            check_close(d64(z), gu, (bnd + HALF[torch.bfloat16] * np.abs(gu)) * 1.01, "gu")


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("out,act", OUTS)
@pytest.mark.parametrize("with_bias,with_res", [(True, True), (False, False)])
def test_fused(M, N, K, accum, out, act, with_bias, with_res):
    announce(f"fused {M}x{N}x{K} {accum} {out} {act} bias={with_bias} residual={with_res}")
    fa, fb = ("e4m3", "e5m2") if out == "f32" else ("e4m3", "e4m3")
    a, b, sa, sb, c, bnd = gemm_case(M, N, K, fa, fb, accum)
    bias = randn(7, N) if with_bias else None
    res = randn(8, M, N, std=2.0) if with_res else None
    z = c + (d64(bias) if with_bias else 0.0)
    v, _ = ff.activation(z, act)
    want = v + (d64(res) if with_res else 0.0)
    bound = LIP * bnd + EW * (np.abs(c) + np.abs(z) + np.abs(v))
    scale = 60.0 if out == "e4m3" else 9000.0
    fp8 = out in ("e4m3", "e5m2")
    for ws, save in ((workspace(), True), (None, False), (workspace(max(16, 2 * M * N * 4)), True)):
        y, zk = new_output(M, N, out), torch.full((M, N), 7.0, dtype=torch.bfloat16, device=device()) if save else None
        amax, sat = (scalar(-1.0), scalar(99, torch.int64)) if fp8 else (None, None)
        fm.fp8_gemm_fused(a, fa, b, fb, scalar(sa), scalar(sb), y, bias=bias, act=act, residual=res, z=zk, out_fmt=out if fp8 else None,
                          out_scale=scalar(scale) if fp8 else None, amax=amax, sat=sat, accum=accum, workspace=ws)
        torch.cuda.synchronize()
        check_output(y, out, want, bound, scale, amax, sat)
        if save:
            check_close(d64(zk), z, (bnd + EW * np.abs(c) + HALF[torch.bfloat16] * np.abs(z)) * 1.01, "z")


@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("gated", [True, False])
def test_products_on_the_largest_tiles(gated, accum):
    """Enough rows, columns and K that the 256 x 256 tiles are chosen, all three ragged; every output in the exact mode,
    rows of every tile row on the FP8 cores (their error model takes a K-deep array per output)."""
    announce(f"largest tiles gated={gated} {accum}")
    M, N, K = 3590, 3600, 4112
    rng = np.random.default_rng(77)
    a, b = rand_codes(71, (M, K), "e4m3"), rand_codes(72, (N, K), "e4m3")
    rows = np.arange(M) if accum == "exact" else np.unique(np.r_[0, M - 1, np.arange(100, M, 256) + rng.integers(0, 100)])
    A = torch.from_numpy(codec.decode(u8(a)[rows], "e4m3")).to(device())
    B = torch.from_numpy(codec.decode(u8(b), "e4m3").T.copy()).to(device())
    c = (A @ B).cpu().numpy()
    sa, sb = np.float32(2.5 / c.std()), np.float32(0.75)
    s = np.float64(sa) * np.float64(sb)
    bnd = 1e-5 * s * (A.abs() @ B.abs()).cpu().numpy()
    del A, B
    if accum == "mfma_fp8":
        bnd = bnd + np.concatenate([mfma8_bound(u8(a)[r:r + 1], "e4m3", u8(b), "e4m3", sa, sb) for r in rows])
    c = c * s
    kw = dict(out_fmt="e4m3", out_scale=scalar(30.0), accum=accum, workspace=workspace())
    amax, sat = scalar(-1.0), scalar(99, torch.int64)
    z = torch.empty((M, N), dtype=torch.bfloat16, device=device())
    if gated:
        y = new_output(M, N // 2, "e4m3")
        fm.fp8_gemm_gated(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), "silu", y, gu=z, amax=amax, sat=sat, **kw)
        g, u = c[:, :N // 2], c[:, N // 2:]
        v, _ = ff.activation(g, "silu")
        want = v * u
        bound = (LIP * bnd[:, :N // 2] + EW * np.abs(g)) * np.abs(u) + np.abs(v) * bnd[:, N // 2:] + LIP * bnd[:, :N // 2] * bnd[:, N // 2:]
        zs = c
    else:
        y = new_output(M, N, "e4m3")
        bias, res = randn(73, N), randn(74, M, N)
        fm.fp8_gemm_fused(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), y, bias=bias, act="gelu", residual=res, z=z, amax=amax, sat=sat, **kw)
        zs = c + d64(bias)
        want = ff.activation(zs, "gelu")[0] + d64(res)[rows]
        bound = LIP * bnd + EW * (np.abs(c) + np.abs(zs) + np.abs(want))
    torch.cuda.synchronize()
    whole = accum == "exact"
    check_codes(y[torch.from_numpy(rows).to(device())], want, bound + EW * np.abs(want), 30.0, "e4m3", amax if whole else None, sat if whole else None)
    check_close(d64(z)[rows], zs, (bnd + EW * np.abs(c) + HALF[torch.bfloat16] * np.abs(zs)) * 1.01, "z")


def test_fused_residual_in_place_and_guarded_buffers():
    """residual may be y; nothing is written past y, z or the workspace that was handed over."""
    announce("fused in place")
    for M, N, K in ((5, 40, 144), (64, 72, 4096), (300, 200, 528)):
        a, b, sa, sb, _, _ = gemm_case(M, N, K, "e4m3", "e4m3", "exact")
        size = 3 * M * N * 4
        big = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=device())
        store = torch.full((2 * M * N + 512,), 7.0, dtype=torch.bfloat16, device=device())
        y, z = store[:M * N].view(M, N), store[M * N + 256:2 * M * N + 256].view(M, N)
        if z.data_ptr() % 16 or y.data_ptr() % 16:
            raise AssertionError("the test's views must be aligned")
        res = randn(9, M, N)
        apart = torch.empty_like(res)
        fm.fp8_gemm_fused(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), apart, act="gelu", residual=res, workspace=big[:size])
        y.copy_(res)
        fm.fp8_gemm_fused(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), y, act="gelu", residual=y, z=z, workspace=big[:size])
        torch.cuda.synchronize()
        assert torch.equal(apart, y)
        assert torch.all(store[M * N:M * N + 256] == 7.0) and torch.all(store[2 * M * N + 256:] == 7.0)
        assert torch.all(big[size:] == 0xA5)


def test_products_nonfinite_stay_in_their_rows_and_columns():
    announce("products nonfinite")
    for M in (8, 100):
        a, b, sa, sb, _, _ = gemm_case(M, 96, 272, "e4m3", "e4m3", "exact")
        clean = torch.empty((M, 48), dtype=torch.uint8, device=device())
        dirty, amax = torch.empty_like(clean), scalar(0.0)
        kw = dict(out_fmt="e4m3", out_scale=scalar(30.0), workspace=workspace())
        fm.fp8_gemm_gated(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), "silu", clean, **kw)
        a[3, 5], b[48 + 7, 9] = 0x7F, 0x7F                           # NaN codes: row 3, and column 7 through its up projection
        fm.fp8_gemm_gated(a, "e4m3", b, "e4m3", scalar(sa), scalar(sb), "silu", dirty, amax=amax, **kw)
        torch.cuda.synchronize()
        c, d = u8(clean), u8(dirty)
        assert np.all((d[3] & 0x7F) == 0x7F) and np.all((d[:, 7] & 0x7F) == 0x7F) and np.isnan(amax.item())
        keep = np.ones_like(c, bool)
        keep[3], keep[:, 7] = False, False
        assert np.array_equal(c[keep], d[keep])


def test_empty_products_report_zero():
    b, one = rand_codes(1, (32, 64), "e4m3"), scalar(1.0)
    for a, w in ((torch.empty((0, 64), dtype=torch.uint8, device=device()), b), (rand_codes(2, (4, 64), "e4m3"), b[:0])):
        amax, sat = scalar(3.0), scalar(3, torch.int64)
        fm.fp8_gemm_fused(a, "e4m3", w, "e4m3", one, one, torch.empty((a.shape[0], w.shape[0]), dtype=torch.uint8, device=device()),
                          out_fmt="e4m3", out_scale=one, amax=amax, sat=sat)
        assert amax.item() == 0.0 and sat.item() == 0
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=device())
    w = torch.ones(64, dtype=torch.bfloat16, device=device())
    for ws in (None, workspace(4096)):
        amax = scalar(3.0)
        fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", one, torch.empty((0, 64), dtype=torch.uint8, device=device()), amax=amax, workspace=ws)
        assert amax.item() == 0.0
        dw, db, amax = torch.full((64,), 5.0, device=device()), torch.full((64,), 5.0, device=device()), scalar(3.0)
        fm.fp8_rmsnorm_backward(x, x, torch.empty(0, device=device()), w, x, dweight=dw, workspace=ws)
        fm.fp8_act_backward(x, None, "none", "e5m2", one, q=torch.empty((0, 64), dtype=torch.uint8, device=device()), dbias=db, amax=amax, workspace=ws)
        assert torch.all(dw == 0) and torch.all(db == 0) and amax.item() == 0.0


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 in the activations, the codes and the outputs."""
    announce("offsets past 32 bits")
    rows, cols = 131136, 16384                                        # 2.1e9 elements
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=device())
    x[-3:] = randn(1, 3, cols)
    w = torch.ones(cols, dtype=torch.bfloat16, device=device())
    q = torch.zeros((rows, cols), dtype=torch.uint8, device=device())
    fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", scalar(50.0), q)
    y, _ = ff.rms_norm(d64(x[-3:]), d64(w), np.float32(1e-5))
    check_codes(q[-3:], y, REL * np.abs(y), 50.0, "e4m3")
    qt = torch.zeros((cols, rows), dtype=torch.uint8, device=device())
    db = torch.empty(cols, device=device())
    q.zero_()
    fm.fp8_act_backward(x, None, "none", "e4m3", scalar(50.0), q=q, q_t=qt, dbias=db, workspace=workspace())
    d = d64(x[-3:])
    check_codes(q[-3:], d, EW * np.abs(d), 50.0, "e4m3")
    assert torch.equal(qt[:, -3:].t(), q[-3:])
    check_close(d64(db), d.sum(0), SUM * np.abs(d).sum(0), "dbias")
    del qt, x
    b = rand_codes(4, (cols, 16), "e4m3")
    a = torch.zeros((rows, 16), dtype=torch.uint8, device=device())
    a[-3:] = rand_codes(5, (3, 16), "e4m3")
    bias = randn(6, cols)
    fm.fp8_gemm_fused(a, "e4m3", b, "e4m3", scalar(1.0), scalar(0.01), q, bias=bias, out_fmt="e4m3", out_scale=scalar(30.0), accum="mfma_fp8")
    c = gemm.dequant_gemm(u8(a[-3:]), "e4m3", u8(b).T, "e4m3", 1.0, np.float32(0.01)) + d64(bias)
    bnd = mfma8_bound(u8(a[-3:]), "e4m3", u8(b), "e4m3", 1.0, np.float32(0.01)) + EW * np.abs(c) + 1e-6
    check_codes(q[-3:], c, bnd, 30.0, "e4m3")


# ---------------------------------------------------------------------------
# gradients of the epilogues
# ---------------------------------------------------------------------------
BACK_SHAPES = [(16, 16), (48, 144), (128, 128), (272, 400), (1040, 256), (144, 2064)]


@pytest.mark.parametrize("M,N", BACK_SHAPES + [(1, 32), (37, 144)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype,fmt", [(torch.bfloat16, "e5m2"), (torch.float32, "e4m3")])
def test_act_backward(M, N, act, dtype, fmt):
    announce(f"act backward {M}x{N} {act} {dtype} {fmt}")
    dy, z = randn(31, M, N, std=0.05, dtype=dtype), randn(32, M, N, std=2.0)
    d = d64(dy) * ff.activation(d64(z), act)[1]
    bound = EW * np.abs(d64(dy)) * (1 + np.abs(d64(z)))
    scale = 3000.0 if fmt == "e4m3" else 500000.0
    trans = M % 16 == 0
    codes = []
    for size in (64 << 20, N * 4 + 16, N * 4):
        q = torch.full((M, N), 0xA5, dtype=torch.uint8, device=device())
        qt = torch.full((N, M), 0x5A, dtype=torch.uint8, device=device()) if trans else None
        db, amax, sat = torch.full((N,), 7.0, device=device()), scalar(-1.0), scalar(77, torch.int64)
        fm.fp8_act_backward(dy, None if act == "none" else z, act, fmt, scalar(scale), q=q, q_t=qt, dbias=db, amax=amax, sat=sat,
                            workspace=workspace(size))
        torch.cuda.synchronize()
        check_codes(q, d, bound, scale, fmt, amax, sat)
        check_close(d64(db), d.sum(0), SUM * np.abs(d).sum(0) + bound.sum(0), "dbias")
        if trans:
            assert torch.equal(qt.t(), q)
        codes.append(q)
    assert torch.equal(codes[0], codes[1]) and torch.equal(codes[0], codes[2])
    q = torch.full((M, N), 0xA5, dtype=torch.uint8, device=device())
    fm.fp8_act_backward(dy, None if act == "none" else z, act, fmt, scalar(scale), q=q)       # nothing but the codes
    assert torch.equal(q, codes[0])
    if trans:
        qt = torch.full((N, M), 0x5A, dtype=torch.uint8, device=device())
        fm.fp8_act_backward(dy, None if act == "none" else z, act, fmt, scalar(scale), q_t=qt)
        assert torch.equal(qt.t(), codes[0])


@pytest.mark.parametrize("M,F", BACK_SHAPES + [(1, 16), (35, 144)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype,fmt", [(torch.bfloat16, "e5m2"), (torch.float32, "e4m3")])
def test_gated_backward(M, F, act, dtype, fmt):
    announce(f"gated backward {M}x{F} {act} {dtype} {fmt}")
    dh, gu = randn(41, M, F, std=0.05, dtype=dtype), randn(42, M, 2 * F, std=2.0)
    g, u = d64(gu[:, :F]), d64(gu[:, F:])
    dg, du = ff.gated_grad(d64(dh), g, u, act)
    d = np.concatenate([dg, du], 1)
    bound = EW * np.abs(np.concatenate([d64(dh) * u * (1 + np.abs(g)), d64(dh) * (1 + np.abs(g))], 1))
    scale = 2000.0 if fmt == "e4m3" else 300000.0
    q = torch.full((M, 2 * F), 0xA5, dtype=torch.uint8, device=device())
    qt = torch.full((2 * F, M), 0x5A, dtype=torch.uint8, device=device()) if M % 16 == 0 else None
    amax, sat = scalar(-1.0), scalar(77, torch.int64)
    fm.fp8_gated_backward(dh, gu, act, fmt, scalar(scale), q=q, q_t=qt, amax=amax, sat=sat, workspace=workspace(65536) if M % 3 else None)
    torch.cuda.synchronize()
    check_codes(q, d, bound, scale, fmt, amax, sat)
    if qt is not None:
        assert torch.equal(qt.t(), q)


def test_act_backward_extreme_values():
    """Huge and infinite z: the slopes' limits, with no NaN made out of 0 * Inf for finite z; a NaN stays in its place."""
    z = torch.tensor([0.0, 30.0, -30.0, 1e20, -1e20, 3e38, -3e38, float("nan")] + [1.0] * 8, device=device()).bfloat16().repeat(16, 1)
    dy = torch.ones((16, 16), dtype=torch.bfloat16, device=device())
    for act in ("silu", "gelu"):
        q, amax = torch.empty((16, 16), dtype=torch.uint8, device=device()), scalar(0.0)
        fm.fp8_act_backward(dy, z, act, "e4m3", scalar(1.0), q=q, amax=amax)
        v = codec.decode(u8(q), "e4m3")
        assert np.allclose(v[:, :7], [0.5, 1, 0, 1, 0, 1, 0]) and np.all(np.isnan(v[:, 7])) and np.all(np.isfinite(v[:, 8:]))
        assert np.isnan(amax.item())


# ---------------------------------------------------------------------------
# how a program has them
# ---------------------------------------------------------------------------
def test_refusals_on_the_device():
    a, b, one = rand_codes(1, (4, 32), "e4m3"), rand_codes(2, (8, 32), "e4m3"), scalar(1.0)
    y = torch.empty((4, 8), dtype=torch.bfloat16, device=device())
    good = dict(a=a, fa="e4m3", b=b, fb="e4m3", sinv_a=one, sinv_b=one, y=y)
    fm.fp8_gemm_fused(**good)
    for exc, change in ((ValueError, dict(a=a.t())), (TypeError, dict(a=a.view(torch.int8))), (ValueError, dict(y=y[:3])),
                        (ValueError, dict(y=torch.empty((8, 4), dtype=torch.bfloat16, device=device()).t())), (TypeError, dict(y=y.half())),
                        (ValueError, dict(fa="e3m4")), (ValueError, dict(act="tanh")), (ValueError, dict(accum="fast")),
                        (ValueError, dict(sinv_a=torch.ones(2, device=device()))), (TypeError, dict(bias=torch.ones(8, device=device()))),
                        (ValueError, dict(residual=y[:, :4])), (ValueError, dict(bias=torch.ones(8, dtype=torch.bfloat16))),
                        (fm.Fp8Error, dict(amax=one)), (TypeError, dict(out_fmt="e4m3", out_scale=one)),
                        (ValueError, dict(workspace=torch.empty(64, dtype=torch.uint8)))):
        with pytest.raises(exc):
            fm.fp8_gemm_fused(**dict(good, **change))
    with pytest.raises(ValueError):
        fm.fp8_gemm_gated(a, "e4m3", b[:7], "e4m3", one, one, "silu", y[:, :3].contiguous())
    x = torch.zeros((4, 40), dtype=torch.bfloat16, device=device())
    with pytest.raises(fm.Fp8Error, match="alignment"):
        fm.fp8_rmsnorm_quantize(x, x[0].contiguous(), 1e-5, "e4m3", one, torch.empty((4, 40), dtype=torch.uint8, device=device()))
    with pytest.raises(fm.Fp8Error, match="workspace"):
        h = torch.zeros((4, 32), device=device())
        fm.fp8_rmsnorm_backward(h, h, torch.ones(4, device=device()), h[0].contiguous(), torch.empty_like(h), dweight=torch.empty(32, device=device()),
                                workspace=torch.empty(64, dtype=torch.uint8, device=device()))


def block(T, H, F, accum="exact"):
    """A feed-forward block with its inputs, its scales settled by one step."""
    ffn = fm.Fp8FeedForward(T, H, F, accum=accum, device=device())
    d = dict(x=randn(1, T, H), residual=randn(2, T, H, std=2.0), weight=(randn(3, H, std=0.1) + 1).bfloat16(),
             w_gu=randn(4, 2 * F, H, std=0.05), w_d=randn(5, H, F, std=0.05), dy=randn(6, T, H, std=0.01))
    o = dict(y=torch.empty((T, H), dtype=torch.bfloat16, device=device()), dx=torch.empty((T, H), dtype=torch.bfloat16, device=device()),
             dweight=torch.empty(H, device=device()), dw_gu=torch.empty((2 * F, H), device=device()), dw_d=torch.empty((H, F), device=device()))

    def step(stream=None):
        ffn.quantize_weights(d["w_gu"], d["w_d"], stream=stream)
        ffn.forward(d["x"], d["residual"], d["weight"], o["y"], stream=stream)
        if T % 16 == 0:
            ffn.backward(d["dy"], d["weight"], o["dx"], o["dweight"], o["dw_gu"], o["dw_d"], stream=stream)
        ffn.update(stream=stream)

    step()
    return ffn, d, o, step


@pytest.mark.parametrize("T,accum", [(1, "exact"), (7, "exact"), (48, "exact"), (320, "exact"), (320, "mfma_fp8")])
def test_feed_forward_block(T, accum):
    """The operators together, as one block: outputs and gradients against the unquantised block in fp64, to the error
    of the casts: E4M3 rounds by at most 2^-4 relative (rms 2^-4 / sqrt(3) and less), E5M2 by 2^-3; four E4M3 and two
    E5M2 casts stand between the inputs and any output, so the relative error in the 2-norm stays below
    sqrt(4 * 2^-8 / 3 + 2 * 2^-6 / 3) = 0.125 of what the casts touch."""
    announce(f"feed-forward block {T} {accum}")
    H, F = 256, 400
    ffn, d, o, step = block(T, H, F, accum)
    step()
    torch.cuda.synchronize()
    x, w, wgu, wd = d64(d["x"]), d64(d["weight"]), d64(d["w_gu"]), d64(d["w_d"])
    s = d64((d["x"].float() + d["residual"].float()).bfloat16())
    n, _ = ff.rms_norm(s, w, 1e-5)
    g, u = n @ wgu[:F].T, n @ wgu[F:].T
    h = ff.gated(g, u, "silu")
    branch = h @ wd.T

    def rel(got, want):
        return np.linalg.norm(got - want) / np.linalg.norm(want)

    got = d64(o["y"])
    assert rel(got - s, branch) < 0.125 + 2.0 ** -8 * np.linalg.norm(s + branch) / np.linalg.norm(branch)
    if T % 16:
        return
    dy = d64(d["dy"])
    dg, du = ff.gated_grad(dy @ wd, g, u, "silu")
    dn = dg @ wgu[:F] + du @ wgu[F:]
    ds, dw = ff.rms_norm_grad(dn, s, w, 1e-5)
    assert rel(d64(o["dw_d"]), dy.T @ h) < 0.125
    assert rel(d64(o["dw_gu"]), np.concatenate([dg.T @ n, du.T @ n])) < 0.125
    assert rel(d64(o["dweight"]), dw) < 0.125
    assert rel(d64(o["dx"]) - dy, ds) < 0.125 + 2.0 ** -8 * np.linalg.norm(ds + dy) / np.linalg.norm(ds)


def test_feed_forward_graph_replays_match_eager():
    """A whole training step of the block in a HIP graph: every replay gives the bits of the same step run eagerly,
    with eager work and synchronisations between the replays, and junk in the outputs beforehand."""
    announce("feed-forward graph")
    _, _, oe, eager = block(96, 256, 272)
    ffn, d, og, step = block(96, 256, 272)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for replay in range(4):
        for t in og.values():
            t.fill_(float(replay))
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for k in og:
            assert torch.equal(og[k], oe[k]), (replay, k)
        torch.zeros(1 << 20, device=device()).add_(1.0).sum().item()


def test_feed_forward_on_another_stream_is_repeatable():
    """Handed a stream that is not the current one, the block's results are those of the current stream, bit for bit,
    and the same from call to call (no sum depends on the order of atomics)."""
    announce("feed-forward stream")
    _, _, o1, step1 = block(160, 256, 528)
    _, _, o2, step2 = block(160, 256, 528)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        step1()
        step2(stream=s)
        torch.cuda.synchronize()
        for k in o1:
            assert torch.equal(o1[k], o2[k]), k
