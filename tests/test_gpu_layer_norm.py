"""GPU parity of the layer norm with dropout and residual against the fp64 oracle.

Tolerances, derived before the first run (EW, REL, SUM, HALF as in test_gpu_feed_forward.py):
* h: the same two fp32 roundings and the type's: equal bits.
* the mean: a sum of N <= 40000 terms over at least 64 lanes is rounded less than 300 times: REL of the mean of |h|.
* rstd: the squares' sum likewise, REL, halved by the root; the mean's own error d changes the variance by d^2 only,
  (REL mean|h|)^2 against a variance that is never below 1e-4 of (mean |h|)^2 here: 4e-6, inside REL.
* y = (h - m) r w + b: the mean's error times r |w|, rstd's and four roundings on the product, EW on |b|.
* gradient: m and r are given; each of its three terms is good to REL (the two means) plus EW, then half a step.
* dweight, dbias: less than 1200 roundings on the sum of magnitudes: SUM."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from oracle import codec, model_ends as me
from test_gpu_feed_forward import EW, HALF, NORM_SHAPES, REL, SUM, check_close, check_codes, d64, randn, scalar, u8, workspace

pytestmark = pytest.mark.gpu
EPS = 1e-5
SEED, OFFSET = (5 << 33) + 77, (9 << 40) + 3


def rng(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device=device())


def factors(shape, p, seed=SEED, offset=OFFSET):
    """The oracle's factors as the fp32 numbers that the kernel multiplies with."""
    return torch.from_numpy(me.dropout_factors(shape, p, seed, offset).astype(np.float32)).to(device())


def norm_inputs(rows, cols, dtype, residual, bias, p, seed=0):
    x = randn(seed + 1, rows, cols, dtype=dtype)
    res = (randn(seed + 2, rows, cols, std=3.0, dtype=torch.float32) + 1).to(dtype) if residual else None
    w = (randn(seed + 3, cols, std=0.2, dtype=torch.float32) + 1).to(dtype)
    b = randn(seed + 4, cols, std=0.3, dtype=dtype) if bias else None
    h = x.float()
    if p:
        h = h * factors((rows, cols), p)
    if residual:
        h = h + res.float()
    return x, res, w, b, h.to(dtype)


def y_bound(h, m, r, w, b):
    """(y, its error bound)."""
    y, _, _ = me.layer_norm(h, w, b, np.float32(EPS))
    part = np.abs((h - m[:, None]) * r[:, None] * w)
    return y, REL * np.mean(np.abs(h), axis=1, keepdims=True) * r[:, None] * np.abs(w) + (2 * REL + EW) * part + EW * (0 if b is None else np.abs(b))


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual,bias,stats,fmt,p", [(True, True, True, "e4m3", 0.1), (False, False, False, "e5m2", 0.0), (True, True, False, "e4m3", 0.0),
                                                       (False, True, True, "e5m2", 0.7)])
def test_norm(rows, cols, dtype, residual, bias, stats, fmt, p):
    announce(f"layer norm {rows}x{cols} {dtype} residual={residual} bias={bias} stats={stats} {fmt} p={p}")
    x, res, w, b, h = norm_inputs(rows, cols, dtype, residual, bias, p)
    scale = 100.0 if fmt == "e4m3" else 9000.0                   # some values saturate
    q = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device=device())
    total = torch.full_like(x, 7.0) if residual or p else None
    mean, rstd = (torch.full((rows,), -1.0, device=device()) for _ in range(2))
    amax, sat = (scalar(-1.0), scalar(12345, torch.int64)) if stats else (None, None)
    fm.fp8_layernorm_quantize(x, w, b, EPS, fmt, scalar(scale), q, residual=res, sum_out=total, mean=mean, rstd=rstd, amax=amax, sat=sat, dropout=p,
                              rng=rng() if p else None, workspace=workspace(65536) if rows % 2 else None)
    torch.cuda.synchronize()
    if total is not None:
        assert torch.equal(total, h)
    H, W, B = d64(h), d64(w), None if b is None else d64(b)
    _, m, r = me.layer_norm(H, W, B, np.float32(EPS))
    check_close(d64(mean), m, REL * np.mean(np.abs(H), axis=1), "mean")
    check_close(d64(rstd), r, REL * r, "rstd")
    y, bound = y_bound(H, m, r, W, B)
    check_codes(q, y, bound, scale, fmt)
    if stats:
        top = np.abs(y).max()
        assert top - bound.max() <= amax.item() <= top + bound.max()
        lo, hi = (np.sum(np.abs(y) * scale > codec.FORMATS[fmt].max_value + s * (bound * scale + EW * np.abs(y) * scale)) for s in (1, -1))
        assert lo <= sat.item() <= hi


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(2000, 1024), (2049, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward(rows, cols, dtype, p):
    announce(f"layer norm backward {rows}x{cols} {dtype} p={p}")
    dy, w = randn(11, rows, cols, std=0.1, dtype=dtype), (randn(12, cols, std=0.2, dtype=torch.float32) + 1).to(dtype)
    h = (randn(13, rows, cols, std=2.0, dtype=torch.float32) + 0.5).to(dtype)
    mean = h.double().mean(1).float()
    rstd = torch.rsqrt(h.double().var(1, unbiased=False) + EPS).float()
    M, R = d64(mean)[:, None], d64(rstd)[:, None]
    dh, dw, db = me.layer_norm_grad(d64(dy), d64(h), d64(w), EPS, d64(mean), d64(rstd))
    g, a = np.abs(d64(dy) * d64(w)), np.abs((d64(h) - M) * R)
    mag = R * (g + np.mean(g, axis=1, keepdims=True) + a * np.mean(g * a, axis=1, keepdims=True))
    f = me.dropout_factors((rows, cols), p, SEED, OFFSET).astype(np.float32).astype(np.float64) if p else 1.0
    for dres in (None, randn(14, rows, cols, std=0.1, dtype=dtype)):
        want = dh if dres is None else dh + d64(dres)
        bound = REL * mag + EW * np.abs(want)
        outs = []
        for size in (64 << 20, cols * 8):                        # many partial rows, and a single pair
            dx, dbranch = torch.full_like(h, 7.0), torch.full_like(h, 7.0)
            dweight, dbias = (torch.full((cols,), 7.0, device=device()) for _ in range(2))
            fm.fp8_layernorm_backward(dy, h, mean, rstd, w, dx, dweight=dweight, dbias=dbias, dresidual=dres, dbranch=dbranch, dropout=p, rng=rng() if p else None,
                                      workspace=workspace(size))
            torch.cuda.synchronize()
            check_close(d64(dx), want, bound + HALF[dtype] * np.abs(want) * 1.001, "dx")
            check_close(d64(dbranch), want * f, bound * f + (EW + HALF[dtype] * 1.001) * np.abs(want * f), "dbranch")
            check_close(d64(dweight), dw, SUM * np.sum(np.abs(d64(dy)) * a, axis=0), "dweight")
            check_close(d64(dbias), db, SUM * np.sum(np.abs(d64(dy)), axis=0), "dbias")
            outs.append((dx, dbranch, dweight, dbias))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        alone = torch.full_like(h, 7.0)
        fm.fp8_layernorm_backward(dy, h, mean, rstd, w, alone, dresidual=dres)     # no sums, no branch, no workspace
        assert torch.equal(alone, outs[0][0])
        for which in ("dweight", "dbias"):                                         # either sum by itself: the same grid, the same bits
            v = torch.full((cols,), 7.0, device=device())
            fm.fp8_layernorm_backward(dy, h, mean, rstd, w, alone, dresidual=dres, workspace=workspace(64 << 20), **{which: v})
            assert torch.equal(v, outs[0][2 if which == "dweight" else 3])


def test_backward_against_differences():
    """The gradient of sum(dy * y) in h, weight and bias, y from the forward's own codes at a fine scale: E4M3 has 3 fraction bits, so the
    differences are taken of the oracle's y; the device's dh has to fit them to their own error, e^2 of the third derivative, under 1e-6."""
    announce("layer norm backward against differences")
    gen = np.random.default_rng(4)
    h, w, dy = gen.normal(size=(2, 16)), gen.normal(size=16) + 1, gen.normal(size=(2, 16))
    ht, wt, dyt = (torch.from_numpy(v.astype(np.float32)).to(device()) for v in (h, w, dy))
    h, w, dy = d64(ht), d64(wt), d64(dyt)
    _, m, r = me.layer_norm(h, w, None, EPS)
    dx = torch.empty_like(ht)
    fm.fp8_layernorm_backward(dyt, ht, torch.from_numpy(m.astype(np.float32)).to(device()), torch.from_numpy(r.astype(np.float32)).to(device()), wt, dx)
    e = 1e-4
    for i in range(2):
        for j in range(16):
            s = np.zeros_like(h)
            s[i, j] = e
            num = np.sum(dy * (me.layer_norm(h + s, w, None, EPS)[0] - me.layer_norm(h - s, w, None, EPS)[0])) / (2 * e)
            # fp32 m and r: a few 2^-24 on terms of the order of r |w| |dy| (1 + |a|) < 200
            assert abs(dx[i, j].item() - num) < 1e-6 + 200 * 16 * 2.0 ** -24


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 80), (7, 1040), (2, 16400)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [2.0 ** -16, 0.5, 1 - 2.0 ** -16])
def test_dropped_places(rows, cols, dtype, p):
    """The mask is the oracle's, value by value; dropped NaN and Inf are 0; a probability under half a step is none."""
    announce(f"dropout places {rows}x{cols} {dtype} p={p}")
    w = torch.ones(cols, dtype=dtype, device=device())
    q = torch.empty((rows, cols), dtype=torch.uint8, device=device())
    for seed, offset in ((0, 0), (-1, -1), (SEED, OFFSET)):
        x, total = torch.ones((rows, cols), dtype=dtype, device=device()), torch.full((rows, cols), 7.0, dtype=dtype, device=device())
        f = factors((rows, cols), p, seed, offset)
        fm.fp8_layernorm_quantize(x, w, None, EPS, "e4m3", scalar(1.0), q, sum_out=total, dropout=p, rng=rng(seed, offset))
        assert torch.equal(total, f.to(dtype))
        x[f == 0] = float("nan") if cols % 32 else float("inf")
        fm.fp8_layernorm_quantize(x, w, None, EPS, "e4m3", scalar(1.0), q, sum_out=total, dropout=p, rng=rng(seed, offset))
        assert torch.equal(total, f.to(dtype))
    fm.fp8_layernorm_quantize(x, w, None, EPS, "e4m3", scalar(1.0), q, sum_out=total, dropout=2.0 ** -18)
    assert torch.equal(total.nan_to_num(), x.nan_to_num())


@pytest.mark.parametrize("cols", [512, 4096, 16400])
@pytest.mark.parametrize("alias", ["x", "residual"])
def test_in_place(cols, alias):
    announce(f"layer norm in place {cols} {alias}")
    x, res, w, b, h = norm_inputs(9, cols, torch.bfloat16, True, True, 0.2)
    q1, q2 = (torch.empty((9, cols), dtype=torch.uint8, device=device()) for _ in range(2))
    kw = dict(residual=res, dropout=0.2, rng=rng())
    fm.fp8_layernorm_quantize(x, w, b, EPS, "e4m3", scalar(50.0), q1, sum_out=torch.empty_like(x), **kw)
    into = x if alias == "x" else res
    fm.fp8_layernorm_quantize(x, w, b, EPS, "e4m3", scalar(50.0), q2, sum_out=into, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(into, h)
    # the gradients over their own inputs
    _, m, r = me.layer_norm(d64(h), d64(w), None, EPS)
    m, r = (torch.from_numpy(v.astype(np.float32)).to(device()) for v in (m, r))
    dy, dres = randn(5, 9, cols), randn(6, 9, cols)
    dx, dbranch = torch.empty_like(h), torch.empty_like(h)
    back = dict(dropout=0.2, rng=rng())
    fm.fp8_layernorm_backward(dy, h, m, r, w, dx, dresidual=dres, dbranch=dbranch, **back)
    fm.fp8_layernorm_backward(dy, h, m, r, w, dres, dresidual=dres, dbranch=dy, **back)
    torch.cuda.synchronize()
    assert torch.equal(dx, dres) and torch.equal(dbranch, dy)


@pytest.mark.parametrize("cols", [512, 4096, 16400])
def test_special_rows(cols):
    """A constant row (variance 0) gives the bias, without eps NaN; an Inf and a NaN touch only their own rows."""
    announce(f"layer norm special rows {cols}")
    x = randn(21, 6, cols, dtype=torch.float32)
    x[1] = 4.0                                                   # its sum and mean are exact
    w, b = torch.ones(cols, device=device()), torch.full((cols,), 0.5, device=device())

    def run(t, eps):
        q = torch.empty(t.shape, dtype=torch.uint8, device=device())
        amax = scalar(0.0)
        fm.fp8_layernorm_quantize(t, w, b, eps, "e4m3", scalar(32.0), q, amax=amax)
        return u8(q), amax.item()

    q0, _ = run(x, EPS)
    assert np.all(codec.decode(q0[1], "e4m3") == 16.0)
    y = x.clone()
    y[2, 5], y[3, 7] = float("inf"), float("nan")
    q1, amax = run(y, EPS)
    assert np.array_equal(q1[[0, 1, 4, 5]], q0[[0, 1, 4, 5]]) and np.all((q1[[2, 3]] & 0x7F) == 0x7F) and np.isnan(amax)
    q2, _ = run(x, 0.0)
    assert np.all((q2[1] & 0x7F) == 0x7F) and not np.any((q2[[0, 2, 3, 4, 5]] & 0x7F) == 0x7F)


def test_empty():
    announce("layer norm empty")
    dev = device()
    for rows, cols in ((0, 64), (5, 0)):
        x, w = torch.empty((rows, cols), device=dev), torch.ones(cols, device=dev)
        q, amax, sat = torch.empty((rows, cols), dtype=torch.uint8, device=dev), scalar(5.0), scalar(7, torch.int64)
        fm.fp8_layernorm_quantize(x, w, w, EPS, "e4m3", scalar(1.0), q, amax=amax, sat=sat, workspace=workspace(4096))
        assert amax.item() == 0.0 and sat.item() == 0
        dw, db = (torch.full((cols,), 3.0, device=dev) for _ in range(2))
        stat = torch.empty(rows, device=dev)
        fm.fp8_layernorm_backward(x, x, stat, stat, w, x, dweight=dw, dbias=db)
        assert (dw == 0).all() and (db == 0).all()


def test_captured_with_a_new_offset_each_replay():
    """A captured forward and backward replayed several times, the offset changed in between: each replay equals the eager calls."""
    announce("layer norm captured")
    rows, cols, p = 300, 1040, 0.25
    x, res, w, b, _ = norm_inputs(rows, cols, torch.bfloat16, True, True, 0.0)
    dy, seeds, ws = randn(8, rows, cols), rng(), workspace(1 << 20)
    dev = device()

    def outputs():
        return dict(sum=torch.full_like(x, 7.0), q=torch.zeros((rows, cols), dtype=torch.uint8, device=dev), mean=torch.zeros(rows, device=dev),
                    rstd=torch.zeros(rows, device=dev), amax=scalar(0.0), dx=torch.zeros_like(x), dbranch=torch.zeros_like(x), dw=torch.zeros(cols, device=dev),
                    db=torch.zeros(cols, device=dev))

    def step(o, r):
        fm.fp8_layernorm_quantize(x, w, b, EPS, "e4m3", one, o["q"], residual=res, sum_out=o["sum"], mean=o["mean"], rstd=o["rstd"], amax=o["amax"], dropout=p, rng=r,
                                  workspace=ws)
        fm.fp8_layernorm_backward(dy, o["sum"], o["mean"], o["rstd"], w, o["dx"], dweight=o["dw"], dbias=o["db"], dbranch=o["dbranch"], dropout=p, rng=r, workspace=ws)

    one, got = scalar(40.0), outputs()
    step(got, seeds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, seeds)
    masks = []
    for k in range(4):
        seeds.copy_(rng(SEED, OFFSET + k))
        for t in got.values():
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = outputs()
        step(want, rng(SEED, OFFSET + k))
        torch.cuda.synchronize()
        for name in got:
            assert torch.equal(got[name], want[name]), (k, name)
        masks.append(got["dbranch"].clone())
    assert not torch.equal(masks[0], masks[1])


def test_on_a_side_stream_beside_another_call():
    """Two calls at once on two streams, each with its own workspace and outputs."""
    announce("layer norm on two streams")
    x, res, w, b, h = norm_inputs(513, 4096, torch.bfloat16, True, True, 0.1)
    one, seeds = scalar(40.0), rng()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o = dict(q=torch.zeros((513, 4096), dtype=torch.uint8, device=device()), total=torch.zeros_like(x), amax=scalar(0.0), ws=workspace(65536))
        outs.append(o)
    for s, o in zip(streams, outs):
        fm.fp8_layernorm_quantize(x, w, b, EPS, "e4m3", one, o["q"], residual=res, sum_out=o["total"], amax=o["amax"], dropout=0.1, rng=seeds, workspace=o["ws"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["q"], outs[1]["q"]) and torch.equal(outs[0]["total"], h) and torch.equal(outs[1]["total"], h)
    assert outs[0]["amax"].item() == outs[1]["amax"].item()


def test_more_than_2_31_elements():
    """Rows past element 2^31: their drops, sums, codes and gradients are the oracle's."""
    rows, cols, p = 131200, 16384, 0.5
    announce(f"layer norm {rows}x{cols}")
    dev = device()
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device=dev)
    last = randn(31, 3, cols)
    x[-3:] = last
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    fm.fp8_layernorm_quantize(x, w, None, EPS, "e4m3", scalar(40.0), q, sum_out=x, mean=mean, rstd=rstd, dropout=p, rng=rng())
    f = torch.from_numpy(me.dropout_factors((3, cols), p, SEED, OFFSET, first=(rows - 3) * cols // 8).astype(np.float32)).to(dev)
    h = (last.float() * f).bfloat16()
    assert torch.equal(x[-3:], h)
    H = d64(h)
    _, m, r = me.layer_norm(H, d64(w), None, np.float32(EPS))
    y, bound = y_bound(H, m, r, d64(w), None)
    check_codes(q[-3:], y, bound, 40.0, "e4m3")
    dbranch = torch.empty_like(x)
    fm.fp8_layernorm_backward(x, x, mean, rstd, w, x, dbranch=dbranch, dropout=p, rng=rng())     # dy = h, over itself
    # dbranch is drop(dh) rounded, dx is dh rounded: the ratio of what is kept is 2, exactly
    assert torch.equal(dbranch[-3:], (x[-3:].float() * f).bfloat16())
