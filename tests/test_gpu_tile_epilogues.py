"""The gated product and the product with epilogue on every tile shape, whole and split along K, ragged in M, N and K,
in both modes (tile_cases.EPILOGUE; the CPU test test_tile_choice.py asserts that these sizes select them).

Tolerances, as in test_gpu_feed_forward.py: the product within 1e-5 * sum |a b| * sinv_a * sinv_b (exact) or
gpu_helpers.mfma8_bound (FP8 cores, for sampled rows); 32 roundings of 2^-24 (EW) on each value of the elementwise
chain behind it; half a step of the output's type.  Slopes: |silu'| < 1.1, |gelu'| < 1.13 (LIP)."""

import functools

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
import tile_cases
from gpu_helpers import announce, device, mfma8_bound, u8
from oracle import codec, feed_forward as ff, gemm

pytestmark = pytest.mark.gpu
EW, LIP = 2e-6, 1.13
HALF = torch.finfo(torch.bfloat16).eps / 2
SB = np.float32(0.75)


def rand_codes(seed, shape, fmt):
    """Codes of moderate magnitudes (a quarter of the exponent range below the top), both signs."""
    top = codec.FORMATS[fmt].max_code
    g = torch.Generator(device=device()).manual_seed(seed)
    mag = torch.randint(top // 3, 2 * top // 3, shape, generator=g, device=device(), dtype=torch.uint8)
    return mag | (torch.randint(0, 2, shape, generator=g, device=device(), dtype=torch.uint8) << 7)


def randn(seed, *shape):
    g = torch.Generator(device=device()).manual_seed(seed)
    return torch.randn(shape, generator=g, device=device()).bfloat16()


def scalar(v, dtype=torch.float32):
    return torch.tensor([v], dtype=dtype, device=device())


@functools.lru_cache(maxsize=1)
def product(case, accum):
    """Codes, inverse scales, and for the rows that are checked (all of them in the exact mode) the product and its bound."""
    M, N, K = case
    a, b = rand_codes(M + K, (M, K), "e4m3"), rand_codes(N + K, (N, K), "e4m3")
    rows = np.arange(M) if accum == "exact" else np.unique(np.r_[0, M - 1, np.linspace(1, M - 2, 6).astype(int)])
    table = torch.from_numpy(codec.decode(np.arange(256, dtype=np.uint8), "e4m3")).to(device())
    A, B = table[a[torch.from_numpy(rows).to(device())].long()], table[b.long()].t().contiguous()
    c, mag = (A @ B).cpu().numpy(), (A.abs() @ B.abs()).cpu().numpy()
    sa = np.float32(2.5 / c.std())
    s = np.float64(sa) * np.float64(SB)
    bound = 1e-5 * s * mag
    if accum == "mfma_fp8":
        bound = bound + np.concatenate([mfma8_bound(u8(a)[r:r + 1], "e4m3", u8(b), "e4m3", sa, SB) for r in rows])
    return a, b, scalar(float(sa)), scalar(float(SB)), rows, c * s, bound


def check(y, z, rows, want, bound, zs, zbound, out, scale, amax, sat):
    on = torch.from_numpy(rows).to(device())
    whole = len(rows) == y.shape[0]
    got = y[on]
    if out == "bf16":
        bad = ~(np.abs(got.double().cpu().numpy() - want) <= bound + HALF * (np.abs(want) + bound))
    else:
        r = gemm.requant_bracket(want, bound, np.float32(scale), out)
        v = codec.decode(u8(got), out)
        bad = ~((v >= r["lo"]) & (v <= r["hi"]))
        if whole:
            assert r["amax"][0] * (1 - 1e-7) <= amax.item() <= r["amax"][1] * (1 + 1e-7)
            assert r["sat"][0] <= sat.item() <= r["sat"][1]
    assert not bad.any(), np.argwhere(bad)[:4]
    if z is not None:
        bad = ~(np.abs(z[on].double().cpu().numpy() - zs) <= zbound + HALF * (np.abs(zs) + zbound))
        assert not bad.any(), np.argwhere(bad)[:4]


def outputs(M, N, out):
    y = torch.empty((M, N), dtype=torch.bfloat16 if out == "bf16" else torch.uint8, device=device())
    y.view(torch.uint8).fill_(0xA5)
    return y


def guarded():
    """A workspace of the cases' size, and the bytes behind it."""
    big = torch.full((tile_cases.WORKSPACE + 4096,), 0xA5, dtype=torch.uint8, device=device())
    return big[:tile_cases.WORKSPACE], big[tile_cases.WORKSPACE:]


@pytest.mark.parametrize("out,act", [("e4m3", "silu"), ("bf16", "gelu"), ("e5m2", "relu")])
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("case", tile_cases.EPILOGUE)
def test_gated(case, accum, out, act):
    announce(f"tile gated {case} {accum} {out} {act}")
    M, N, K = case
    F = N // 2
    a, b, sa, sb, rows, c, bnd = product(case, accum)
    ws, behind = guarded()
    h, gu = outputs(M, F, out), torch.full((M, N), 7.0, dtype=torch.bfloat16, device=device())
    scale = 30.0 if out == "e4m3" else 4000.0
    fp8 = out != "bf16"
    amax, sat = (scalar(-1.0), scalar(99, torch.int64)) if fp8 else (None, None)
    fm.fp8_gemm_gated(a, "e4m3", b, "e4m3", sa, sb, act, h, gu=gu, out_fmt=out if fp8 else None, out_scale=scalar(scale) if fp8 else None,
                      amax=amax, sat=sat, accum=accum, workspace=ws)
    torch.cuda.synchronize()
    g, u, bg, bu = c[:, :F], c[:, F:], bnd[:, :F], bnd[:, F:]
    v, _ = ff.activation(g, act)
    want = v * u
    bound = (LIP * bg + EW * np.abs(g)) * np.abs(u) + np.abs(v) * bu + LIP * bg * bu + EW * np.abs(want)
    check(h, gu, rows, want, bound, c, bnd + EW * np.abs(c), out, scale, amax, sat)
    assert torch.all(behind == 0xA5)


@pytest.mark.parametrize("out,act,extras", [("e4m3", "gelu", True), ("bf16", "silu", True), ("e5m2", "none", False)])
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("case", tile_cases.EPILOGUE)
def test_fused(case, accum, out, act, extras):
    announce(f"tile fused {case} {accum} {out} {act} bias, residual and z: {extras}")
    M, N, K = case
    a, b, sa, sb, rows, c, bnd = product(case, accum)
    ws, behind = guarded()
    bias, res = (randn(7, N), randn(8, M, N)) if extras else (None, None)
    y = outputs(M, N, out)
    zk = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=device()) if extras else None
    scale = 60.0 if out == "e4m3" else 9000.0
    fp8 = out != "bf16"
    amax, sat = (scalar(-1.0), scalar(99, torch.int64)) if fp8 else (None, None)
    fm.fp8_gemm_fused(a, "e4m3", b, "e4m3", sa, sb, y, bias=bias, act=act, residual=res, z=zk, out_fmt=out if fp8 else None,
                      out_scale=scalar(scale) if fp8 else None, amax=amax, sat=sat, accum=accum, workspace=ws)
    torch.cuda.synchronize()
    z = c + (bias.double().cpu().numpy() if extras else 0.0)
    v, _ = ff.activation(z, act)
    want = v + (res.double().cpu().numpy()[rows] if extras else 0.0)
    chain = EW * (np.abs(c) + np.abs(z) + np.abs(v) + np.abs(want))
    check(y, zk, rows, want, LIP * bnd + chain, z, bnd + EW * (np.abs(c) + np.abs(z)), out, scale, amax, sat)
    assert torch.all(behind == 0xA5)
