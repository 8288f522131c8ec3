"""Every tile shape of the dense GEMMs, ragged in M, N and K, in both modes and layouts (tile_cases.py; the CPU test
test_tile_choice.py asserts that these sizes select them).

Tolerances: exact mode 1e-5 * sum |a b| * sinv_a * sinv_b; FP8 cores gpu_helpers.mfma8_bound, for sampled rows (a
K-deep array an output); bf16 outputs half a step, 2^-8, of the value more.  Every shape adds an output's products in
the same order, so 64 of the rows on their own, which take a 64 x 128 tile, have the same bits."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
import tile_cases
from gpu_helpers import announce, device, f32, mfma8_bound, u8
from oracle import codec

pytestmark = pytest.mark.gpu
ACCUMS = ["exact", "mfma_fp8"]
SA, SB = np.float32(0.37), np.float32(2.5e-3)


def rand_codes(seed, shape, fmt):
    """Every finite code of the format, both signs."""
    g = torch.Generator(device=device()).manual_seed(seed)
    mag = torch.randint(0, codec.FORMATS[fmt].max_code + 1, shape, generator=g, device=device(), dtype=torch.uint8)
    return mag | (torch.randint(0, 2, shape, generator=g, device=device(), dtype=torch.uint8) << 7)


def values(q, fmt):
    table = torch.from_numpy(codec.decode(np.arange(256, dtype=np.uint8), fmt)).to(device())
    return table[q.long()]


def scalar(v):
    return torch.tensor([float(v)], dtype=torch.float32, device=device())


def product(a, fa, b, fb, out, accum, b_trans=False):
    c = torch.full((a.shape[0], b.shape[1 if b_trans else 0]), 7.0, dtype=out, device=device())
    fm.fp8_gemm(a, fa, b, fb, scalar(SA), scalar(SB), c, accum=accum, b_trans=b_trans)
    torch.cuda.synchronize()
    return c


def edge_rows(M, count):
    """Rows of every tile row, the first and the last of the product among them."""
    return np.unique(np.r_[0, M - 1, np.linspace(1, M - 2, count - 2).astype(int)])


def check_product(c, a, fa, b, fb, accum):
    s = float(SA) * float(SB)
    A, B = values(a, fa), values(b, fb).t().contiguous()
    want = (A @ B) * s
    if accum == "exact":
        bound = (A.abs() @ B.abs()) * (1e-5 * s)
        got = c.double()
    else:
        rows = edge_rows(a.shape[0], 12)
        bound = torch.from_numpy(np.concatenate([mfma8_bound(u8(a)[r:r + 1], fa, u8(b), fb, SA, SB) for r in rows])).to(device())
        rows = torch.from_numpy(rows).to(device())
        got, want = c[rows].double(), want[rows]
    if c.dtype == torch.bfloat16:
        bound = bound + torch.finfo(c.dtype).eps / 2 * (want.abs() + bound)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (bad.nonzero()[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


@pytest.mark.parametrize("accum", ACCUMS)
@pytest.mark.parametrize("out,fa,fb", [(torch.float32, "e4m3", "e4m3"), (torch.bfloat16, "e5m2", "e4m3"), (torch.float32, "e4m3", "e5m2")])
@pytest.mark.parametrize("case", tile_cases.PLAIN)
def test_plain(case, out, fa, fb, accum):
    M, N, K = case
    announce(f"tile {case} {fa}x{fb} {accum}")
    a, b = rand_codes(M + K, (M, K), fa), rand_codes(N + K, (N, K), fb)
    c = product(a, fa, b, fb, out, accum)
    check_product(c, a, fa, b, fb, accum)
    rows = torch.from_numpy(edge_rows(M, 64)).to(device())
    assert torch.equal(product(a[rows], fa, b, fb, out, accum), c[rows])


@pytest.mark.parametrize("accum", ACCUMS)
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("case", tile_cases.PLAIN_BT)
def test_b_stored_k_by_n(case, fa, accum):
    M, N, K = case
    announce(f"tile {case} b_trans {fa} {accum}")
    a, b = rand_codes(M + K, (M, K), fa), rand_codes(N + K, (N, K), "e4m3")
    c = product(a, fa, b.t().contiguous(), "e4m3", torch.float32, accum, b_trans=True)
    check_product(c, a, fa, b, "e4m3", accum)
    assert torch.equal(product(a, fa, b, "e4m3", torch.float32, accum), c)


@pytest.mark.parametrize("accum", ACCUMS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("case", tile_cases.PLAIN)
def test_requantised(case, fmt, accum):
    """Codes, amax and count of the re-quantising epilogue: those of the fp32 product and the cast, some saturating."""
    M, N, K = case
    announce(f"tile {case} requant {fmt} {accum}")
    a, b = rand_codes(M + K, (M, K), "e4m3"), rand_codes(N + K, (N, K), "e4m3")
    c = product(a, "e4m3", b, "e4m3", torch.float32, accum)
    scale = scalar(codec.FORMATS[fmt].max_value / (0.6 * c.abs().max().item()))
    outs = []
    for fused in (True, False):
        q = torch.full((M, N), 0xA5, dtype=torch.uint8, device=device())
        amax, sat = scalar(-1.0), torch.full((1,), 99, dtype=torch.int64, device=device())
        if fused:
            fm.fp8_gemm_requant(a, "e4m3", b, "e4m3", scalar(SA), scalar(SB), fmt, scale, q, amax=amax, sat=sat, accum=accum)
        else:
            fm.fp8_quantize(c, fmt, scale, q=q, amax=amax, sat=sat)
        torch.cuda.synchronize()
        outs.append((q, amax, sat))
    assert all(torch.equal(x, y) for x, y in zip(*outs)) and outs[0][2].item() > 0


def codes_of(vals):
    return torch.from_numpy(codec.encode(np.asarray(vals, dtype=np.float32), "e4m3")).to(device())


@pytest.mark.parametrize("accum", ACCUMS)
@pytest.mark.parametrize("case,b_trans", [(c, False) for c in tile_cases.LARGEST_K] + [(c, True) for c in tile_cases.LARGEST_KN_BT])
def test_largest_k(case, b_trans, accum):
    """Rows (b_trans: columns) of one power of two each: every partial sum is exact, so the result is K a b bit for bit."""
    M, N, K = case
    announce(f"tile {case} largest K b_trans={b_trans} {accum}")
    av, bv = 2.0 ** (np.arange(M) % 4 - 2), 2.0 ** (np.arange(N) % 3 - 1)
    a = torch.empty((M, K), dtype=torch.uint8, device=device())
    a.copy_(codes_of(av).view(-1, 1).expand(-1, K))
    b = torch.empty((K, N) if b_trans else (N, K), dtype=torch.uint8, device=device())
    b.copy_(codes_of(bv).view(1, -1).expand(K, -1) if b_trans else codes_of(bv).view(-1, 1).expand(-1, K))
    c = torch.full((M, N), float("nan"), dtype=torch.float32, device=device())
    fm.fp8_gemm(a, "e4m3", b, "e4m3", scalar(2.0 ** -3), scalar(2.0 ** -2), c, accum=accum, b_trans=b_trans)
    torch.cuda.synchronize()
    got = f32(c)
    del a, b, c
    torch.cuda.empty_cache()
    assert np.array_equal(got, (K * np.outer(av, bv) * 2.0 ** -5).astype(np.float32))
