"""The vocabulary's cross entropy in pieces: the longest hidden size, whose vocabulary is longer than one piece may be, the least
workspaces, more columns than one launch has, and what pieces and cut products leave (statistics, sums, either gradient alone).
Tolerances as in test_gpu_vocab_cross_entropy.py."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
import vocab_cases
import vocab_product_cases
from gpu_helpers import announce, device
from test_gpu_feed_forward import EW
from test_gpu_vocab_cross_entropy import Problem, check_backward, check_forward, check_product, decoded, gradient

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_one_piece_asked_for_where_there_are_two():
    """300 columns of 2^22 values: the longest piece is 256 columns, so the size for one piece holds dx's sums."""
    M, V, K = 17, 300, 1 << 22
    announce(f"cross entropy {M}x{V}x{K}, workspace of one piece")
    p = Problem(M, V, K)
    ws = torch.full((fm.vocab_workspace_bytes(M, V, K, 1),), 0xA5, dtype=torch.uint8, device=device())
    loss, lse = p.forward(workspace=ws)
    check_forward(p, "exact", loss, lse, np.arange(M))
    out = p.backward(lse, workspace=ws, scale=2000.0, types=(BF, BF))
    check_backward(p, "exact", lse, (None,) + out[1:], "e5m2", 2000.0, cols=np.array([0, 255, 256, V - 1]), types=(BF, BF))
    # dx at its first, middle and last columns
    d, err = gradient(p, "exact", lse, None, None, "e5m2", 2000.0)
    at = torch.cat([torch.arange(0, 64), torch.arange(K // 2, K // 2 + 64), torch.arange(K - 64, K)]).to(device())
    check_product(out[0][:, at], d, err, p.w[:, at].contiguous(), p.fw, p.sw, 2000.0, 1 / 2000.0, "e5m2", "exact", ("dx", BF))
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("M,V,K", [(1, 32000, 256), (3, 4100, 1040), (8, 70000, 64), (16, 9000, 48)])
def test_few_rows_with_the_least_that_holds_the_vocabulary(M, V, K):
    """A pair a row for every 128 columns, as documented, serves the vocabulary whole; half of it in two pieces; nothing behind it is touched."""
    announce(f"cross entropy of few rows {M}x{V}x{K}, least workspace of the whole vocabulary")
    p = Problem(M, V, K)
    up16 = lambda n: (n + 15) // 16 * 16  # noqa: E731
    for columns in (V, V // 2, 256):
        size = up16(M * 4) + up16(M * 8) + M * 8 * -(-columns // 128)
        space = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=device())
        loss, lse = p.forward(workspace=space[:size])
        check_forward(p, "exact", loss, lse, np.arange(M))
        assert (space[size:] == 0xA5).all()


def test_a_vocabulary_of_more_columns_than_one_launch_has():
    """2^30 + 300 columns: more threads than a launch takes, so two pieces, though the workspace holds more.  A row of x that is 1 at
    its first place makes each logit a code of the weight, one of nine in turn, so lse is a sum of nine terms: SUMS of it for the exponentials and
    their sums (a lane of the joining kernel adds 2^15 pairs, each tile's over 128 columns: 2^15 roundings of 2^-24 at most)."""
    announce("cross entropy 1 x (2^30 + 300) x 16")
    V, K = (1 << 30) + 300, 16
    codes = torch.arange(0x28, 0x31, dtype=torch.uint8, device=device())
    w = torch.zeros((V, K), dtype=torch.uint8, device=device())
    step = 9 << 24
    for v in range(0, V, step):
        n = min(step, V - v)
        w[v:v + n, 0] = codes.repeat(-(-n // 9))[:n]
    x = torch.zeros((1, K), dtype=torch.uint8, device=device())
    x[0, 0] = 0x38                                                                   # 1
    one, loss, lse = torch.ones(1, device=device()), torch.zeros(1, device=device()), torch.zeros(1, device=device())
    z = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
    count = np.array([len(range(i, V, 9)) for i in range(9)], dtype=np.float64)
    want = np.log(np.sum(count * np.exp(z)))
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=device())
    for target in (0, (1 << 29) + 5, V - 1):
        fm.fp8_vocab_cross_entropy(x, "e4m3", w, "e4m3", one, one, torch.tensor([target], device=device()), loss, lse, workspace=ws)
        tol = 2.0 ** -9 + 1e-5 + 32 * 2.0 ** -24 * want
        assert abs(lse.item() - want) <= tol and abs(loss.item() - (want - z[target % 9])) <= tol


def check_statistics(p, accum, lse, amax, sat, fmt, scale):
    """amax and the count against d of all rows and columns, in fp64 on the device.  The bound of a logit on the FP8 cores: a run of eight products
    loses less than 2^(E - 12) of each, E the exponent of the largest (gpu_helpers), so less than 8 2^-12 of that one, hence of the sum of magnitudes; then its fp32 sums."""
    a, s = decoded(p.x, p.fx), p.sx.double() * p.sw.double()
    part = 1e-5 if accum == "exact" or p.M <= 16 else 2.0 ** -9 + 2 * (p.K / 8 + 2) * 2.0 ** -24
    t, g, l = torch.from_numpy(p.t).to(device())[:, None], p.dloss.double()[:, None], lse.double()[:, None]
    live = (t >= 0) & (t < p.V)
    limit = 448.0 if fmt == "e4m3" else 57344.0
    low = high = 0.0
    least = most = 0
    for c in range(0, p.V, 1024):
        b = decoded(p.w[c:c + 1024], p.fw)
        z, B = a @ b.t() * s, part * (a.abs() @ b.abs().t()) * s
        hit = (t == torch.arange(c, c + b.shape[0], device=device())).double()
        prob = (z - l).exp()
        d = torch.where(live, (g * (prob - hit)).abs(), 0.0)
        err = torch.where(live, g.abs() * (prob * torch.expm1(B) + EW * (prob * (1 + (z - l).abs()) + hit)), 0.0)
        low, high = max(low, (d - err).max().item()), max(high, (d + err).max().item())
        least += ((d - err) * scale * (1 - 1e-6) > limit).sum().item()
        most += ((d + err) * scale * (1 + 1e-6) > limit).sum().item()
    assert low <= amax.item() * (1 + 1e-6) and amax.item() <= high * (1 + 1e-6), (low, amax.item(), high)
    assert least <= sat.item() <= most and most > 0, (least, sat.item(), most)


@pytest.mark.parametrize("M,V,K", list(vocab_cases.LOGITS) + [c for c in vocab_product_cases.CUT if c not in vocab_cases.LOGITS])
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_statistics_of_large_products(M, V, K, accum):
    """On every tile shape of the logits, in one launch and in two, in one piece and in several."""
    announce(f"cross entropy statistics {M}x{V}x{K} {accum}")
    p = Problem(M, V, K, seed=5)
    lse = p.forward(accum)[1]
    for pieces in (1, 2):
        _, _, amax, sat = p.backward(lse, accum, pieces, "e5m2", 30000.0, (BF, BF))
        check_statistics(p, accum, lse, amax, sat, "e5m2", 30000.0)


@pytest.mark.parametrize("case", vocab_product_cases.CUT)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_products_cut_in_two(case, accum):
    """Rows on either side of the cut: dx where earlier pieces are added to it, dw."""
    announce(f"cross entropy cut products {case} {accum}")
    M, V, K = case
    pieces, P, dx_cut, dw_cut = vocab_product_cases.CUT[case]
    p = Problem(M, V, K, seed=8)
    lse = p.forward(accum)[1]
    rows, cols = np.unique([0, dx_cut - 1, min(dx_cut, M - 1), M - 1]), np.unique([0, dw_cut - 1, min(dw_cut, V - 1), min(P + 1, V - 1), V - 1])
    for types in ((BF, BF), (torch.float32, torch.float32)):
        out = p.backward(lse, accum, pieces, "e5m2", 30000.0, types)
        check_backward(p, accum, lse, out, "e5m2", 30000.0, rows, cols, types)
        assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[1].float()).all()
        assert (out[0][torch.from_numpy((p.t < 0) | (p.t >= V)).to(device())] == 0).all()


@pytest.mark.parametrize("M,V,K", [(5, 2000, 4096), (33, 2500, 80), (130, 1515, 256), (300, 5000, 144)])
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_either_gradient_alone(M, V, K, accum):
    """The same bits as together, whatever the pieces: their length goes by the sizes and the workspace, not by what is asked for."""
    announce(f"cross entropy one gradient {M}x{V}x{K} {accum}")
    p = Problem(M, V, K)
    lse = p.forward(accum)[1]
    for pieces in (0, 1, 2, 3):
        for types in ((BF, torch.float32), (torch.float32, BF)):
            both = p.backward(lse, accum, pieces, "e5m2", 40000.0, types)
            dx = p.backward(lse, accum, pieces, "e5m2", 40000.0, (types[0], None))
            dw = p.backward(lse, accum, pieces, "e5m2", 40000.0, (None, types[1]))
            assert torch.equal(dx[0], both[0]) and torch.equal(dw[1], both[1]), (pieces, types)
            for alone in (dx, dw):
                assert torch.equal(alone[2], both[2]) and torch.equal(alone[3], both[3])


@pytest.mark.parametrize("M,V,K", [(300, 30001, 4096), (509, 116000, 1024)])
def test_short_products_of_many_tiles(M, V, K):
    """dw of three and four steps on the FP8 cores, whose tiles are more than seven a compute unit: the rows of the first and the last of them."""
    announce(f"cross entropy dw {M}x{V}x{K}")
    assert 256 < M <= 512 and -(-V // 256) * -(-K // 256) > 7 * 256
    p = Problem(M, V, K, seed=4)
    lse = p.forward("mfma_fp8")[1]
    cols = np.array([0, 255, V // 2, V - V % 256 - 1, V - 1])
    for types in ((None, BF), (None, torch.float32)):
        out = p.backward(lse, "mfma_fp8", 1, "e5m2", 20000.0, types)
        check_backward(p, "mfma_fp8", lse, out, "e5m2", 20000.0, cols=cols, types=types)
        assert torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("case", vocab_product_cases.SPLIT)
@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_split_products_of_several_pieces(case, accum):
    """dx's parts are joined and added to the sums of the pieces before."""
    announce(f"cross entropy split products {case} {accum}")
    M, V, K = case
    p = Problem(M, V, K, seed=6)
    lse = p.forward(accum)[1]
    rows, cols = np.array([0, 1, M // 2, M - 1]), np.array([0, 30207 % V, V - 1])
    for types in ((BF, BF), (torch.float32, torch.float32)):
        space = torch.full((vocab_product_cases.SPLIT[case][0] + 4096,), 0xA5, dtype=torch.uint8, device=device())
        out = p.backward(lse, accum, None, "e5m2", 20000.0, types, workspace=space[:-4096])
        assert (space[-4096:] == 0xA5).all()
        check_backward(p, accum, lse, out, "e5m2", 20000.0, rows, cols, types)
