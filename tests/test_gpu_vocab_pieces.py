"""The vocabulary's cross entropy in pieces: the longest hidden size, whose vocabulary is longer than one piece may be.
Tolerances as in test_gpu_vocab_cross_entropy.py."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from test_gpu_vocab_cross_entropy import Problem, check_backward, check_forward, check_product, gradient

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
