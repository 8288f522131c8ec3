"""The layer norm's gradient at sizes that its other tests leave out: columns of which one launch cannot sum all."""

import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from test_gpu_feed_forward import EW

pytestmark = pytest.mark.gpu


def test_sums_of_more_columns_than_one_launch_has():
    """2 rows of 2^25 + 48 columns, two partial rows: dbias is the sum of two bf16 values, dweight of two products of a few roundings each (EW)."""
    rows, cols = 2, (1 << 25) + 48
    announce(f"layer norm backward {rows}x{cols}")
    g = torch.Generator(device=device()).manual_seed(3)
    dy, h = (torch.randn(rows, cols, generator=g, device=device()).bfloat16() for _ in range(2))
    mean, rstd = torch.tensor([0.25, -0.5], device=device()), torch.tensor([1.5, 0.75], device=device())
    w = torch.ones(cols, dtype=torch.bfloat16, device=device())
    dx = torch.empty_like(dy)
    want_w, mag = torch.zeros(cols, dtype=torch.float64, device=device()), torch.zeros(cols, dtype=torch.float64, device=device())
    for r in range(rows):
        term = dy[r].double() * (h[r].double() - mean[r].item()) * rstd[r].item()
        want_w += term
        mag += term.abs()
    want_b = dy.double().sum(0)
    for names in (("dweight", "dbias"), ("dbias",)):
        out = {n: torch.full((cols,), -3.0, device=device()) for n in names}
        ws = torch.full((rows * len(names) * cols * 4,), 0xA5, dtype=torch.uint8, device=device())
        fm.fp8_layernorm_backward(dy, h, mean, rstd, w, dx, workspace=ws, **out)
        assert ((out["dbias"].double() - want_b).abs() <= 2.0 ** -24 * want_b.abs()).all()
        if "dweight" in out:
            assert ((out["dweight"].double() - want_w).abs() <= EW * mag).all()


def test_no_rows_of_many_columns():
    """The sums of no rows are zeros, however many columns there are."""
    cols = (1 << 26) + 16
    announce(f"layer norm backward 0x{cols}")
    e = torch.empty((0, cols), dtype=torch.bfloat16, device=device())
    m = torch.empty(0, device=device())
    dw, db = (torch.full((cols,), -3.0, device=device()) for _ in range(2))
    fm.fp8_layernorm_backward(e, e, m, m, torch.ones(cols, dtype=torch.bfloat16, device=device()), e, dweight=dw, dbias=db, workspace=torch.empty(8 * cols, dtype=torch.uint8, device=device()))
    assert (dw == 0).all() and (db == 0).all()
