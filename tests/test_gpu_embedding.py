"""GPU parity of the embedding lookup and its gradient.

Tolerances, derived before the first run: the lookup is one fp32 product (codes: two, one after the
other) and one rounding, so its bits are torch's.  A gradient of small whole numbers and a scale that is a
power of two is exact in any order, so those bits are the oracle's.  Of other values: a sum passes
through at most 16 + 4096 roundings of 2^-24 on the sum of magnitudes (a chunk of at least 16, then the chunks of one
token), 2.5e-4, the scale's and base's fused step EW, and half a step of the type."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from oracle import model_ends as me
from test_gpu_feed_forward import EW, HALF, check_close, d64, rand_codes, randn, scalar

pytestmark = pytest.mark.gpu
LONG = 2.5e-4


def tokens_of(kind, rows, vocab, seed=0):
    gen = np.random.default_rng(seed)
    if kind == "same":
        t = np.full(rows, vocab - 1)
    elif kind == "none":
        t = np.where(gen.random(rows) < 0.5, -1, vocab)
    elif kind == "down":
        t = (np.arange(rows)[::-1] * 7) % vocab
    elif kind == "two":                                   # long runs that meet inside a chunk
        t = np.where(gen.random(rows) < 0.7, 0, vocab - 1)
    else:
        t = np.floor(gen.random(rows) ** 3 * vocab).astype(np.int64)
        t[gen.random(rows) < 0.1] = -100
        t[gen.random(rows) < 0.05] = vocab                # one past the end
        t[gen.random(rows) < 0.02] = np.iinfo(np.int64).max - 5
    return t.astype(np.int64)


def to_tokens(t, dtype):
    return torch.from_numpy(np.clip(t, -2 ** 31, 2 ** 31 - 1) if dtype == torch.int32 else t).to(dtype).to(device())


@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 16), (1, 1000, 4096), (7, 5, 48), (300, 1000, 1040), (33, 100, 8192), (9000, 64, 256), (70000, 50, 32)])
@pytest.mark.parametrize("table", ["f32", "bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_lookup(rows, vocab, cols, table, index):
    announce(f"embedding {rows} of {vocab} x {cols} {table} {index}")
    t = tokens_of("some", rows, vocab, 1)
    if table.startswith("e"):
        w, fmt, inv = rand_codes(2, (vocab, cols), table), table, scalar(0.037)
        wide = w.view(torch.float8_e4m3fn if table == "e4m3" else torch.float8_e5m2).float() * inv
    else:
        w, fmt, inv = randn(2, vocab, cols, dtype=torch.float32 if table == "f32" else torch.bfloat16), None, None
        wide = w.float()
    inside = torch.from_numpy((t >= 0) & (t < vocab)).to(device())
    at = torch.from_numpy(np.where((t >= 0) & (t < vocab), t, 0)).to(device())
    scale = np.float32(np.sqrt(cols))
    want = torch.where(inside[:, None], wide[at] * torch.tensor(scale, device=device()), 0.0)
    for out in (torch.float32, torch.bfloat16):
        got = torch.full((rows, cols), 7.0, dtype=out, device=device())
        fm.fp8_embedding(to_tokens(t, index), w, got, scale=float(scale), fmt=fmt, sinv=inv)
        assert torch.equal(got, want.to(out))


def test_lookup_special_values():
    """NaN and Inf of the table's row come through, those of other rows do not; NaN codes are NaN."""
    announce("embedding special values")
    w = randn(3, 4, 32, dtype=torch.float32)
    w[1, 3], w[2, 4] = float("nan"), float("inf")
    out = torch.zeros((5, 32), device=device())
    fm.fp8_embedding(to_tokens(np.array([0, 1, 2, 3, -1]), torch.int64), w, out)
    assert torch.isfinite(out[[0, 3, 4]]).all() and torch.isnan(out[1, 3]) and torch.isinf(out[2, 4]) and (out[4] == 0).all()
    q = torch.full((2, 16), 0x7F, dtype=torch.uint8, device=device())
    q[1] = 0x38                                           # 1 in E4M3
    out = torch.zeros((2, 16), dtype=torch.bfloat16, device=device())
    fm.fp8_embedding(to_tokens(np.array([0, 1]), torch.int32), q, out, fmt="e4m3", sinv=scalar(2.0))
    assert torch.isnan(out[0]).all() and (out[1] == 2.0).all()


SIZES = [(1, 1, 16), (1, 900, 4096), (15, 3, 32), (16, 4, 48), (17, 4, 2064), (64, 1, 16), (100, 1000, 256), (1000, 7, 1040), (8191, 300, 64),
         (8192, 50021, 32), (8193, 40, 16), (20000, 1000, 48), (70000, 3, 16)]


@pytest.mark.parametrize("rows,vocab,cols", SIZES)
@pytest.mark.parametrize("kind", ["some", "same", "none", "down", "two"])
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
def test_gradient_of_whole_numbers(rows, vocab, cols, kind, dtype, out):
    announce(f"embedding gradient {rows} of {vocab} x {cols} {kind} {dtype} -> {out}")
    t = tokens_of(kind, rows, vocab, 4)
    gen = np.random.default_rng(5)
    small = 1 if out == torch.bfloat16 else 8
    dy = gen.integers(-small, small + 1, size=(rows, cols)).astype(np.float32)
    base = gen.integers(-3, 4, size=(vocab, cols)).astype(np.float32)
    want = torch.from_numpy(me.embedding_grad(t, dy, vocab, 0.5)).to(device())
    index = torch.int32 if rows % 2 else torch.int64
    ids, dyt, ws = to_tokens(t, index), torch.from_numpy(dy).to(dtype).to(device()), fm.embedding_workspace_bytes(rows, cols)
    got = torch.full((vocab, cols), 7.0, dtype=out, device=device())
    # a guard behind the workspace that the call was promised
    space = torch.full((ws + 64,), 0xA5, dtype=torch.uint8, device=device())
    fm.fp8_embedding_backward(ids, dyt, got, scale=0.5, workspace=space[:ws])
    assert torch.equal(got.double(), want.to(out).double()) and (space[ws:] == 0xA5).all()
    b = torch.from_numpy(base).to(out).to(device())
    fm.fp8_embedding_backward(ids, dyt, got, scale=0.5, base=b, workspace=space[:ws])
    assert torch.equal(got.double(), (want + b.double()).to(out).double())
    fm.fp8_embedding_backward(ids, dyt, b, scale=0.5, base=b, workspace=space[:ws])            # added in place
    assert torch.equal(b, got)


@pytest.mark.parametrize("rows,vocab,cols", [(5000, 700, 1040), (8192, 50021, 256), (30000, 11, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_any_numbers(rows, vocab, cols, dtype):
    announce(f"embedding gradient {rows} of {vocab} x {cols} {dtype}")
    t = tokens_of("some", rows, vocab, 6)
    dy, base = randn(7, rows, cols, std=0.1, dtype=dtype), randn(8, vocab, cols, dtype=dtype)
    scale = float(np.float32(1.7))
    want = me.embedding_grad(t, d64(dy), vocab, scale, d64(base))
    mag = me.embedding_grad(t, np.abs(d64(dy)), vocab, scale)
    ws = torch.empty(fm.embedding_workspace_bytes(rows, cols), dtype=torch.uint8, device=device())
    outs = []
    for _ in range(2):
        got = torch.full((vocab, cols), 7.0, dtype=dtype, device=device())
        fm.fp8_embedding_backward(to_tokens(t, torch.int64), dy, got, scale=scale, base=base, workspace=ws)
        check_close(d64(got), want, LONG * mag + EW * np.abs(want) + HALF[dtype] * 1.001 * np.abs(want), "dtable")
        outs.append(got)
        ws.fill_(0xFF)
    assert torch.equal(outs[0], outs[1])
    inplace = base.clone()
    fm.fp8_embedding_backward(to_tokens(t, torch.int32), dy, inplace, scale=scale, base=inplace, workspace=ws)
    assert torch.equal(inplace, outs[0])


@pytest.mark.parametrize("cols", [16, 528])
@pytest.mark.parametrize("shift", [0, 5])
@pytest.mark.parametrize("in_place", [False, True])
def test_runs_of_many_lengths(cols, shift, in_place):
    """Runs of one token over 1 to 200 pieces of the sorted list of 16 each, and one value less and more, from two places in a piece; exact."""
    announce(f"embedding runs {cols} {shift} {in_place}")
    lengths = [shift] + [16 * n + more for n in (1, 2, 3, 4, 5, 8, 9, 32, 33, 62, 63, 64, 65, 66, 67, 128, 129, 200) for more in (-1, 0, 1)]
    t = np.repeat(np.arange(len(lengths)), lengths)
    assert 8192 < len(t) <= 65536                                # pieces of 16
    vocab, gen = len(lengths) + 3, np.random.default_rng(shift)
    gen.shuffle(t)
    dy = gen.integers(-4, 5, size=(len(t), cols)).astype(np.float32)
    base = gen.integers(-9, 10, size=(vocab, cols)).astype(np.float32)
    dtable = torch.from_numpy(base).to(device()) if in_place else torch.full((vocab, cols), 7.0, device=device())
    ws = torch.full((fm.embedding_workspace_bytes(len(t), cols),), 0xA5, dtype=torch.uint8, device=device())
    fm.fp8_embedding_backward(to_tokens(t, torch.int32), torch.from_numpy(dy).to(device()), dtable, scale=0.5, base=dtable if in_place else None, workspace=ws)
    want = me.embedding_grad(t, dy, vocab, 0.5, base if in_place else None)
    assert np.array_equal(d64(dtable), want)


def test_rows_are_added_in_the_order_of_the_tokens():
    announce("embedding gradient order")
    dy = randn(9, 16, 32, dtype=torch.float32)
    got = torch.zeros((3, 32), device=device())
    ws = torch.empty(fm.embedding_workspace_bytes(16, 32), dtype=torch.uint8, device=device())
    fm.fp8_embedding_backward(torch.ones(16, dtype=torch.int32, device=device()), dy, got, workspace=ws)
    want = np.zeros(32, dtype=np.float32)
    for row in dy.cpu().numpy():
        want = want + row
    assert np.array_equal(got[1].cpu().numpy(), want) and (got[[0, 2]] == 0).all()


def test_gradient_against_differences():
    """sum(dy * lookup(table)) on the device, differenced in one entry: whole numbers, so the difference is exact."""
    announce("embedding gradient against differences")
    gen = np.random.default_rng(10)
    t = to_tokens(gen.integers(-1, 6, size=40), torch.int64)
    table = torch.from_numpy(gen.integers(-4, 5, size=(6, 16)).astype(np.float32)).to(device())
    dy = torch.from_numpy(gen.integers(-4, 5, size=(40, 16)).astype(np.float32)).to(device())
    got, out = torch.zeros((6, 16), device=device()), torch.zeros((40, 16), device=device())
    fm.fp8_embedding_backward(t, dy, got, scale=2.0, workspace=torch.empty(fm.embedding_workspace_bytes(40, 16), dtype=torch.uint8, device=device()))

    def value(w):
        fm.fp8_embedding(t, w, out, scale=2.0)
        return (out * dy).sum().item()

    for i in range(6):
        for j in range(16):
            up, down = table.clone(), table.clone()
            up[i, j] += 1
            down[i, j] -= 1
            assert got[i, j].item() == (value(up) - value(down)) / 2


def test_special_rows_and_no_tokens():
    announce("embedding gradient special rows")
    dy = randn(11, 3, 16, dtype=torch.float32)
    dy[0, 0], dy[2] = float("nan"), float("inf")
    ws = torch.empty(fm.embedding_workspace_bytes(3, 16), dtype=torch.uint8, device=device())
    got = torch.full((5, 16), 7.0, device=device())
    fm.fp8_embedding_backward(to_tokens(np.array([1, 4, -1]), torch.int64), dy, got, workspace=ws)   # the Inf row has no token
    assert torch.isnan(got[1, 0]) and torch.equal(got[1, 1:], dy[0, 1:]) and torch.equal(got[4], dy[1]) and (got[[0, 2, 3]] == 0).all()
    none = torch.empty(0, dtype=torch.int64, device=device())
    base = randn(12, 5, 16, dtype=torch.float32)
    fm.fp8_embedding_backward(none, dy[:0], got, base=base)
    assert torch.equal(got, base)
    fm.fp8_embedding_backward(none, dy[:0], got)
    assert (got == 0).all()
    fm.fp8_embedding(none, base, got[:0])
    fm.fp8_embedding_backward(to_tokens(np.array([0, 0, 0]), torch.int64), dy, got[:0], workspace=ws)
    out = torch.full((3, 16), 7.0, device=device())
    fm.fp8_embedding(to_tokens(np.array([0, 1, -1]), torch.int64), base[:0], out)                       # an empty table
    assert (out == 0).all()


def test_the_most_tokens():
    rows, vocab, cols = 1 << 20, 4099, 16
    announce(f"embedding gradient {rows} tokens")
    t = tokens_of("some", rows, vocab, 13)
    dy = torch.from_numpy(np.random.default_rng(14).integers(-4, 5, size=(rows, cols)).astype(np.float32)).to(device())
    want = torch.from_numpy(me.embedding_grad(t, dy.cpu().numpy(), vocab)).to(device())
    got = torch.full((vocab, cols), 7.0, device=device())
    ws = torch.empty(fm.embedding_workspace_bytes(rows, cols), dtype=torch.uint8, device=device())
    fm.fp8_embedding_backward(to_tokens(t, torch.int64), dy, got, workspace=ws)
    assert torch.equal(got.double(), want)


def test_a_table_of_more_than_2_31_elements():
    vocab, cols = 131200, 16384
    announce(f"embedding {vocab}x{cols}")
    t = to_tokens(np.array([vocab - 1, 5, vocab - 1, 131073, vocab, 7]), torch.int64)
    table = torch.zeros((vocab, cols), dtype=torch.bfloat16, device=device())
    last = randn(15, 2, cols)
    table[vocab - 1], table[131073] = last[0], last[1]
    out = torch.full((6, cols), 7.0, dtype=torch.bfloat16, device=device())
    fm.fp8_embedding(t, table, out)
    assert torch.equal(out[[0, 2, 3]], last[[0, 0, 1]]) and (out[[1, 4, 5]] == 0).all()
    dy = randn(16, 6, cols)
    fm.fp8_embedding_backward(t, dy, table, base=table, workspace=torch.empty(fm.embedding_workspace_bytes(6, cols), dtype=torch.uint8, device=device()))
    assert torch.equal(table[131073], (last[1].float() + dy[3].float()).bfloat16()) and torch.equal(table[7], dy[5])
    assert torch.equal(table[vocab - 1], (last[0].float() + (dy[0].float() + dy[2].float())).bfloat16()) and (table[8:131000] == 0).all()


def test_captured_with_new_tokens_each_replay():
    announce("embedding captured")
    rows, vocab, cols = 9000, 500, 256
    w, dy = randn(17, vocab, cols, dtype=torch.float32), randn(18, rows, cols)
    ids = to_tokens(tokens_of("some", rows, vocab, 19), torch.int64)
    ws = torch.empty(fm.embedding_workspace_bytes(rows, cols), dtype=torch.uint8, device=device())

    def step(out, dw):
        fm.fp8_embedding(ids, w, out, scale=2.0)
        fm.fp8_embedding_backward(ids, dy, dw, base=w, workspace=ws)

    out, dw = torch.zeros((rows, cols), device=device()), torch.zeros_like(w)
    step(out, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, dw)
    for k in range(4):
        ids.copy_(to_tokens(tokens_of(("some", "same", "two", "none")[k], rows, vocab, 20 + k), torch.int64))
        out.fill_(3)
        dw.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        out2, dw2 = torch.zeros_like(out), torch.zeros_like(dw)
        step(out2, dw2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(dw, dw2), k


def test_refusals_of_the_binding():
    w, out = randn(1, 4, 32), torch.zeros((3, 32), dtype=torch.bfloat16, device=device())
    ids = torch.zeros(3, dtype=torch.int64, device=device())
    ws = torch.empty(4096, dtype=torch.uint8, device=device())
    for bad in (ids.float(), ids.view(1, 3), ids.cpu(), None):
        with pytest.raises((TypeError, ValueError)):
            fm.fp8_embedding(bad, w, out)
    with pytest.raises(ValueError, match="out must have shape"):
        fm.fp8_embedding(ids, w, out[:2])
    with pytest.raises(TypeError):
        fm.fp8_embedding(ids, w, out, fmt="e4m3", sinv=scalar(1.0))
    with pytest.raises(fm.Fp8Error, match="NULL"):
        fm.fp8_embedding(ids, torch.zeros((4, 32), dtype=torch.uint8, device=device()), out, fmt="e4m3")
    with pytest.raises(fm.Fp8Error, match="workspace"):
        fm.fp8_embedding_backward(ids, out, w, workspace=ws[:16])
    with pytest.raises(ValueError, match="base must have shape"):
        fm.fp8_embedding_backward(ids, out, w, base=w[:3], workspace=ws)
    with pytest.raises(ValueError, match="contiguous"):
        fm.fp8_embedding_backward(ids, randn(1, 32, 3).t(), w, workspace=ws)
