"""What Fp8FeedForward keeps between its calls, on the GPU (tests/test_feed_forward_state.py follows the same orders
of calls on the CPU).  Tolerance of a forward: four E4M3 casts, each off by at most half a step, 2^-4 relative
(rms 2^-4 / sqrt(3) and less): sqrt(4 * 2^-8 / 3) = 0.073 of the branch in the 2-norm, and bf16's half step, 2^-8,
of its sum with the residual stream."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu
T, H, F = 64, 256, 400


def randn(seed, *shape, std=1.0):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, std, shape).astype(np.float32)).bfloat16().to(device())


def inputs(seed=0):
    return dict(x=randn(seed + 1, T, H), residual=randn(seed + 2, T, H), weight=(randn(seed + 3, H, std=0.1) + 1).bfloat16(),
                w_gu=randn(seed + 4, 2 * F, H, std=0.25), w_d=randn(seed + 5, H, F, std=0.25), dy=randn(seed + 6, T, H))


def block(accum="exact"):
    return fm.Fp8FeedForward(T, H, F, accum=accum, device=device())


def forward(ffn, d, train=True, y=None):
    y = torch.empty(T, H, dtype=torch.bfloat16, device=device()) if y is None else y
    ffn.forward(d["x"], d["residual"], d["weight"], y, train=train)
    return y


def backward(ffn, d):
    o = dict(dx=torch.empty(T, H, dtype=torch.bfloat16, device=device()), dweight=torch.empty(H, device=device()),
             dw_gu=torch.empty(2 * F, H, device=device()), dw_d=torch.empty(H, F, device=device()))
    ffn.backward(d["dy"], d["weight"], o["dx"], o["dweight"], o["dw_gu"], o["dw_d"])
    return o


def check_forward(y, d):
    s = d["x"].float() if d["residual"] is None else (d["x"].float() + d["residual"].float()).bfloat16().float()
    s = s.double().cpu().numpy()
    w = {k: d[k].double().cpu().numpy() for k in ("weight", "w_gu", "w_d")}
    n, _ = ff.rms_norm(s, w["weight"], 1e-5)
    branch = ff.gated(n @ w["w_gu"][:F].T, n @ w["w_gu"][F:].T, "silu") @ w["w_d"].T
    off = np.linalg.norm(y.double().cpu().numpy() - s - branch)
    assert off <= 0.073 * np.linalg.norm(branch) + 2.0 ** -8 * np.linalg.norm(s + branch), off / np.linalg.norm(branch)


@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
def test_weights_cast_once_serve_any_number_of_updates(accum):
    """The codes of the weights keep the scale they were cast with, whatever update() makes of the next one."""
    announce(f"weights cast once {accum}")
    ffn, d = block(accum), inputs()
    ffn.quantize_weights(d["w_gu"], d["w_d"])
    forward(ffn, d)                                    # h saturates at the first step's scale of 1
    for _ in range(3):
        ffn.update()
        check_forward(forward(ffn, d), d)
        backward(ffn, d)


@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("with_residual", [True, False])
def test_inference_leaves_a_training_step_as_it_is(with_residual, accum):
    """forward(train=False) between a training forward and its backward and update: the gradients are those of the
    training batch, bit for bit, and the next scales come from its amaxes."""
    announce(f"inference between residual={with_residual} {accum}")
    d, other = inputs(), inputs(50)
    if not with_residual:
        d["residual"] = None
    out = []
    for between in (False, True):
        ffn = block(accum)
        ffn.quantize_weights(d["w_gu"], d["w_d"])
        for _ in range(2):
            y = forward(ffn, d)
            if between:
                assert torch.equal(forward(ffn, d, train=False), y)
                forward(ffn, other, train=False)
            o = backward(ffn, d)
            ffn.update()
        out.append(dict(o, y=y, **{k: getattr(ffn, k).history.clone() for k in ("state_n", "state_h", "state_dy", "state_dgu")}))
    for k in out[0]:
        assert torch.equal(out[0][k], out[1][k]), k


def test_without_a_residual_the_step_owes_nothing_to_the_callers_x():
    """With residual=None the step is that of a residual of zeros, also where y is written over x or x is changed before
    the backward; an output over a part of x, which is read meanwhile, is refused."""
    d = inputs()
    cases = [dict(d, residual=torch.zeros_like(d["x"])), dict(d, residual=None), dict(d, residual=None, x=d["x"].clone()),
             dict(d, residual=None, x=d["x"].clone())]
    out = []
    for i, e in enumerate(cases):
        ffn = block()
        ffn.quantize_weights(e["w_gu"], e["w_d"])
        y = forward(ffn, e, y=e["x"] if i == 2 else None)
        if i == 3:
            e["x"].mul_(2)
        out.append(dict(y=y, **backward(ffn, e)))
    for other in out[1:]:
        for k in out[0]:
            assert torch.equal(out[0][k], other[k]), k
    x, d["residual"] = d["x"].clone(), None
    assert torch.equal(forward(ffn, d, train=False, y=d["x"]), out[0]["y"])                # inference in place
    store = torch.empty(2 * T * H, dtype=torch.bfloat16, device=device())
    part, over = store[:T * H].view(T, H), store[T * H // 2:3 * T * H // 2].view(T, H)     # they share half their memory
    part.copy_(x)
    for train in (True, False):
        with pytest.raises(ValueError, match="memory"):
            forward(ffn, dict(d, x=part), y=over, train=train)
        assert torch.equal(part, x)                                                        # refused before anything ran
    for name in ("stream", "handle", "null"):                                              # the copy follows the step's stream
        ffn, side = block(), torch.cuda.Stream()
        stream = {"stream": side, "handle": side.cuda_stream, "null": 0}[name]
        y = torch.empty_like(x)
        o = dict(dx=torch.empty_like(x), dweight=torch.empty(H, device=device()), dw_gu=torch.empty(2 * F, H, device=device()),
                 dw_d=torch.empty(H, F, device=device()))
        torch.cuda.synchronize()
        ffn.quantize_weights(d["w_gu"], d["w_d"], stream=stream)
        ffn.forward(x, None, d["weight"], y, stream=stream)
        ffn.backward(d["dy"], d["weight"], o["dx"], o["dweight"], o["dw_gu"], o["dw_d"], stream=stream)
        torch.cuda.synchronize()
        for k, v in dict(o, y=y).items():
            assert torch.equal(out[0][k], v), k


def test_calls_out_of_order_are_errors():
    """A backward needs a training forward whose codes still have their scales and weights."""
    ffn, d = block(), inputs()
    ffn.quantize_weights(d["w_gu"], d["w_d"])
    with pytest.raises(RuntimeError, match="training forward"):
        backward(ffn, d)
    forward(ffn, d, train=False)
    with pytest.raises(RuntimeError, match="training forward"):
        backward(ffn, d)
    for between in (ffn.update, lambda: ffn.quantize_weights(d["w_gu"], d["w_d"])):
        forward(ffn, d)
        first, again = backward(ffn, d), backward(ffn, d)          # any number of gradients of one forward
        for k in first:
            assert torch.equal(first[k], again[k]), k
        between()
        with pytest.raises(RuntimeError, match="training forward"):
            backward(ffn, d)
    forward(ffn, d)
    with pytest.raises(ValueError, match="y must be"):
        forward(ffn, d, y=torch.empty(T, 2 * H, dtype=torch.bfloat16))
    backward(ffn, d)                                               # refused before anything was written: still whole
    with pytest.raises(Exception):                                 # refused by the norm, halfway
        forward(ffn, dict(d, weight=d["weight"][:5]))
    with pytest.raises(RuntimeError, match="training forward"):
        backward(ffn, d)


def test_a_block_restored_from_codes_and_snapshots_goes_on_as_it_was():
    """A weight state's snapshot carries the inverse scale that the codes were cast with, so codes and snapshots put
    into another block give the same bits, without another cast."""
    ffn, d = block(), inputs()
    for _ in range(2):
        ffn.quantize_weights(d["w_gu"], d["w_d"])
        forward(ffn, d)
        ffn.update()
    ffn.quantize_weights((d["w_gu"].float() * 3).bfloat16(), d["w_d"])      # the scale it sets differs from the one it used
    y, other = forward(ffn, d, train=False), block()
    for name in ("state_n", "state_gu", "state_h", "state_d"):
        getattr(other, name).restore(getattr(ffn, name).snapshot())
    other.qw_gu.copy_(ffn.qw_gu)
    other.qw_d.copy_(ffn.qw_d)
    assert torch.equal(forward(other, d, train=False), y)


def test_graph_replays_without_a_residual_match_eager():
    """A training step with residual=None and y over x in a HIP graph: every replay gives the bits of the same step run
    eagerly, with eager work and synchronisations between the replays, and junk in the outputs beforehand."""
    announce("feed-forward graph without a residual")
    d = dict(inputs(), residual=None)

    def program():
        ffn, x = block(), d["x"].clone()
        o = dict(x=x, dx=torch.empty_like(x), dweight=torch.empty(H, device=device()), dw_gu=torch.empty(2 * F, H, device=device()),
                 dw_d=torch.empty(H, F, device=device()))

        def step():
            ffn.quantize_weights(d["w_gu"], d["w_d"])
            ffn.forward(x, None, d["weight"], x)
            ffn.backward(d["dy"], d["weight"], o["dx"], o["dweight"], o["dw_gu"], o["dw_d"])
            ffn.update()

        step()
        return o, step

    (oe, eager), (og, step) = program(), program()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for replay in range(4):
        for o in (og, oe):
            o["x"].copy_(d["x"] * (replay + 1))
        for k in ("dx", "dweight", "dw_gu", "dw_d"):
            og[k].fill_(float(replay))
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for k in og:
            assert torch.equal(og[k], oe[k]), (replay, k)
        torch.zeros(1 << 20, device=device()).add_(1.0).sum().item()
