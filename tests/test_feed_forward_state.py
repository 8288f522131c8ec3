"""What Fp8FeedForward keeps between its calls, on the CPU: the class is run with its entry points replaced by
plain fp32 forms of the same operators (HOST), which act on host tensors, so that every order of calls can be
followed to its numbers without a GPU.

Tolerance of a forward: four E4M3 casts stand between the inputs and the output (norm, both weights, h), each off
by at most half a step, 2^-4 relative (rms 2^-4 / sqrt(3) and less), so the branch is off by less than
sqrt(4 * 2^-8 / 3) = 0.073 in the 2-norm; its sum with the residual stream is rounded to bf16, 2^-8 of the sum."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from oracle import feed_forward as ff

T, H, F = 32, 64, 96
TYPES = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def encode(v, fmt, scale):
    t, top = TYPES[fmt]
    return (v * scale).clamp(-top, top).to(t).view(torch.uint8)


def decode(q, fmt):
    return q.view(TYPES[fmt][0]).float()


def act_slope(z, act):
    s = torch.sigmoid(z)
    return (z, torch.ones_like(z)) if act == "none" else (z * s, s * (1 + z * (1 - s)))


def top_of(v):
    return v.abs().max().reshape(1)


class HOST:
    @staticmethod
    def fp8_quantize(x, fmt, scale=None, q=None, q_t=None, amax=None, sat=None, workspace=None, stream=None):
        c = encode(x.float(), fmt, scale)
        if q is not None:
            q.copy_(c)
        if q_t is not None:
            q_t.copy_(c.t())
        if amax is not None:
            amax.copy_(top_of(x.float()))

    @staticmethod
    def fp8_amax_update(history, head, amax, fmt, scale, scale_inv, status=None, stream=None):
        history[int(head)] = amax[0]
        head.copy_((head + 1) % len(history))
        top = history.max()
        if top > 0:
            scale.copy_(TYPES[fmt][1] / top.reshape(1))
            scale_inv.copy_(1 / scale)

    @staticmethod
    def fp8_quantize_update(x, fmt, history, head, scale, scale_inv, amax, q=None, q_t=None, sat=None, status=None,
                            workspace=None, scale_inv_used=None, stream=None):
        HOST.fp8_quantize(x, fmt, scale, q, q_t, amax)
        scale_inv_used.copy_(scale_inv)
        HOST.fp8_amax_update(history, head, amax, fmt, scale, scale_inv)

    @staticmethod
    def fp8_rmsnorm_quantize(x, weight, eps, fmt, scale, q, residual=None, sum_out=None, rstd=None, amax=None, sat=None,
                             workspace=None, stream=None):
        h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        if sum_out is not None:
            sum_out.copy_(h)
        r = 1 / torch.sqrt(h.float().square().mean(1) + eps)
        y = h.float() * r[:, None] * weight.float()
        q.copy_(encode(y, fmt, scale))
        if rstd is not None:
            rstd.copy_(r)
        if amax is not None:
            amax.copy_(top_of(y))

    @staticmethod
    def fp8_gemm_gated(a, fa, b, fb, sinv_a, sinv_b, act, h, gu=None, out_fmt=None, out_scale=None, amax=None, sat=None,
                       accum="exact", workspace=None, stream=None):
        z = decode(a, fa) @ decode(b, fb).t() * (sinv_a * sinv_b)
        g, u = z.chunk(2, 1)
        v = act_slope(g, act)[0] * u
        h.copy_(encode(v, out_fmt, out_scale))
        if gu is not None:
            gu.copy_(z)
        if amax is not None:
            amax.copy_(top_of(v))

    @staticmethod
    def fp8_gemm_fused(a, fa, b, fb, sinv_a, sinv_b, y, bias=None, act="none", residual=None, z=None, out_fmt=None,
                       out_scale=None, amax=None, sat=None, accum="exact", workspace=None, stream=None):
        y.copy_(decode(a, fa) @ decode(b, fb).t() * (sinv_a * sinv_b) + residual.float())

    @staticmethod
    def fp8_gemm(a, fa, b, fb, sinv_a, sinv_b, c, accum="exact", b_trans=False, stream=None):
        w = decode(b, fb)
        c.copy_(decode(a, fa) @ (w if b_trans else w.t()) * (sinv_a * sinv_b))

    @staticmethod
    def fp8_act_backward(dy, z, act, fmt, scale, q=None, q_t=None, dbias=None, amax=None, sat=None, workspace=None,
                         stream=None):
        HOST.fp8_quantize(dy, fmt, scale, q, q_t, amax)

    @staticmethod
    def fp8_gated_backward(dh, gu, act, fmt, scale, q=None, q_t=None, amax=None, sat=None, workspace=None, stream=None):
        g, u = gu.float().chunk(2, 1)
        v, d = act_slope(g, act)
        HOST.fp8_quantize(torch.cat([dh.float() * u * d, dh.float() * v], 1), fmt, scale, q, q_t, amax)

    @staticmethod
    def fp8_rmsnorm_backward(dy, h, rstd, weight, dx, dweight=None, dresidual=None, workspace=None, stream=None):
        d, f, r = dy.float(), h.float(), rstd[:, None]
        g = d * weight.float()
        dx.copy_(r * (g - f * (r * r * (g * f).mean(1, keepdim=True))) + dresidual.float())
        dweight.copy_((d * f * r).sum(0))


@pytest.fixture(autouse=True)
def host_operators(monkeypatch):
    for name, f in vars(HOST).items():
        if name.startswith("fp8_"):
            monkeypatch.setattr(fm._binding, name, f.__func__)


def randn(seed, *shape, std=1.0):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, std, shape).astype(np.float32)).bfloat16()


def inputs(seed=0):
    return dict(x=randn(seed + 1, T, H), residual=randn(seed + 2, T, H), weight=(randn(seed + 3, H, std=0.1) + 1).bfloat16(),
                w_gu=randn(seed + 4, 2 * F, H, std=0.25), w_d=randn(seed + 5, H, F, std=0.25), dy=randn(seed + 6, T, H))


def block():
    return fm.Fp8FeedForward(T, H, F, device="cpu")


def forward(ffn, d, train=True, y=None):
    y = torch.empty(T, H, dtype=torch.bfloat16) if y is None else y
    ffn.forward(d["x"], d["residual"], d["weight"], y, train=train)
    return y


def backward(ffn, d):
    o = dict(dx=torch.empty(T, H, dtype=torch.bfloat16), dweight=torch.empty(H), dw_gu=torch.empty(2 * F, H), dw_d=torch.empty(H, F))
    ffn.backward(d["dy"], d["weight"], o["dx"], o["dweight"], o["dw_gu"], o["dw_d"])
    return o


def check_forward(y, d):
    s = d["x"].float() if d["residual"] is None else (d["x"].float() + d["residual"].float()).bfloat16().float()
    s = s.double().numpy()
    w = {k: d[k].double().numpy() for k in ("weight", "w_gu", "w_d")}
    n, _ = ff.rms_norm(s, w["weight"], 1e-5)
    branch = ff.gated(n @ w["w_gu"][:F].T, n @ w["w_gu"][F:].T, "silu") @ w["w_d"].T
    off = np.linalg.norm(y.double().numpy() - s - branch)
    assert off <= 0.073 * np.linalg.norm(branch) + 2.0 ** -8 * np.linalg.norm(s + branch), off / np.linalg.norm(branch)


def test_weights_cast_once_serve_any_number_of_updates():
    """The codes of the weights keep the scale they were cast with, whatever update() makes of the next one."""
    ffn, d = block(), inputs()
    ffn.quantize_weights(d["w_gu"], d["w_d"])
    for _ in range(3):
        check_forward(forward(ffn, d), d)
        backward(ffn, d)
        ffn.update()


def test_weights_recast_every_step_step_their_history_once():
    """A step that recasts the weights first pushes one amax of each weight into its history, and casts with the scale
    that the steps before have set."""
    ffn, d = block(), inputs()
    scale = 1.0
    for step in range(3):
        w = (d["w_gu"].float() * (step + 1)).bfloat16()
        ffn.quantize_weights(w, d["w_d"])
        assert torch.equal(ffn.qw_gu, encode(w.float(), "e4m3", torch.tensor([scale])))
        forward(ffn, d)
        backward(ffn, d)
        ffn.update()
        scale = float(448.0 / top_of(w.float()))
        assert torch.equal(ffn.state_gu.history[:step + 1], torch.stack([top_of((d["w_gu"].float() * (k + 1)).bfloat16().float())[0] for k in range(step + 1)]))
        assert not ffn.state_gu.history[step + 1:].any()


@pytest.mark.parametrize("with_residual", [True, False])
def test_inference_leaves_a_training_step_as_it_is(with_residual):
    """forward(train=False) between a training forward and its backward and update: the gradients are those of the
    training batch, bit for bit, and the next scales come from its amaxes."""
    d, other = inputs(), inputs(50)
    if not with_residual:
        d["residual"] = None
    out = []
    for between in (False, True):
        ffn = block()
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
    store = torch.empty(2 * T * H, dtype=torch.bfloat16)
    part, over = store[:T * H].view(T, H), store[T * H // 2:3 * T * H // 2].view(T, H)     # they share half their memory
    part.copy_(x)
    for train in (True, False):
        with pytest.raises(ValueError, match="memory"):
            forward(ffn, dict(d, x=part), y=over, train=train)
        assert torch.equal(part, x)                                                        # refused before anything ran


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
