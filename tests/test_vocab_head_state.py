"""What Fp8VocabHead keeps between its calls, on the CPU: the class is run with its entry points replaced by
plain fp32 forms of the same operators, which act on host tensors, so that every order of calls can be
followed to its numbers without a GPU (the casts and the history are test_feed_forward_state.py's)."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from oracle import model_ends as me
from test_feed_forward_state import HOST as CASTS, decode, encode, top_of

T, H, V = 12, 32, 50


class HOST:
    calls = []

    @staticmethod
    def fp8_layernorm_quantize(x, weight, bias, eps, fmt, scale, q, residual=None, sum_out=None, mean=None, rstd=None, amax=None, sat=None, dropout=0.0, rng=None,
                               workspace=None, stream=None):
        h = x.float()
        if dropout:
            h = h * torch.from_numpy(me.dropout_factors(tuple(x.shape), dropout, *rng.tolist()).astype(np.float32))
        h = (h if residual is None else h + residual.float()).to(x.dtype)
        m = h.float().mean(1)
        r = 1 / torch.sqrt(h.float().var(1, unbiased=False) + eps)
        y = (h.float() - m[:, None]) * r[:, None] * weight.float() + (0 if bias is None else bias.float())
        q.copy_(encode(y, fmt, scale))
        for to, v in ((sum_out, h), (mean, m), (rstd, r), (amax, top_of(y))):
            if to is not None:
                to.copy_(v)

    @staticmethod
    def fp8_layernorm_backward(dy, h, mean, rstd, weight, dx, dweight=None, dbias=None, dresidual=None, dbranch=None, dropout=0.0, rng=None, workspace=None,
                               stream=None):
        dh, dw, db = me.layer_norm_grad(*(t.double().numpy() for t in (dy, h, weight)), 0.0, mean.numpy(), rstd.numpy())
        f = me.dropout_factors(dh.shape, dropout, *rng.tolist()) if dropout else 1.0
        for to, v in ((dx, dh), (dweight, dw), (dbias, db), (dbranch, dh * f)):
            if to is not None:
                to.copy_(torch.from_numpy(v))

    @staticmethod
    def fp8_vocab_cross_entropy(x, fx, w, fw, sinv_x, sinv_w, targets, loss, lse, accum="exact", workspace=None, stream=None):
        l, s = me.cross_entropy((decode(x, fx) @ decode(w, fw).t() * (sinv_x * sinv_w)).numpy(), targets.numpy())
        for to, v in ((loss, l), (lse, s)):
            if to is not None:
                to.copy_(torch.from_numpy(v))

    @staticmethod
    def fp8_vocab_cross_entropy_backward(x, fx, w, fw, sinv_x, sinv_w, targets, lse, dloss, fmt, scale, scale_inv, dx=None, dw=None, amax=None, sat=None,
                                         accum="exact", workspace=None, stream=None):
        z = (decode(x, fx) @ decode(w, fw).t() * (sinv_x * sinv_w)).numpy()
        d = torch.from_numpy(me.cross_entropy_grad(z, targets.numpy(), dloss.numpy(), lse.numpy())).float()
        c = decode(encode(d, fmt, scale), fmt)
        dx.copy_(c @ decode(w, fw) * (scale_inv * sinv_w))
        if dw is not None:
            dw.copy_(c.t() @ decode(x, fx) * (scale_inv * sinv_x))
        amax.copy_(top_of(d))

    @staticmethod
    def fp8_embedding(tokens, table, out, scale=1.0, fmt=None, sinv=None, stream=None):
        out.copy_(torch.from_numpy(me.embedding(tokens.numpy(), (decode(table, fmt) * sinv).numpy(), scale)))

    @staticmethod
    def fp8_embedding_backward(tokens, dy, dtable, scale=1.0, base=None, workspace=None, stream=None):
        dtable.copy_(torch.from_numpy(me.embedding_grad(tokens.numpy(), dy.double().numpy(), dtable.shape[0], scale, base.double().numpy())))


@pytest.fixture(autouse=True)
def host(monkeypatch):
    for source in (CASTS, HOST):
        for name in dir(source):
            if name.startswith("fp8_"):
                monkeypatch.setattr(fm._binding, name, getattr(source, name))


def randn(seed, *shape, std=1.0):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, std, shape).astype(np.float32)).bfloat16()


def inputs(seed=0):
    gen = np.random.default_rng(seed + 9)
    return dict(x=randn(seed + 1, T, H), residual=randn(seed + 2, T, H, std=2.0), norm_weight=(randn(seed + 3, H, std=0.1) + 1).bfloat16(),
                norm_bias=randn(seed + 4, H, std=0.1), weight=randn(seed + 5, V, H, std=0.5), targets=torch.from_numpy(gen.integers(-1, V, T)),
                dloss=torch.from_numpy(gen.normal(size=T).astype(np.float32)), rng=torch.tensor([seed + 1, 5]))


def head(dropout=0.25):
    return fm.Fp8VocabHead(T, H, V, dropout=dropout, device="cpu")


def forward(hd, d, train=True):
    loss, lse = torch.zeros(T), torch.zeros(T)
    hd.forward(d["x"], d["residual"], d["norm_weight"], d["norm_bias"], d["targets"], loss, lse, rng=d["rng"] if train else None, train=train)
    return loss, lse


def backward(hd, d):
    o = dict(dx=torch.zeros(T, H, dtype=torch.bfloat16), dweight=torch.zeros(H), dbias=torch.zeros(H), dw=torch.zeros(V, H), dbranch=torch.zeros(T, H, dtype=torch.bfloat16))
    hd.backward(d["dloss"], d["norm_weight"], **o)
    return o


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def step(hd, d):
    """A settled training step: scales that fit."""
    hd.quantize_weights(d["weight"])
    hd.quantize_weights(d["weight"])
    forward(hd, d)
    backward(hd, d)
    hd.update()
    forward(hd, d)
    backward(hd, d)
    hd.update()


def test_the_order_of_calls_is_checked():
    hd, d = head(), inputs()
    with pytest.raises(RuntimeError, match="no codes"):
        forward(hd, d)
    with pytest.raises(RuntimeError, match="no codes"):
        hd.embed(d["targets"], torch.zeros(T, H))
    hd.quantize_weights(d["weight"])
    with pytest.raises(RuntimeError, match="training forward"):
        backward(hd, d)
    forward(hd, d, train=False)
    with pytest.raises(RuntimeError, match="training forward"):
        backward(hd, d)
    with pytest.raises(ValueError, match="rng"):
        hd.forward(d["x"], None, d["norm_weight"], None, d["targets"], torch.zeros(T))
    forward(hd, d)
    first = backward(hd, d)
    assert same(first, backward(hd, d))                       # as often as wanted
    for ends in (lambda: hd.update(), lambda: hd.quantize_weights(d["weight"])):
        forward(hd, d)
        ends()
        with pytest.raises(RuntimeError, match="training forward"):
            backward(hd, d)


def test_refusals():
    with pytest.raises(ValueError, match="HYBRID"):
        fm.Fp8VocabHead(4, 32, 20, recipe=fm.Recipe(fmt_bwd="e4m3"), device="cpu")
    with pytest.raises(ValueError, match="dropout"):
        fm.Fp8VocabHead(4, 32, 20, dropout=1.0, device="cpu")
    hd, d = head(), inputs()
    with pytest.raises(ValueError, match="weight must be"):
        hd.quantize_weights(d["weight"][:-1])
    hd.quantize_weights(d["weight"])
    with pytest.raises(ValueError, match="targets must be"):
        hd.forward(d["x"], None, d["norm_weight"], None, d["targets"][:-1], torch.zeros(T), rng=d["rng"])
    with pytest.raises(ValueError, match="at most"):
        hd.embed_backward(torch.zeros(T + 1, dtype=torch.int64), torch.zeros(T + 1, H), torch.zeros(V, H))


def test_evaluation_between_a_training_forward_and_its_backward_changes_neither():
    d, other = inputs(), inputs(50)
    out = []
    for between in (False, True):
        hd = head()
        step(hd, d)
        hd.quantize_weights(d["weight"])
        forward(hd, d)
        if between:
            loss, lse = forward(hd, other, train=False)
            # nothing is dropped in an evaluation
            h = (other["x"].float() + other["residual"].float()).bfloat16().double().numpy()
            y, _, _ = me.layer_norm(h, other["norm_weight"].double().numpy(), other["norm_bias"].double().numpy(), 1e-5)
            w = d["weight"].double().numpy()
            want, _ = me.cross_entropy(y @ w.T, other["targets"].numpy())
            # each factor of a logit is off by at most half a step of E4M3, 2^-4 (and what lies below its range); the loss moves by at most two logits' worth
            off = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(y) @ np.abs(w).T) + 1e-3
            assert np.all(np.abs(loss.numpy() - want) <= 2 * off.max(axis=1))
        grads = backward(hd, d)
        hd.update()
        out.append((grads, hd.state_n.snapshot(), hd.state_d.snapshot()))
    assert same(out[0][0], out[1][0]) and same(out[0][1], out[1][1]) and same(out[0][2], out[1][2])


def test_targets_and_rng_of_the_forward_are_kept():
    """The caller may overwrite both between a training forward and its backward."""
    d = inputs()
    out = []
    for overwrite in (False, True):
        hd, e = head(), dict(inputs())
        step(hd, d)
        hd.quantize_weights(d["weight"])
        forward(hd, e)
        if overwrite:
            e["targets"].fill_(3)
            e["rng"].fill_(8)
        out.append(backward(hd, e))
    assert same(out[0], out[1])


def test_codes_keep_the_scale_they_were_cast_with():
    """Lookups, losses and gradients after any number of updates, and after a weight cast whose next scale differs."""
    hd, d = head(0.0), inputs()
    step(hd, d)
    hd.quantize_weights(d["weight"] * 3)                      # codes at the old scale; the next scale is another
    assert not torch.equal(hd.state_w.scale_inv, hd.state_w.scale_inv_used)
    out = torch.zeros(T, H)
    hd.embed(d["targets"].clamp(min=0), out, scale=2.0)
    want = (d["weight"] * 3).float()[d["targets"].clamp(min=0)].clamp(max=1e9) * 2
    top = 448.0 * hd.state_w.scale_inv_used.item()
    want = want.clamp(-2 * top, 2 * top)
    assert (out - want).abs().max() <= 2.0 ** -4 * want.abs().max()
    for _ in range(3):
        hd.update()
        again = torch.zeros(T, H)
        hd.embed(d["targets"].clamp(min=0), again, scale=2.0)
        assert torch.equal(again, out)


def test_tied_gradient_is_the_sum_of_both():
    hd, d = head(0.0), inputs()
    step(hd, d)
    hd.quantize_weights(d["weight"])
    forward(hd, d)
    g = backward(hd, d)
    tokens = torch.from_numpy(np.random.default_rng(4).integers(-1, V, T - 2))
    dy, total = randn(77, T - 2, H), g["dw"].clone()
    hd.embed_backward(tokens, dy, total, scale=0.5)
    want = me.embedding_grad(tokens.numpy(), dy.double().numpy(), V, 0.5, g["dw"].double().numpy())
    assert np.allclose(total.double().numpy(), want, atol=1e-5)
