"""Fp8VocabHead on the GPU, and a whole small model between its two ends: embedding, a feed-forward block, dropout, norm
and loss, and all gradients back to the tied weight.  Every stage is held to the fp64 oracle on the inputs that it was given
(the codes that the stage before it left), with the tolerances of the operators' own tests."""

import numpy as np
import pytest
import torch

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device
from oracle import codec, model_ends as me
from test_gpu_feed_forward import EW, HALF, REL, SUM, check_close, check_codes, d64, u8
from test_gpu_layer_norm import EPS, factors, y_bound
from test_gpu_vocab_cross_entropy import SUMS, Problem, check_backward

pytestmark = pytest.mark.gpu
P, SEED, OFFSET = 0.2, 91, 4


def randn(seed, *shape, std=1.0, mean=0.0):
    return torch.from_numpy((np.random.default_rng(seed).normal(mean, std, shape)).astype(np.float32)).bfloat16().to(device())


def bf(*shape):
    return torch.full(shape, 7.0, dtype=torch.bfloat16, device=device())


def f32(*shape):
    return torch.full(shape, 7.0, device=device())


class Model:
    """embedding -> feed-forward block -> head, tied; one call of step() is a training step without the optimiser."""

    def __init__(self, T, H, F, V, accum, pieces):
        self.shape, self.scale = (T, H, F, V), float(np.sqrt(H))
        self.ffn = fm.Fp8FeedForward(T, H, F, accum=accum, device=device())
        self.head = fm.Fp8VocabHead(T, H, V, dropout=P, pieces=pieces, accum=accum, device=device())
        self.w, self.w_gu, self.w_d = randn(1, V, H, std=0.3), randn(2, 2 * F, H, std=0.2), randn(3, H, F, std=0.2)
        self.n1, self.n2, self.b2 = randn(4, H, std=0.1, mean=1.0), randn(5, H, std=0.1, mean=1.0), randn(6, H, std=0.1)
        gen = np.random.default_rng(7)
        t = gen.integers(0, V, T)
        t[::9] = -100
        self.targets, self.tokens = torch.from_numpy(t).to(device()), torch.from_numpy(gen.integers(-1, V, T).astype(np.int32)).to(device())
        self.dloss = torch.full((T,), 1.0 / T, device=device())
        self.rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device=device())
        o = self.o = dict(x0=bf(T, H), y=bf(T, H), loss=f32(T), lse=f32(T), dh=bf(T, H), dbranch=bf(T, H), dn2=f32(H), db2=f32(H), dw=f32(V, H), dx=bf(T, H), dn1=f32(H),
                          dw_gu=f32(2 * F, H), dw_d=f32(H, F))
        o["dx0"] = bf(T, H)

    def step(self, update=True):
        o, hd, ffn = self.o, self.head, self.ffn
        hd.quantize_weights(self.w)
        ffn.quantize_weights(self.w_gu, self.w_d)
        hd.embed(self.tokens, o["x0"], scale=self.scale)
        ffn.forward(o["x0"], None, self.n1, o["y"])
        hd.forward(o["y"], o["x0"], self.n2, self.b2, self.targets, o["loss"], o["lse"], rng=self.rng)
        hd.backward(self.dloss, self.n2, o["dh"], o["dn2"], o["db2"], o["dw"], dbranch=o["dbranch"])
        ffn.backward(o["dbranch"], self.n1, o["dx"], o["dn1"], o["dw_gu"], o["dw_d"])
        torch.add(o["dh"], o["dx"], out=o["dx0"])
        self.dw_head = o["dw"].clone()
        hd.embed_backward(self.tokens, o["dx0"], o["dw"], scale=self.scale)
        if update:
            hd.update()
            ffn.update()


@pytest.mark.parametrize("accum", ["exact", "mfma_fp8"])
@pytest.mark.parametrize("T,H,F,V,pieces", [(32, 128, 160, 1003, 1), (272, 256, 96, 517, 3)])
def test_a_model_between_both_ends(T, H, F, V, pieces, accum):
    announce(f"model T={T} H={H} F={F} V={V} pieces={pieces} {accum}")
    m = Model(T, H, F, V, accum, pieces)
    for _ in range(3):                                    # the scales settle
        m.step()
    m.step(update=False)
    o, hd = m.o, m.head
    w = codec.decode(u8(hd.qw), "e4m3") * hd.state_w.scale_inv_used.item()
    tokens = m.tokens.cpu().numpy()
    # lookup: two fp32 products and a rounding
    want = me.embedding(tokens, w, m.scale)
    check_close(d64(o["x0"]), want, (EW + HALF[torch.bfloat16] * 1.001) * np.abs(want), "x0")
    # dropout, residual and norm
    h = (o["y"].float() * factors((T, H), P, SEED, OFFSET) + o["x0"].float()).bfloat16()
    assert torch.equal(hd.sum, h)
    H64 = d64(h)
    _, mu, r = me.layer_norm(H64, d64(m.n2), d64(m.b2), np.float32(EPS))
    y, bound = y_bound(H64, mu, r, d64(m.n2), d64(m.b2))
    check_codes(hd.qn, y, bound, hd.state_n.scale.item(), "e4m3")
    # loss and its gradient's products, from the codes
    p = Problem.__new__(Problem)
    p.M, p.V, p.K, p.fx, p.fw = T, V, H, "e4m3", "e4m3"
    p.x, p.w, p.sx, p.sw, p.t, p.dloss = hd.qn, hd.qw, hd.state_n.scale_inv, hd.state_w.scale_inv_used, m.targets.cpu().numpy(), m.dloss
    z, B = p.logits(accum)
    loss, lse = me.cross_entropy(z, p.t)
    tol = B.max(axis=1) + SUMS + EW * np.abs(lse)
    check_close(d64(o["lse"]), lse, tol, "lse")
    check_close(d64(o["loss"]), loss, np.where(loss != 0, tol + B.max(axis=1) + EW * np.abs(z).max(axis=1), 0.0), "loss")
    check_backward(p, accum, o["lse"], (hd.dn, m.dw_head, hd.state_d.amax, None), "e5m2", hd.state_d.scale.item(), types=(torch.bfloat16, torch.float32), inv=hd.state_d.scale_inv)
    # the norm's gradient
    M, R = d64(hd.mean)[:, None], d64(hd.rstd)[:, None]
    dh, dw, db = me.layer_norm_grad(d64(hd.dn), H64, d64(m.n2), 0.0, d64(hd.mean), d64(hd.rstd))
    g, a = np.abs(d64(hd.dn) * d64(m.n2)), np.abs((H64 - M) * R)
    mag = R * (g + g.mean(axis=1, keepdims=True) + a * (g * a).mean(axis=1, keepdims=True))
    check_close(d64(o["dh"]), dh, REL * mag + (EW + HALF[torch.bfloat16] * 1.001) * np.abs(dh), "dh")
    f = me.dropout_factors((T, H), P, SEED, OFFSET)
    check_close(d64(o["dbranch"]), dh * f, REL * mag * f + (2 * EW + HALF[torch.bfloat16] * 1.001) * np.abs(dh * f), "dbranch")
    check_close(d64(o["dn2"]), dw, SUM * np.sum(np.abs(d64(hd.dn)) * a, axis=0), "dweight")
    check_close(d64(o["db2"]), db, SUM * np.sum(np.abs(d64(hd.dn)), axis=0), "dbias")
    # the tied weight's gradient: the head's and the lookup's
    total = me.embedding_grad(tokens, d64(o["dx0"]), V, m.scale, d64(m.dw_head))
    size = me.embedding_grad(tokens, np.abs(d64(o["dx0"])), V, m.scale)
    check_close(d64(o["dw"]), total, 2.5e-4 * size + EW * np.abs(total), "dw")


def test_a_step_captured_and_replayed():
    """Weight casts, both ends, the block between them, all gradients and the scales' updates in one graph: replays equal eager steps."""
    announce("model captured")
    a, b = (Model(64, 128, 96, 700, "exact", 2) for _ in range(2))
    for m in (a, b):
        for _ in range(2):
            m.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for k in range(4):
        for m in (a, b):
            m.rng.copy_(torch.tensor([SEED, OFFSET + k], device=device()))
            m.targets.copy_(torch.from_numpy(np.random.default_rng(k).integers(-3, 700, 64)).to(device()))
        graph.replay()
        torch.cuda.synchronize()
        b.step()
        torch.cuda.synchronize()
        for name in a.o:
            assert torch.equal(a.o[name], b.o[name]), (k, name)
        for sa, sb in ((a.head.state_n, b.head.state_n), (a.head.state_w, b.head.state_w), (a.head.state_d, b.head.state_d)):
            assert all(torch.equal(u, v) for u, v in zip(sa.snapshot().values(), sb.snapshot().values()))


def test_evaluation_between_and_one_token():
    """An evaluation between a training forward and its backward changes neither; a head of one token serves."""
    announce("head evaluation")
    out = []
    for between in (False, True):
        m = Model(32, 128, 96, 300, "exact", 1)
        m.step()
        m.step(update=False)
        if between:
            m.head.forward(randn(20, 32, 128), None, m.n2, None, m.targets.flip(0).contiguous(), f32(32), train=False)
        m.head.backward(m.dloss, m.n2, m.o["dh"], m.o["dn2"], m.o["db2"], m.o["dw"], dbranch=m.o["dbranch"])
        m.head.update()
        out.append([m.o[k].clone() for k in ("dh", "dbranch", "dn2", "db2", "dw")] + list(m.head.state_n.snapshot().values()) + list(m.head.state_d.snapshot().values()))
    assert all(torch.equal(u, v) for u, v in zip(*out))
    hd = fm.Fp8VocabHead(1, 128, 300, device=device())
    hd.quantize_weights(m.w[:300].contiguous())
    x, loss, lse = bf(1, 128), f32(1), f32(1)
    hd.embed(torch.tensor([17], device=device()), x)
    hd.forward(x, None, m.n2, None, torch.tensor([5], device=device()), loss, lse, train=False)
    a, b = codec.decode(u8(hd.qn_infer), "e4m3"), codec.decode(u8(hd.qw), "e4m3")
    inv = hd.state_n.scale_inv.item() * hd.state_w.scale_inv_used.item()
    want, want_lse = me.cross_entropy(a @ b.T * inv, np.array([5]))
    B = 1e-5 * (np.abs(a) @ np.abs(b).T).max() * inv
    tol = 2 * B + SUMS + EW * 3 * np.abs(want_lse[0])
    assert abs(loss.item() - want[0]) < tol and abs(lse.item() - want_lse[0]) < tol
