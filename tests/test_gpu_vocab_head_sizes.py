"""Fp8VocabHead at sizes that its other tests leave out: no tokens (a rank whose batch is empty), and a lookup of fewer tokens than
the head's where those take the larger scratch."""

import torch

import pytest

import fp8_precision_numerics_amd as fm
from gpu_helpers import announce, device

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_no_tokens():
    """All sums are zeros, nothing is refused, and the scales stay: no value has been seen."""
    announce("head of no tokens")
    H, V = 128, 300
    hd = fm.Fp8VocabHead(0, H, V, dropout=0.1, device=device())
    w = torch.randn(V, H, device=device()).to(BF)
    hd.quantize_weights(w)
    e, f = torch.empty((0, H), dtype=BF, device=device()), torch.empty(0, device=device())
    ids, rng = torch.empty(0, dtype=torch.int64, device=device()), torch.tensor([1, 2], device=device())
    nw = torch.ones(H, dtype=BF, device=device())
    scales = [s.scale.clone() for s in (hd.state_n, hd.state_d)]
    hd.embed(ids, e)
    hd.forward(e, e, nw, nw, ids, f, f, rng=rng)
    for dtype in (BF, torch.float32):
        dw, dn, db = torch.full((V, H), 7.0, dtype=dtype, device=device()), torch.full((H,), 7.0, device=device()), torch.full((H,), 7.0, device=device())
        hd.backward(f, nw, e, dn, db, dw, dbranch=torch.empty_like(e))
        hd.embed_backward(ids, e, dw)
        assert (dw == 0).all() and (dn == 0).all() and (db == 0).all()
    assert hd.state_n.amax.item() == 0 and hd.state_d.amax.item() == 0
    hd.update()
    assert all(torch.equal(s.scale, old) for s, old in zip((hd.state_n, hd.state_d), scales))


def test_a_lookup_of_fewer_tokens():
    """A head of 70000 tokens adds the gradient of 65536: whole numbers, so the sums are exact."""
    announce("head of 70000 tokens, lookup of 65536")
    T, H, V, n = 70000, 1024, 40, 65536
    hd = fm.Fp8VocabHead(T, H, V, pieces=1, device=device())
    hd.workspace = hd.workspace[:fm.embedding_workspace_bytes(T, H)]        # no more than the lookup asks for
    g = torch.Generator(device=device()).manual_seed(1)
    tokens = torch.randint(0, V, (n,), generator=g, device=device())
    dy = torch.randint(-4, 5, (n, H), generator=g, device=device()).to(BF)
    dw = torch.randint(-9, 9, (V, H), generator=g, device=device()).float()
    want = dw.double().index_add_(0, tokens, dy.double())
    hd.embed_backward(tokens, dy, dw)
    assert torch.equal(dw.double(), want)
