"""Host-only checks of the entry points at both ends of a model: argument combinations the
library refuses before touching a device (fake pointers, never dereferenced), and
the binding's own refusals.  Nothing here can reach a kernel."""

import ctypes

import pytest
import torch

import fp8_precision_numerics_amd as fm
from fp8_precision_numerics_amd import _binding as binding

OK, ENULL, ESHAPE, EALIGN, EFMT, EDTYPE, EACCUM, EWS = 0, -1, -2, -3, -4, -5, -8, -10
P, P8, P4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10004)   # 16-B, 8-B and 4-B aligned
P2 = ctypes.c_void_p(0x20000)
BIG = 1 << 41


@pytest.fixture(scope="module")
def lib():
    return fm.load_library()


def call(fn, defaults, **changes):
    args = dict(defaults, **changes)
    assert args.keys() == defaults.keys()
    return fn(*args.values())


NORM = dict(x=P, residual=P, weight=P, bias=P, xtype=1, rows=4, cols=64, eps=1e-5, dropout=0.1, rng=P, fmt=0, scale=P, sum_out=P, q=P,
            mean=None, rstd=None, amax=None, sat=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(xtype=7)), (EFMT, dict(fmt=5)), (ESHAPE, dict(rows=-1)), (ESHAPE, dict(rows=BIG)), (ESHAPE, dict(cols=-16)),
    (ESHAPE, dict(eps=-1.0)), (ESHAPE, dict(eps=float("nan"))), (EALIGN, dict(cols=72)), (ENULL, dict(x=None)), (ENULL, dict(weight=None)),
    (ENULL, dict(q=None)), (ENULL, dict(scale=None)), (EALIGN, dict(x=P8)), (EALIGN, dict(residual=P8)), (EALIGN, dict(weight=P8)),
    (EALIGN, dict(bias=P8)), (EALIGN, dict(sum_out=P8)), (EALIGN, dict(q=P8)), (EALIGN, dict(ws=P8, ws_bytes=64)), (EALIGN, dict(ws=P, ws_bytes=8)),
    (ESHAPE, dict(dropout=-0.1)), (ESHAPE, dict(dropout=1.0)), (ESHAPE, dict(dropout=float("nan"))), (ESHAPE, dict(dropout=0.999995)),
    (ENULL, dict(rng=None)), (EALIGN, dict(rng=P4)), (OK, dict(rows=0)), (OK, dict(cols=0, x=None, q=None, weight=None, scale=None))])
def test_norm_refusals(lib, want, change):
    assert call(lib.fp8_layernorm_quantize, NORM, **change) == want


NORM_BACK = dict(dy=P, h=P, mean=P, rstd=P, weight=P, dres=None, xtype=0, rows=4, cols=64, dropout=0.5, rng=P, dx=P, dbranch=P2, dweight=P, dbias=P,
                 ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(xtype=3)), (ESHAPE, dict(rows=-2)), (EALIGN, dict(cols=24)), (ENULL, dict(dy=None)), (ENULL, dict(h=None)), (ENULL, dict(mean=None)),
    (ENULL, dict(rstd=None)), (ENULL, dict(weight=None)), (ENULL, dict(dx=None)), (EALIGN, dict(dy=P8)), (EALIGN, dict(h=P8)),
    (EALIGN, dict(weight=P8)), (EALIGN, dict(dres=P8)), (EALIGN, dict(dx=P8)), (EALIGN, dict(dbranch=P8)), (EALIGN, dict(dweight=P8)),
    (EALIGN, dict(dbias=P8)), (EALIGN, dict(ws=P8)), (ENULL, dict(ws=None, ws_bytes=0)), (EWS, dict(ws_bytes=511)), (EWS, dict(ws_bytes=255, dbias=None)),
    (ESHAPE, dict(dbranch=P)), (ESHAPE, dict(dropout=1.5)), (ENULL, dict(rng=None)), (OK, dict(rows=0, dweight=None, dbias=None)), (OK, dict(cols=0))])
def test_norm_backward_refusals(lib, want, change):
    assert call(lib.fp8_layernorm_backward, NORM_BACK, **change) == want


EMBED = dict(tokens=P, itype=1, rows=4, table=P, ttype=2, vocab=100, cols=64, sinv=P, scale=1.0, out=P, otype=1, stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(itype=2)), (EDTYPE, dict(ttype=4)), (EDTYPE, dict(otype=2)), (ESHAPE, dict(rows=-1)), (ESHAPE, dict(vocab=-1)), (ESHAPE, dict(vocab=1 << 31)),
    (ESHAPE, dict(cols=-16)), (ESHAPE, dict(cols=(1 << 20) + 16)), (EALIGN, dict(cols=72)), (ENULL, dict(tokens=None)), (ENULL, dict(table=None)),
    (ENULL, dict(out=None)), (ENULL, dict(sinv=None)), (EALIGN, dict(tokens=P4)), (EALIGN, dict(tokens=ctypes.c_void_p(0x10002), itype=0)), (EALIGN, dict(table=P8)),
    (EALIGN, dict(out=P8)), (OK, dict(rows=0, tokens=None)), (OK, dict(cols=0))])
def test_embedding_refusals(lib, want, change):
    assert call(lib.fp8_embedding, EMBED, **change) == want


EMBED_BACK = dict(tokens=P, itype=0, rows=40, dy=P, dytype=1, vocab=100, cols=64, scale=1.0, base=None, dtable=P, ttype=0, ws=P, ws_bytes=2 * 160 + 3 * 2 * 64 * 4,
                  stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(itype=-1)), (EDTYPE, dict(dytype=2)), (EDTYPE, dict(ttype=3)), (ESHAPE, dict(rows=-1)), (ESHAPE, dict(rows=(1 << 20) + 1)), (ESHAPE, dict(vocab=-1)),
    (ESHAPE, dict(cols=(1 << 20) + 16)), (EALIGN, dict(cols=24)), (ENULL, dict(tokens=None)), (ENULL, dict(dy=None)), (ENULL, dict(dtable=None)), (ENULL, dict(ws=None)),
    (EALIGN, dict(dy=P8)), (EALIGN, dict(base=P8)), (EALIGN, dict(dtable=P8)), (EALIGN, dict(ws=P8)), (EALIGN, dict(tokens=ctypes.c_void_p(0x10002))),
    (EWS, dict(ws_bytes=2 * 160 + 3 * 2 * 64 * 4 - 1)), (OK, dict(vocab=0)), (OK, dict(cols=0)), (OK, dict(rows=0, base=P))])
def test_embedding_backward_refusals(lib, want, change):
    assert call(lib.fp8_embedding_backward, EMBED_BACK, **change) == want


def test_embedding_workspace():
    """Keys and places of 4 bytes a token (twice where blocks of 8192 are merged), two partial rows for each chunk of 16 (or a 4096th of the tokens, up to eights)."""
    assert fm.embedding_workspace_bytes(0, 64) == 0 and fm.embedding_workspace_bytes(-1, 64) == 0 and fm.embedding_workspace_bytes((1 << 20) + 1, 64) == 0
    assert fm.embedding_workspace_bytes(16, 64) == 2 * 64 and fm.embedding_workspace_bytes(17, 64) == 2 * 80 + 2 * 2 * 64 * 4
    assert fm.embedding_workspace_bytes(8192, 64) == 2 * 32768 + 512 * 512 and fm.embedding_workspace_bytes(8193, 64) == 4 * 32784 + 513 * 512
    assert fm.embedding_workspace_bytes(1 << 20, 64) == 4 * (4 << 20) + 4096 * 512


LEAST = 256 * 32 + 256 * 128 + 32 * 64 * 4   # 32 rows: codes both ways for 256 columns (rows padded to 128), and dx's sums
VOCAB = dict(x=P, fx=0, w=P, fw=0, M=32, V=1000, K=64, sx=P, sw=P, targets=P, itype=1, loss=P, lse=P, accum=0, ws=P, ws_bytes=32 * 4 + 32 * 8 + 32 * 8 * 2, stream=None)
VOCAB_BACK = dict(x=P, fx=0, w=P, fw=0, M=32, V=1000, K=64, sx=P, sw=P, targets=P, itype=0, lse=P, dloss=P, fmt=1, scale=P, inv=P, dx=P, dxtype=1, dw=P, dwtype=0,
                  amax=None, sat=None, accum=1, ws=P, ws_bytes=LEAST, stream=None)
VOCAB_BAD = [(EFMT, dict(fx=2)), (EFMT, dict(fw=-1)), (EDTYPE, dict(itype=2)), (EACCUM, dict(accum=2)), (ESHAPE, dict(M=-1)), (ESHAPE, dict(V=0)), (ESHAPE, dict(K=0)),
             (ESHAPE, dict(V=1 << 31)), (ESHAPE, dict(M=(1 << 23) - 15, K=16)), (ESHAPE, dict(M=1 << 20, K=2048)), (ESHAPE, dict(K=(1 << 22) + 16)), (EALIGN, dict(K=72)),
             (EALIGN, dict(ws=P8)), (ENULL, dict(x=None)), (ENULL, dict(w=None)), (ENULL, dict(sx=None)), (ENULL, dict(sw=None)), (ENULL, dict(targets=None)),
             (ENULL, dict(ws=None)), (EALIGN, dict(x=P8)), (EALIGN, dict(w=P8)), (EALIGN, dict(targets=ctypes.c_void_p(0x10002)))]


@pytest.mark.parametrize("want,change", VOCAB_BAD + [
    (EALIGN, dict(targets=P4)), (ENULL, dict(loss=None, lse=None)), (EWS, dict(ws_bytes=32 * 4 + 32 * 8 + 32 * 8 * 2 - 1)), (OK, dict(M=0, x=None, ws=None, ws_bytes=0)),
    (OK, dict(M=0, loss=None, lse=None))])
def test_vocab_refusals(lib, want, change):
    assert call(lib.fp8_vocab_cross_entropy, VOCAB, **change) == want


@pytest.mark.parametrize("want,change", VOCAB_BAD + [
    (EFMT, dict(fmt=2)), (EDTYPE, dict(dxtype=2)), (EDTYPE, dict(dwtype=-1)), (ENULL, dict(dx=None, dw=None)), (EALIGN, dict(dx=P8)), (EALIGN, dict(dw=P8)),
    (ENULL, dict(lse=None)), (ENULL, dict(dloss=None)), (ENULL, dict(scale=None)), (ENULL, dict(inv=None)), (EWS, dict(ws_bytes=LEAST - 1)),
    (OK, dict(M=0, dw=None)), (OK, dict(M=0, dx=None, dw=None, x=None))])
def test_vocab_backward_refusals(lib, want, change):
    assert call(lib.fp8_vocab_cross_entropy_backward, VOCAB_BACK, **change) == want


def test_vocab_workspace():
    assert fm.vocab_workspace_bytes(0, 1000, 64) == 0 and fm.vocab_workspace_bytes(32, 0, 64) == 0 and fm.vocab_workspace_bytes(32, 1000, (1 << 22) + 16) == 0
    assert fm.vocab_workspace_bytes(32, 1000, 64, 0) == LEAST and fm.vocab_workspace_bytes(32, 1000, 64, 4) == LEAST
    # one piece: codes of 1000 columns, rows of 1024 and of 128, each rounded up to 256
    assert fm.vocab_workspace_bytes(32, 1000, 64) == 32768 + 128000
    # a whole vocabulary of few columns needs no sums of dx, and less than a piece with them
    assert fm.vocab_workspace_bytes(16, 300, 1024, 0) == fm.vocab_workspace_bytes(16, 300, 1024) == 16 * 384 + 300 * 128
    assert fm.vocab_workspace_bytes(16, 300, 64, 0) == 16 * 256 + 256 * 128 + 16 * 64 * 4


@pytest.mark.parametrize("name", ["layer", "layer_back", "embed", "embed_back", "vocab", "vocab_back"])
def test_a_wrong_number_of_arguments_is_a_type_error(name):
    module = binding._MODULE or binding._load_module()
    with pytest.raises(TypeError):
        getattr(module, name)(0, 0)
    with pytest.raises(TypeError):
        getattr(module, name)(*[None] * 40)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 32), torch.zeros(32)
    q, one = torch.zeros(4, 32, dtype=torch.uint8), torch.ones(1)
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_layernorm_quantize(x, w, w, 1e-5, "e4m3", one, q)
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_layernorm_backward(x, x, torch.ones(4), torch.ones(4), w, x)
