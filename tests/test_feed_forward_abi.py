"""Host-only checks of the feed-forward entry points: argument combinations the
library refuses before touching a device (fake pointers, never dereferenced), and
the binding's own refusals.  Nothing here can reach a kernel."""

import ctypes

import pytest
import torch

import fp8_precision_numerics_amd as fm

OK, ENULL, ESHAPE, EALIGN, EFMT, EDTYPE, EACCUM, EACT, EWS = 0, -1, -2, -3, -4, -5, -8, -9, -10
P, P8 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)   # 16-B aligned, misaligned
BIG = 1 << 41


@pytest.fixture(scope="module")
def lib():
    return fm.load_library()


def call(fn, defaults, **changes):
    args = dict(defaults, **changes)
    assert args.keys() == defaults.keys()
    return fn(*args.values())


NORM = dict(x=P, residual=P, weight=P, xtype=1, rows=4, cols=64, eps=1e-5, fmt=0, scale=P, sum_out=P, q=P, rstd=None, amax=None,
            sat=None, ws=None, ws_bytes=0, stream=None)


def test_status_strings():
    assert "activation" in fm.status_string(EACT) and "workspace" in fm.status_string(EWS)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(xtype=7)), (EFMT, dict(fmt=5)), (ESHAPE, dict(rows=-1)), (ESHAPE, dict(rows=BIG)), (ESHAPE, dict(cols=-16)),
    (ESHAPE, dict(eps=-1.0)), (ESHAPE, dict(eps=float("nan"))), (EALIGN, dict(cols=72)), (ENULL, dict(x=None)), (ENULL, dict(weight=None)),
    (ENULL, dict(q=None)), (ENULL, dict(scale=None)), (ENULL, dict(residual=None)), (EALIGN, dict(x=P8)), (EALIGN, dict(residual=P8)),
    (EALIGN, dict(weight=P8)), (EALIGN, dict(sum_out=P8)), (EALIGN, dict(q=P8)), (EALIGN, dict(ws=P8, ws_bytes=64)),
    (EALIGN, dict(ws=P, ws_bytes=8)), (OK, dict(rows=0)), (OK, dict(cols=0, x=None, q=None, weight=None, scale=None))])
def test_norm_refusals(lib, want, change):
    assert call(lib.fp8_rmsnorm_quantize, NORM, **change) == want


NORM_BLOCKS = dict(x=P, residual=P, weight=P, xtype=1, rows=4, cols=64, eps=1e-5, fmt=0, sum_out=P, q=P, scale_inv=P, rstd=None, stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(xtype=2)), (EFMT, dict(fmt=-1)), (EALIGN, dict(cols=40)), (ENULL, dict(scale_inv=None)), (ENULL, dict(residual=None)),
    (ENULL, dict(q=None)), (EALIGN, dict(q=P8)), (ESHAPE, dict(eps=-1e-9)), (OK, dict(rows=0))])
def test_norm_blockwise_refusals(lib, want, change):
    assert call(lib.fp8_rmsnorm_quantize_blockwise, NORM_BLOCKS, **change) == want


NORM_BACK = dict(dy=P, h=P, rstd=P, weight=P, dres=None, xtype=0, rows=4, cols=64, dx=P, dweight=P, ws=P, ws_bytes=256, stream=None)


@pytest.mark.parametrize("want,change", [
    (EDTYPE, dict(xtype=3)), (ESHAPE, dict(rows=-2)), (EALIGN, dict(cols=24)), (ENULL, dict(dy=None)), (ENULL, dict(h=None)),
    (ENULL, dict(rstd=None)), (ENULL, dict(weight=None)), (ENULL, dict(dx=None)), (EALIGN, dict(dy=P8)), (EALIGN, dict(h=P8)),
    (EALIGN, dict(weight=P8)), (EALIGN, dict(dres=P8)), (EALIGN, dict(dx=P8)), (EALIGN, dict(dweight=P8)), (EALIGN, dict(ws=P8)), (ENULL, dict(ws=None, ws_bytes=0)),
    (EWS, dict(ws_bytes=255)), (OK, dict(rows=0, dweight=None)), (OK, dict(cols=0))])
def test_norm_backward_refusals(lib, want, change):
    assert call(lib.fp8_rmsnorm_backward, NORM_BACK, **change) == want


GATED = dict(a=P, fa=0, b=P, fb=0, M=32, F=48, K=64, sa=P, sb=P, act=2, h=P, htype=2, scale=P, gu=None, amax=None, sat=None, accum=0, ws=None,
             ws_bytes=0, stream=None)
FUSED = dict(a=P, fa=0, b=P, fb=0, M=32, N=48, K=64, sa=P, sb=P, bias=None, act=0, residual=None, y=P, ytype=1, scale=None, z=None, amax=None,
             sat=None, accum=0, ws=None, ws_bytes=0, stream=None)
GEMM_BAD = [(EFMT, dict(fa=2)), (EFMT, dict(fb=-1)), (EACT, dict(act=4)), (EACT, dict(act=-1)), (EACCUM, dict(accum=2)), (ESHAPE, dict(M=-1)),
            (ESHAPE, dict(K=0)), (ESHAPE, dict(K=(1 << 23) + 16)), (ESHAPE, dict(M=1 << 32)), (EALIGN, dict(K=72)), (ENULL, dict(a=None)),
            (ENULL, dict(b=None)), (ENULL, dict(sa=None)), (ENULL, dict(sb=None)), (EALIGN, dict(a=P8)), (EALIGN, dict(b=P8)),
            (EALIGN, dict(ws=P8, ws_bytes=64)), (OK, dict(M=0))]


@pytest.mark.parametrize("want,change", GEMM_BAD + [
    (EDTYPE, dict(htype=4)), (EDTYPE, dict(htype=1, amax=P)), (EDTYPE, dict(htype=0, sat=P)), (ENULL, dict(scale=None)), (ENULL, dict(h=None)),
    (EALIGN, dict(h=P8)), (EALIGN, dict(gu=P8)), (ESHAPE, dict(F=-1)), (ESHAPE, dict(F=1 << 30)), (OK, dict(F=0))])
def test_gated_refusals(lib, want, change):
    assert call(lib.fp8_gemm_gated, GATED, **change) == want


@pytest.mark.parametrize("want,change", GEMM_BAD + [
    (EDTYPE, dict(ytype=-1)), (EDTYPE, dict(amax=P)), (ENULL, dict(ytype=3)), (ENULL, dict(y=None)), (EALIGN, dict(y=P8)), (EALIGN, dict(z=P8)),
    (EALIGN, dict(bias=P8)), (EALIGN, dict(residual=P8)), (ESHAPE, dict(N=-1)), (OK, dict(N=0))])
def test_fused_refusals(lib, want, change):
    assert call(lib.fp8_gemm_fused, FUSED, **change) == want


ACT_BACK = dict(dy=P, xtype=1, z=P, act=3, M=32, N=48, fmt=1, scale=P, q=P, qt=P, dbias=P, amax=None, sat=None, ws=P, ws_bytes=4 * 48, stream=None)
GATED_BACK = dict(dh=P, xtype=1, gu=P, act=2, M=32, F=48, fmt=1, scale=P, q=P, qt=P, amax=None, sat=None, ws=None, ws_bytes=0, stream=None)
BACK_BAD = [(EDTYPE, dict(xtype=2)), (EFMT, dict(fmt=2)), (EACT, dict(act=9)), (ESHAPE, dict(M=-1)), (EALIGN, dict(M=24)), (ENULL, dict(scale=None)),
            (EALIGN, dict(q=P8)), (EALIGN, dict(qt=P8)), (EALIGN, dict(ws=P8, ws_bytes=4096)), (EALIGN, dict(ws=P, ws_bytes=8)), (ESHAPE, dict(M=BIG))]


@pytest.mark.parametrize("want,change", BACK_BAD + [
    (EALIGN, dict(N=40)), (ESHAPE, dict(N=-16)), (ESHAPE, dict(N=(1 << 25) + 16)), (ENULL, dict(dy=None)), (ENULL, dict(z=None)),
    (EALIGN, dict(dy=P8)), (EALIGN, dict(z=P8)), (ENULL, dict(ws=None, ws_bytes=0)), (EWS, dict(ws_bytes=4 * 48 - 1)),
    (ENULL, dict(q=None, qt=None, dbias=None)), (OK, dict(M=0, dbias=None)), (OK, dict(N=0))])
def test_act_backward_refusals(lib, want, change):
    assert call(lib.fp8_act_backward, ACT_BACK, **change) == want


@pytest.mark.parametrize("want,change", BACK_BAD + [
    (EALIGN, dict(F=40)), (ESHAPE, dict(F=-16)), (ESHAPE, dict(F=(1 << 24) + 16)), (ENULL, dict(dh=None)), (ENULL, dict(gu=None)),
    (ENULL, dict(gu=None, act=0)), (EALIGN, dict(dh=P8)), (EALIGN, dict(gu=P8)), (ENULL, dict(q=None, qt=None)), (OK, dict(M=0)), (OK, dict(F=0))])
def test_gated_backward_refusals(lib, want, change):
    assert call(lib.fp8_gated_backward, GATED_BACK, **change) == want


def test_binding_refuses_host_tensors_and_unknown_names():
    x, w = torch.zeros(4, 32), torch.zeros(32)
    q, one = torch.zeros(4, 32, dtype=torch.uint8), torch.ones(1)
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_rmsnorm_quantize(x, w, 1e-5, "e4m3", one, q)
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_rmsnorm_backward(x, x, torch.ones(4), w, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_gemm_fused(q, "e4m3", q, "e4m3", one, one, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        fm.fp8_act_backward(x, None, "none", "e5m2", one, q=q)
    with pytest.raises(ValueError, match="activation"):
        fm.Fp8FeedForward(16, 32, 32, act="tanh", device="cpu")
    with pytest.raises(ValueError, match="HYBRID"):
        fm.Fp8FeedForward(16, 32, 32, recipe=fm.Recipe(fmt_fwd="e5m2"), device="cpu")
