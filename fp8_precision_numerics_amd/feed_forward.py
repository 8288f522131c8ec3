"""One gated feed-forward block on FP8 operands: residual addition and norm, gate
and up projections with activation and product, down projection with the
residual added; forward and backward under the HYBRID delayed-scaling recipe.

    s = x + residual                 the residual stream after the block before
    n = rms_norm(s) * weight         codes (E4M3)
    h = act(n Wg^T) * (n Wu^T)       codes (E4M3), both projections in one GEMM
    y = h Wd^T + s                   bf16

"4.2 Hopper I — Transformer Engine·FP8", §4.2.3 and §4.2.6: forward operands are
E4M3, gradients E5M2; §4.2.4: each tensor has its own delayed scale, and a GEMM's
restore is combined with the next stage's scale, so the activations between the
three products only ever exist as codes.

The class only sequences libfp8mi's kernels and owns the buffers, as Fp8Linear.
Any number of tokens runs forward (one token: the few-row kernels); the backward
needs a multiple of 16, the K granule of its weight-gradient GEMMs.
"""

from __future__ import annotations

import contextlib

import torch

from . import _binding as _b
from .state import DelayedScalingState, Recipe

# Scratch of one block: split products' partial sums, the norm's and the
# activation gradients' column sums, the statistics.
WORKSPACE_BYTES = 64 << 20


def _straddle(a, b):
    """Whether two contiguous tensors share memory without beginning at the same address."""
    p, q = a.data_ptr(), b.data_ptr()
    return p != q and p < q + b.numel() * b.element_size() and q < p + a.numel() * a.element_size()


def _on(stream):
    """Context in which torch works on what a `stream` argument names."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


class Fp8FeedForward:
    """Buffers and delayed-scaling states of one block: x, residual and y
    [tokens x hidden] bf16, w_gate_up [2 ffn x hidden] (the gate's rows, then the
    up projection's) and w_down [hidden x ffn] bf16, weight [hidden] bf16.  The calls share one
    workspace and the scales: on several streams, the caller puts them in order."""

    def __init__(self, tokens: int, hidden: int, ffn: int, act: str = "silu", eps: float = 1e-5,
                 recipe: Recipe = Recipe(), accum: str = "exact", device="cuda"):
        if recipe.fmt_fwd != "e4m3" or recipe.fmt_bwd != "e5m2":
            raise ValueError("Fp8FeedForward implements the HYBRID recipe (E4M3 forward, E5M2 backward)")
        if act not in _b.ACTIVATIONS:
            raise ValueError(f"unknown activation {act!r}")
        dev = torch.device(device)
        self.shape, self.act, self.eps, self.accum = (tokens, hidden, ffn), act, eps, accum

        def state(fmt):
            return DelayedScalingState(fmt, recipe.history_len, device=dev)

        fwd, bwd = recipe.fmt_fwd, recipe.fmt_bwd
        self.state_n, self.state_gu, self.state_h, self.state_d = state(fwd), state(fwd), state(fwd), state(fwd)
        self.state_dy, self.state_dgu = state(bwd), state(bwd)
        u8, bf = dict(dtype=torch.uint8, device=dev), dict(dtype=torch.bfloat16, device=dev)
        T, H, F = tokens, hidden, ffn
        self.sum, self.rstd = torch.empty((T, H), **bf), torch.empty(T, dtype=torch.float32, device=dev)
        # forward(train=False) has its own, so that what a backward takes stays as it is
        self.sum_infer = torch.empty((T, H), **bf)
        self.qn_infer, self.qh_infer = torch.empty((T, H), **u8), torch.empty((T, F), **u8)
        self.qn, self.qh, self.gu = torch.empty((T, H), **u8), torch.empty((T, F), **u8), torch.empty((T, 2 * F), **bf)
        self.qw_gu, self.qw_d = torch.empty((2 * F, H), **u8), torch.empty((H, F), **u8)
        self.qdy, self.qdy_t = torch.empty((T, H), **u8), torch.empty((H, T), **u8)
        self.dh, self.dn = torch.empty((T, F), **bf), torch.empty((T, H), **bf)
        self.qdgu, self.qdgu_t = torch.empty((T, 2 * F), **u8), torch.empty((2 * F, T), **u8)
        self.workspace = torch.empty(WORKSPACE_BYTES, **u8)
        self._kept = False  # the buffers and scales are those of one training forward

    def _check(self, t, shape, name):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")

    def quantize_weights(self, w_gate_up, w_down, stream=None):
        """Cast the weights with their current scales and set the scales of the next cast: once a
        training step, or once before serving.  The products take the inverse of the scale that
        the codes were cast with (scale_inv_used)."""
        T, H, F = self.shape
        self._check(w_gate_up, (2 * F, H), "w_gate_up")
        self._check(w_down, (H, F), "w_down")
        self._kept = False
        self.state_gu.quantize_update(w_gate_up, q=self.qw_gu, stream=stream)
        self.state_d.quantize_update(w_down, q=self.qw_d, stream=stream)

    def forward(self, x, residual, weight, y, train=True, stream=None):
        """y = down(act(gate(n)) * up(n)) + s, with the weights' codes as they are.
        residual may be None (s = x; a training forward keeps a copy).  y may be x or the residual.

        train: keep what backward needs, and the amaxes that update() takes.  Without it the
        call changes nothing that a backward or an update() sees, so it may come between a
        training forward and those; the scales that serving needs are settled by a few training
        forwards, each with an update()."""
        T, H, F = self.shape
        self._check(x, (T, H), "x")
        self._check(y, (T, H), "y")
        if residual is None and _straddle(x, y):
            raise ValueError("y shares part of its memory with x, which is the residual (residual=None)")
        if train:
            self._kept = False
        n, h, ws = self.state_n, self.state_h, self.workspace
        total, qn, qh = (self.sum, self.qn, self.qh) if train else (self.sum_infer, self.qn_infer, self.qh_infer)
        _b.fp8_rmsnorm_quantize(x, weight, self.eps, n.fmt, n.scale, qn, residual=residual,
                                sum_out=None if residual is None else total, rstd=self.rstd if train else None,
                                amax=n.amax if train else None, workspace=ws, stream=stream)
        if train and residual is None:
            with _on(stream):
                total.copy_(x)
        s = x if residual is None else total
        _b.fp8_gemm_gated(qn, n.fmt, self.qw_gu, self.state_gu.fmt, n.scale_inv, self.state_gu.scale_inv_used,
                          self.act, qh, gu=self.gu if train else None, out_fmt=h.fmt, out_scale=h.scale,
                          amax=h.amax if train else None, accum=self.accum, workspace=ws, stream=stream)
        _b.fp8_gemm_fused(qh, h.fmt, self.qw_d, self.state_d.fmt, h.scale_inv, self.state_d.scale_inv_used, y,
                          residual=s, accum=self.accum, workspace=ws, stream=stream)
        if train:
            self._kept = True

    def backward(self, dy, weight, dx, dweight, dw_gate_up, dw_down, stream=None):
        """Gradients of the last forward(train=True), as often as wanted until the weights are cast
        again or update() sets new scales: dx [tokens x hidden] bf16 (of x, hence of
        the residual too), dweight fp32 [hidden], dw_gate_up and dw_down (fp32 or bf16)."""
        T, H, F = self.shape
        if T % 16:
            raise ValueError(f"backward needs a multiple of 16 tokens, got {T}")
        self._check(dy, (T, H), "dy")
        self._check(dw_gate_up, (2 * F, H), "dw_gate_up")
        self._check(dw_down, (H, F), "dw_down")
        if not self._kept:
            raise RuntimeError("backward needs a training forward, with no quantize_weights or update since")
        sy, sg, ws = self.state_dy, self.state_dgu, self.workspace
        kw = dict(accum=self.accum, b_trans=True, stream=stream)
        # The cast of fp8_quantize with the same bits: 512 x 4096 7.7 us a call against 15.5, 8192 x 4096 31 against 28,
        # 8192 x 16384 93 against 111.
        _b.fp8_act_backward(dy, None, "none", sy.fmt, sy.scale, q=self.qdy, q_t=self.qdy_t, amax=sy.amax, workspace=ws,
                            stream=stream)
        _b.fp8_gemm(self.qdy, sy.fmt, self.qw_d, self.state_d.fmt, sy.scale_inv, self.state_d.scale_inv_used, self.dh,
                    **kw)
        _b.fp8_gemm(self.qdy_t, sy.fmt, self.qh, self.state_h.fmt, sy.scale_inv, self.state_h.scale_inv, dw_down, **kw)
        _b.fp8_gated_backward(self.dh, self.gu, self.act, sg.fmt, sg.scale, q=self.qdgu, q_t=self.qdgu_t, amax=sg.amax,
                              workspace=ws, stream=stream)
        _b.fp8_gemm(self.qdgu, sg.fmt, self.qw_gu, self.state_gu.fmt, sg.scale_inv, self.state_gu.scale_inv_used,
                    self.dn, **kw)
        _b.fp8_gemm(self.qdgu_t, sg.fmt, self.qn, self.state_n.fmt, sg.scale_inv, self.state_n.scale_inv, dw_gate_up, **kw)
        _b.fp8_rmsnorm_backward(self.dn, self.sum, self.rstd, weight, dx, dweight=dweight, dresidual=dy, workspace=ws,
                                stream=stream)

    def update(self, stream=None):
        """Push the activations' and gradients' amaxes into their histories and set the next step's
        scales.  The weights' are stepped where they are cast, so their codes outlive any number of updates."""
        self._kept = False
        for st in (self.state_n, self.state_h, self.state_dy, self.state_dgu):
            st.update(stream=stream)
