"""Both ends of a model on FP8 operands that share one weight: the embedding in front
of its blocks, and behind them the last norm, the vocabulary's projection and
the loss; forward and backward under the HYBRID delayed-scaling recipe.

    x0 = scale * W[token]                       embedding, from the weight's codes
    h = drop(x) + residual                      the last block's branch and the stream
    n = layer_norm(h) * weight + bias           codes (E4M3)
    loss = log sum exp(n W^T) - (n W^T)[target] per row; the logits are never stored

"4.2 Hopper I — Transformer Engine·FP8", §4.2.3 and §4.2.6: forward operands are
E4M3, gradients E5M2; §4.2.4: each tensor has its own delayed scale.  The gradient
of the logits exists only as codes, of a piece of the vocabulary at a time.

The class only sequences libfp8mi's kernels and owns the buffers, as Fp8FeedForward.
"""

from __future__ import annotations

import torch

from . import _binding as _b
from .feed_forward import WORKSPACE_BYTES, _on
from .state import DelayedScalingState, Recipe


class Fp8VocabHead:
    """Buffers and delayed-scaling states for x, residual [tokens x hidden] bf16, a weight [vocab x hidden] (bf16 or
    fp32, hidden a multiple of 16), norm weight and bias [hidden] bf16 and one target a row.  `pieces`: in how many
    pieces of the vocabulary the gradient is taken, which sizes the workspace (vocab_workspace_bytes).  The calls share that
    workspace and the scales: on several streams, the caller puts them in order."""

    def __init__(self, tokens: int, hidden: int, vocab: int, eps: float = 1e-5, dropout: float = 0.0, pieces: int = 4,
                 recipe: Recipe = Recipe(), accum: str = "exact", device="cuda"):
        if recipe.fmt_fwd != "e4m3" or recipe.fmt_bwd != "e5m2":
            raise ValueError("Fp8VocabHead implements the HYBRID recipe (E4M3 forward, E5M2 backward)")
        if not 0.0 <= dropout < 1.0 or round(dropout * 65536) > 65535:
            raise ValueError(f"dropout must be in [0, 1), in steps of 2^-16, got {dropout}")
        dev = torch.device(device)
        self.shape, self.eps, self.dropout, self.accum = (tokens, hidden, vocab), eps, dropout, accum
        self.state_n, self.state_w = (DelayedScalingState(recipe.fmt_fwd, recipe.history_len, device=dev) for _ in range(2))
        self.state_d = DelayedScalingState(recipe.fmt_bwd, recipe.history_len, device=dev)
        u8, bf, f32 = (dict(dtype=t, device=dev) for t in (torch.uint8, torch.bfloat16, torch.float32))
        T, H, V = tokens, hidden, vocab
        self.qw, self.qn, self.qn_infer = torch.empty((V, H), **u8), torch.empty((T, H), **u8), torch.empty((T, H), **u8)
        self.sum, self.dn = torch.empty((T, H), **bf), torch.empty((T, H), **bf)
        self.mean, self.rstd, self.lse = (torch.empty(T, **f32) for _ in range(3))
        # what a training forward was given and its backward needs again
        self.targets, self.rng = torch.empty(T, dtype=torch.int64, device=dev), torch.zeros(2, dtype=torch.int64, device=dev)
        self.workspace = torch.empty(max(WORKSPACE_BYTES, _b.vocab_workspace_bytes(T, V, H, pieces), _b.embedding_workspace_bytes(T, H)), **u8)
        self._cast = False  # the weight has codes
        self._kept = False  # the buffers and scales are those of one training forward

    def _check(self, t, shape, name, dtype=None):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")

    def _need_codes(self):
        if not self._cast:
            raise RuntimeError("the weight has no codes yet: call quantize_weights first")

    def quantize_weights(self, weight, stream=None):
        """Cast the weight with its current scale and set the scale of the next cast: once a training step, or once
        before serving.  Lookups and products take the inverse of the scale that the codes were cast with."""
        T, H, V = self.shape
        self._check(weight, (V, H), "weight")
        self._kept = False
        self.state_w.quantize_update(weight, q=self.qw, stream=stream)
        self._cast = True

    def embed(self, tokens, out, scale: float = 1.0, stream=None):
        """out [n x hidden] (bf16 or fp32) = scale * the weight's rows, from its codes; zeros for a token outside the vocabulary."""
        self._need_codes()
        _b.fp8_embedding(tokens, self.qw, out, scale=scale, fmt=self.state_w.fmt, sinv=self.state_w.scale_inv_used, stream=stream)

    def embed_backward(self, tokens, dy, dw, scale: float = 1.0, stream=None):
        """Adds the lookup's gradient (dy [n x hidden], n up to the head's tokens and 2^20) to dw [vocab x hidden], which holds the projection's."""
        T, H, V = self.shape
        self._check(dw, (V, H), "dw")
        if tokens.numel() > T:
            raise ValueError(f"at most {T} tokens, got {tokens.numel()}")
        _b.fp8_embedding_backward(tokens, dy, dw, scale=scale, base=dw, workspace=self.workspace, stream=stream)

    def forward(self, x, residual, norm_weight, norm_bias, targets, loss, lse=None, rng=None, train=True, stream=None):
        """loss fp32 [tokens] of the targets (int32 or int64; 0 for a row whose target lies outside the vocabulary), and
        its log sum exp into lse where that is given.  residual and norm_bias may be None.

        train: values of x are dropped (with a dropout, rng is needed: int64[2], {seed, offset}), and what
        backward and update() need is kept.  Without it nothing is dropped and the call changes nothing that a backward or
        an update() sees, so it may come between a training forward and those."""
        T, H, V = self.shape
        self._need_codes()
        self._check(x, (T, H), "x")
        self._check(targets, (T,), "targets")
        drop = self.dropout if train else 0.0
        if drop:
            if rng is None:
                raise ValueError("a training forward with dropout needs rng")
            self._check(rng, (2,), "rng", torch.int64)
        if lse is not None:
            self._check(lse, (T,), "lse", torch.float32)
        if train:
            self._kept = False
            with _on(stream):
                self.targets.copy_(targets)
                if drop:
                    self.rng.copy_(rng)
        n, w, ws = self.state_n, self.state_w, self.workspace
        qn = self.qn if train else self.qn_infer
        _b.fp8_layernorm_quantize(x, norm_weight, norm_bias, self.eps, n.fmt, n.scale, qn, residual=residual,
                                  sum_out=self.sum if train else None, mean=self.mean if train else None,
                                  rstd=self.rstd if train else None, amax=n.amax if train else None, dropout=drop,
                                  rng=self.rng if drop else None, workspace=ws, stream=stream)
        kept = self.lse if train else lse
        _b.fp8_vocab_cross_entropy(qn, n.fmt, self.qw, w.fmt, n.scale_inv, w.scale_inv_used, targets, loss, kept,
                                   accum=self.accum, workspace=ws, stream=stream)
        if train:
            if lse is not None:
                with _on(stream):
                    lse.copy_(kept)
            self._kept = True

    def backward(self, dloss, norm_weight, dx, dweight, dbias, dw, dbranch=None, stream=None):
        """Gradients of sum(dloss * loss) for the last forward(train=True), as often as wanted until the weight is cast
        again or update() sets new scales: dx [tokens x hidden] bf16 (of h, hence of the residual), dbranch likewise
        (of x, through the dropout; may be None), dweight and dbias fp32 [hidden] (either may be None), dw [vocab x hidden]
        (fp32 or bf16; None where the weight is frozen)."""
        T, H, V = self.shape
        self._check(dloss, (T,), "dloss")
        if dw is not None:
            self._check(dw, (V, H), "dw")
        if not self._kept:
            raise RuntimeError("backward needs a training forward, with no quantize_weights or update since")
        n, w, d, ws = self.state_n, self.state_w, self.state_d, self.workspace
        _b.fp8_vocab_cross_entropy_backward(self.qn, n.fmt, self.qw, w.fmt, n.scale_inv, w.scale_inv_used, self.targets, self.lse,
                                            dloss, d.fmt, d.scale, d.scale_inv, dx=self.dn, dw=dw, amax=d.amax, accum=self.accum,
                                            workspace=ws, stream=stream)
        drop = self.dropout if dbranch is not None else 0.0
        _b.fp8_layernorm_backward(self.dn, self.sum, self.mean, self.rstd, norm_weight, dx, dweight=dweight, dbias=dbias,
                                  dbranch=dbranch, dropout=drop, rng=self.rng if drop else None, workspace=ws, stream=stream)

    def update(self, stream=None):
        """Push the amaxes of the norm's output and of the logits' gradient into their histories and set the next step's
        scales.  The weight's is stepped where it is cast, so its codes outlive any number of updates."""
        self._kept = False
        for st in (self.state_n, self.state_d):
            st.update(stream=stream)
