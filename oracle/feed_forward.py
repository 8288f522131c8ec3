"""The feed-forward operators around the FP8 GEMM in fp64 (test infrastructure; CPU oracle).

Definitions
-----------
``rms_norm``        y = h * r * w, r = (mean h^2 + eps)^(-1/2) along the last axis.
``rms_norm_grad``   its gradient: dh = r (g - h r^2 mean(g h)), g = dy * w, and
                    dw = sum over the rows of dy h r.
``activation``      value and derivative of none, relu, silu (z / (1 + e^-z)) and
                    gelu (the tanh form, z (1 + tanh(sqrt(2/pi)(z + 0.044715 z^3))) / 2).
``gated``           act(g) * u, and its gradient (dh u act'(g), dh act(g)).

Everything is fp64; rounding to the operator's output types is the caller's.

Parity status: pinned in tests/test_oracle_feed_forward.py: the norm by closed forms
(constant rows, rows of one nonzero), the activations by their limits and by
independent forms (tanh against the logistic function), every
gradient by central differences of the value.
"""

from __future__ import annotations

import numpy as np

__all__ = ["rms_norm", "rms_norm_grad", "activation", "gated", "gated_grad"]

C, A = np.sqrt(2.0 / np.pi), 0.044715


def rms_norm(h, w, eps):
    """(y, r) of rows h [M x N]."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
        return h * r[:, None] * np.asarray(w, dtype=np.float64), r


def rms_norm_grad(dy, h, w, eps, r=None):
    """(dh, dw); `r`: the forward's reciprocal norms, where they are given rather than taken from h."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, w))
    if r is None:
        r = rms_norm(h, w, eps)[1]
    r = np.asarray(r, dtype=np.float64)[:, None]
    g = dy * w
    dh = r * (g - h * r * r * np.mean(g * h, axis=1, keepdims=True))
    return dh, np.sum(dy * h * r, axis=0)


def activation(z, act):
    """(value, derivative)."""
    z = np.asarray(z, dtype=np.float64)
    if act == "none":
        return z.copy(), np.ones_like(z)
    if act == "relu":
        return np.where(np.isnan(z), z, np.maximum(z, 0.0)), (z > 0).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "silu":
            s = 1.0 / (1.0 + np.exp(-z))
            return z * s, s + z * s * (1.0 - s)
        t = np.tanh(C * (z + A * z ** 3))
        return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C * (1.0 + 3.0 * A * z * z)


def gated(g, u, act):
    return activation(g, act)[0] * np.asarray(u, dtype=np.float64)


def gated_grad(dh, g, u, act):
    """(dg, du)."""
    v, d = activation(g, act)
    dh = np.asarray(dh, dtype=np.float64)
    return dh * np.asarray(u, dtype=np.float64) * d, dh * v
