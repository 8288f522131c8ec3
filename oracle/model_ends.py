"""The operators at both ends of a model in fp64 (test infrastructure; CPU oracle).

Definitions
-----------
``philox4x32``       the counter-based generator of Salmon, Moraes, Dror and Shaw ("Parallel
                     random numbers: as easy as 1, 2, 3", SC 2011), 10 rounds.
``dropout_factors``  what each value of a tensor is multiplied with: 0 where its 16 random
                     bits are below T = round(65536 p), else 65536 / (65536 - T).  Value i takes
                     half-word i % 8 of the generator's 128 bits for the counter (i // 8, offset)
                     and the key seed.
``layer_norm``       y = (h - m) r w + b, m the mean and r = (mean (h - m)^2 + eps)^(-1/2) along the last axis.
``layer_norm_grad``  dh = r (g - mean g - a mean(g a)), g = dy w, a = (h - m) r; dw = sum dy a; db = sum dy.
``cross_entropy``    log sum exp of each row of logits, and that minus the target's logit
                     (0 where the target lies outside the row).
``cross_entropy_grad``  dloss (exp(z - lse) - [column = target]); a row of zeros where the target lies outside.
``embedding``        scale * table[id], zeros where the id lies outside the table.
``embedding_grad``   base + scale * the sum of dy over the places of each id.

Everything is fp64 (the generator: integers); rounding to the operator's output types is the caller's.

Parity status: pinned in tests/test_oracle_model_ends.py: the generator by the known answers its
authors publish, the norm and the loss by closed forms, every gradient by central
differences of the value.
"""

from __future__ import annotations

import numpy as np

__all__ = ["philox4x32", "dropout_cut", "dropout_factors", "layer_norm", "layer_norm_grad", "cross_entropy",
           "cross_entropy_grad", "embedding", "embedding_grad"]

MASK = 0xFFFFFFFF


def philox4x32(counter, key, rounds=10):
    """Four words of 32 bits for one counter (four words) and key (two words), in Python integers."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & MASK, (a >> 32) ^ c[3] ^ k[1], a & MASK]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return c


def dropout_cut(p):
    """T = round(65536 p) of an fp32 probability (ties to even)."""
    return int(np.rint(float(np.float32(p)) * 65536.0))


def dropout_factors(shape, p, seed, offset, first=0):
    """Factors of a tensor of `shape` (fp64); `first`: number of its first octet."""
    n = int(np.prod(shape))
    groups = (n + 7) // 8
    u = np.uint64
    lo, half = u(MASK), u(32)
    g = np.arange(groups, dtype=np.uint64) + u(first)
    seed, offset = int(seed) & (1 << 64) - 1, int(offset) & (1 << 64) - 1
    c = [g & lo, g >> half, np.full(groups, offset & MASK, dtype=np.uint64), np.full(groups, offset >> 32, dtype=np.uint64)]
    k = [seed & MASK, seed >> 32]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ u(k[0]), b & lo, (a >> half) ^ c[3] ^ u(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    words = np.stack(c, axis=1)
    bits = np.stack([words & u(0xFFFF), words >> u(16)], axis=2).reshape(-1)[:n].astype(np.int64)
    cut = dropout_cut(p)
    return np.where(bits < cut, 0.0, 65536.0 / (65536 - cut)).reshape(shape)


def layer_norm(h, w, b, eps):
    """(y, mean, r) of rows h [M x N]; b may be None."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        m = np.mean(h, axis=1)
        d = h - m[:, None]
        r = 1.0 / np.sqrt(np.mean(d * d, axis=1) + eps)
        y = d * r[:, None] * np.asarray(w, dtype=np.float64)
        return (y if b is None else y + np.asarray(b, dtype=np.float64)), m, r


def layer_norm_grad(dy, h, w, eps, m=None, r=None):
    """(dh, dw, db); `m`, `r`: the forward's, where they are given rather than taken from h."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, w))
    if m is None or r is None:
        _, m, r = layer_norm(h, w, None, eps)
    m, r = (np.asarray(t, dtype=np.float64)[:, None] for t in (m, r))
    a, g = (h - m) * r, dy * w
    dh = r * (g - np.mean(g, axis=1, keepdims=True) - a * np.mean(g * a, axis=1, keepdims=True))
    return dh, np.sum(dy * a, axis=0), np.sum(dy, axis=0)


def cross_entropy(z, target):
    """(loss, lse) of rows of logits z [M x V]."""
    z = np.asarray(z, dtype=np.float64)
    t = np.asarray(target, dtype=np.int64)
    top = np.max(z, axis=1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = top + np.log(np.sum(np.exp(z - top[:, None]), axis=1))
    inside = (t >= 0) & (t < z.shape[1])
    mine = z[np.arange(len(t)), np.where(inside, t, 0)]
    return np.where(inside, lse - mine, 0.0), lse


def cross_entropy_grad(z, target, dloss, lse=None):
    """Gradient of sum(dloss * loss) in the logits; `lse`: the forward's, where it is given."""
    z = np.asarray(z, dtype=np.float64)
    t = np.asarray(target, dtype=np.int64)
    if lse is None:
        lse = cross_entropy(z, t)[1]
    inside = (t >= 0) & (t < z.shape[1])
    d = np.exp(z - np.asarray(lse, dtype=np.float64)[:, None])
    d[np.flatnonzero(inside), t[inside]] -= 1.0
    return np.where(inside[:, None], d * np.asarray(dloss, dtype=np.float64)[:, None], 0.0)


def embedding(ids, table, scale=1.0):
    table = np.asarray(table, dtype=np.float64)
    ids = np.asarray(ids, dtype=np.int64)
    inside = (ids >= 0) & (ids < table.shape[0])
    return np.where(inside[:, None], table[np.where(inside, ids, 0)] * scale, 0.0)


def embedding_grad(ids, dy, vocab, scale=1.0, base=None):
    ids = np.asarray(ids, dtype=np.int64)
    dy = np.asarray(dy, dtype=np.float64)
    inside = (ids >= 0) & (ids < vocab)
    out = np.zeros((vocab, dy.shape[1]))
    np.add.at(out, ids[inside], dy[inside] * scale)
    return out if base is None else out + np.asarray(base, dtype=np.float64)
