"""Plain fp64 definitions of the streaming operators: sliding-window attention with sinks.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Everything is written out from the
definition with explicit masks, in numpy doubles.
"""
from __future__ import annotations

import numpy as np

from . import _as_f64


def sink_mask(T, window, sinks, doc_start=None):
    """[T, T] bool, True = visible: key j in query i's document, not after it, and within the window
    or among the document's first `sinks` tokens.  doc_start: T ints (None: one document)."""
    a = np.zeros(T, dtype=np.int64) if doc_start is None else np.asarray(doc_start, dtype=np.int64)
    i, j = np.arange(T)[:, None], np.arange(T)[None, :]
    near = (i - j < window) if window > 0 else np.ones((T, T), dtype=bool)
    return (j <= i) & (j >= a[:, None]) & (near | (j - a[:, None] < sinks))


def masked_softmax(x, vis):
    """Row softmax of scores x over the visible keys, and the natural-log row sum.  A row that sees
    nothing has p = 0 and lse = -inf."""
    x = np.where(vis, x, -np.inf)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - np.where(np.isinf(m), 0.0, m))
    z = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(np.isinf(m), 0.0, m) + np.log(z)
    return p / np.where(z > 0, z, 1.0), lse[..., 0]


def attn_sinks(q, k, v, scale, windows, sinks, doc_start=None, dO=None):
    """(o, lse) of [B, H, T, D] inputs, and (dq, dk, dv) of sum(o * dO) if dO is given.
    windows: one int, or one per head; doc_start: [B, T] or None."""
    q, k, v = (_as_f64(x) for x in (q, k, v))
    B, H, T, D = q.shape
    ws = [windows] * H if isinstance(windows, int) else list(windows)
    o, lse = np.empty_like(q), np.empty((B, H, T))
    g = [np.empty_like(q) for _ in range(3)] if dO is not None else None
    do = _as_f64(dO) if dO is not None else None
    for b in range(B):
        for h in range(H):
            vis = sink_mask(T, ws[h], sinks, None if doc_start is None else doc_start[b])
            p, lse[b, h] = masked_softmax(scale * q[b, h] @ k[b, h].T, vis)
            o[b, h] = p @ v[b, h]
            if g is not None:
                dp = do[b, h] @ v[b, h].T
                ds = p * (dp - (p * dp).sum(-1, keepdims=True))
                g[0][b, h] = scale * ds @ k[b, h]
                g[1][b, h] = scale * ds.T @ q[b, h]
                g[2][b, h] = p.T @ do[b, h]
    return (o, lse) if g is None else (o, lse, *g)
