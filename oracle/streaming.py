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


# ------------------------------------------------------------------------------ paged cache
def ancestors(parents, n):
    """Node n and the nodes it continues, by the parents before it (anything else: the context)."""
    out = [n]
    while 0 <= parents[n] < n:
        n = int(parents[n])
        out.append(n)
    return out[::-1]


def paged_rows(pool, table_row, n):
    """Rows [n, Hkv, D] of a sequence's first n positions, and which of them have a page."""
    P, Hkv, page, D = pool.shape
    rows, there = np.zeros((n, Hkv, D)), np.zeros(n, dtype=bool)
    for x in range(n):
        e = int(table_row[x // page])
        if 0 <= e < P:
            rows[x], there[x] = pool[e, :, x % page], True
    return rows, there


def paged_decode(q, k_pages, v_pages, table, lens, parents=None, n_new=None, scale=1.0, window=0, sinks=0):
    """(o, lse) of new tokens q [B, H, N, D] at the end of paged sequences: node n sees the cached
    tokens and its ancestors, under a window those within it of its position, and the first `sinks`."""
    q, k_pages, v_pages = (_as_f64(x) for x in (q, k_pages, v_pages))
    B, H, N, D = q.shape
    P, Hkv, page, _ = k_pages.shape
    cap = table.shape[1] * page
    o, lse = np.zeros((B, H, N, D)), np.full((B, H, N), -np.inf)
    for b in range(B):
        L = min(max(int(lens[b]), 0), cap)
        n_b = N if n_new is None else min(max(int(n_new[b]), 0), N)
        k, there = paged_rows(k_pages, table[b], min(L + n_b, cap))
        v, _ = paged_rows(v_pages, table[b], min(L + n_b, cap))
        par = [n - 1 for n in range(N)] if parents is None else [int(x) for x in parents[b]]
        for n in range(n_b):
            chain = ancestors(par, n)
            at = L + len(chain) - 1
            seen = [(x, x) for x in range(L)] + [(L + c, L + i) for i, c in enumerate(chain)]
            rows = [r for r, x in seen if r < cap and there[r] and (window <= 0 or at - x < window or x < sinks)]
            if not rows:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                p, z = masked_softmax(scale * k[rows, g] @ q[b, h, n], np.ones(len(rows), dtype=bool))
                o[b, h, n], lse[b, h, n] = p @ v[rows, g], z
    return o, lse


def _take(need, refs):
    """Serves the slots' wishes in order (None: nothing asked, -1: refused): status and pages of each.  A slot
    that asks for no page needs none to be left."""
    free = [p for p, r in enumerate(refs) if r <= 0]
    status, got, base = [], [], 0
    for n in need:
        if n is None or n < 0:
            status.append(0 if n is None else -1)
            got.append([])
            continue
        ok = n == 0 or base + n <= len(free)
        status.append(1 if ok else -2)
        got.append(free[base:base + n] if ok else [])
        base += n
    return status, got


def pages_reserve(table, lens, refs, page, tokens):
    """New (table, refs) and the status of every slot."""
    table, refs = table.copy(), refs.copy()
    M = table.shape[1]
    held = [next((j for j in range(M) if row[j] < 0), M) for row in table]
    need = []
    for s, t in enumerate(tokens):
        n = int(lens[s]) + int(t)
        bad = lens[s] < 0 or n > M * page or (table[s, held[s]:] >= 0).any()
        need.append(None if t <= 0 else -1 if bad else max(0, -(-n // page) - held[s]))
    status, got = _take(need, refs)
    for s, pages in enumerate(got):
        table[s, held[s]:held[s] + len(pages)] = pages
        refs[pages] = 1
    return table, refs, status


def pages_fork(table, lens, refs, page, parents):
    """New (table, lens, refs), the status of every slot and the (old, new) pages to copy."""
    S, M = table.shape
    P = len(refs)
    need = []
    for s, src in enumerate(parents):
        if src < 0:
            need.append(None)
            continue
        ok = src < S and parents[src] < 0 and lens[s] == 0 and (table[s] < 0).all()
        ok = ok and 0 <= lens[src] <= M * page
        if ok:
            used = table[src, :-(-lens[src] // page)]
            ok = all(0 <= e < P and refs[e] > 0 for e in used)
        need.append(int(lens[src] % page > 0) if ok else -1)
    status, got = _take(need, refs)
    t, n, r, pairs = table.copy(), lens.copy(), refs.copy(), []
    for s, src in enumerate(parents):
        pair = (-1, -1)
        if status[s] == 1:
            full = lens[src] // page
            t[s, :full] = table[src, :full]
            for e in table[src, :full]:
                r[e] += 1
            if got[s]:
                pair = (int(table[src, full]), got[s][0])
                t[s, full] = got[s][0]
                r[got[s][0]] = 1
            n[s] = lens[src]
        pairs.append(pair)
    return t, n, r, status, pairs


def pages_free(table, lens, refs, drop):
    """New (table, lens, refs) without the dropped slots' pages."""
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    for s in np.nonzero(np.asarray(drop) > 0)[0]:
        for e in table[s]:
            if 0 <= e < len(refs):
                refs[e] = max(0, refs[e] - 1)
        table[s], lens[s] = -1, 0
    return table, lens, refs


def pages_compact(table, refs):
    """New (table, refs) with the pages in use in the lowest places, and the (from, to) moves."""
    P = len(refs)
    n = int((refs > 0).sum())
    late = [p for p in range(n, P) if refs[p] > 0]
    holes = [p for p in range(n) if refs[p] <= 0]
    to = list(range(P))
    r = refs.copy()
    r[n:] = 0
    for a, b in zip(late, holes):
        to[a], r[b] = b, refs[a]
    t = np.array([[to[e] if 0 <= e < P else -1 for e in row] for row in table], dtype=table.dtype)
    return t, r, list(zip(late, holes))
