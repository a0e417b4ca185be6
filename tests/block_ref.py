"""Plain references of the operators of include/moe_block.h in float64 (numpy),
and small seeded inputs.  Test infrastructure only; nothing here calls the
library."""

from __future__ import annotations

import numpy as np

# half a step of a type, relative to the value (round to nearest)
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
EPS32 = 2.0 ** -24


def norm(x, res, w, eps):
    """(s, y) of the residual norm."""
    s = x.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    rho = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s, s * rho * w.astype(np.float64)


def norm_backward(s, w, dy, dsum, eps):
    """(dx, dw, size of dx's terms, size of dw's terms)."""
    s, w, dy = (a.astype(np.float64) for a in (s, w, dy))
    H = s.shape[1]
    rho = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    g = dy * w
    gs = (g * s).sum(axis=1, keepdims=True)
    dx = rho * g - s * rho ** 3 * gs / H
    size = np.abs(rho * g) + np.abs(s) * rho ** 3 * np.abs(g * s).sum(axis=1, keepdims=True) / H
    if dsum is not None:
        dx = dx + dsum.astype(np.float64)
        size = size + np.abs(dsum.astype(np.float64))
    t = dy * s * rho
    return dx, t.sum(axis=0), size, np.abs(t).sum(axis=0)


def product(xq, xs, wq, ws):
    """Exact integer sums times the scales, float64."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T   # below 2^53: exact
    return acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]


def silu(g):
    """g / (1 + exp(-g)) without overflow."""
    return np.where(g >= 0, g, g * np.exp(np.minimum(g, 0.0))) / (1.0 + np.exp(-np.abs(g)))


def routing(rng, T, E, k, tile, gran, n_shared, idx=None):
    """Routing tables by their definition (float32 weights that sum to one)."""
    if idx is None:
        idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    w = rng.random((T, k)).astype(np.float32) + 0.05
    w /= w.sum(axis=1, keepdims=True)
    flat = idx.reshape(-1)
    order = np.argsort(flat, kind="stable")
    pos = np.empty_like(order)
    pos[order] = np.arange(T * k)
    counts = np.bincount(flat, minlength=E)
    blocks, row = [], 0
    for g, c in enumerate(list(counts) + [T] * n_shared):
        nb = -(-int(c) // tile)
        for b in range(nb):
            lo, hi = c * b // nb, c * (b + 1) // nb
            blocks.append([g, row + lo, hi - lo, -(-(-(-int(c) // nb)) // gran) * gran])
        row += c
    i32 = np.int32
    return dict(topk_idx=idx.astype(i32), topk_w=w, counts=counts.astype(i32),
                offsets=np.concatenate([[0], np.cumsum(counts)]).astype(i32),
                sorted_slot=order.astype(i32), slot_pos=pos.astype(i32).reshape(T, k),
                blocks=np.array(blocks, dtype=i32).reshape(-1, 4),
                n_blocks=np.array([len(blocks)], dtype=i32))


def row_tokens(r, T, k, n_shared):
    tok = r["sorted_slot"] // k
    return np.concatenate([tok, np.arange(T)]) if n_shared else tok


def row_groups(r, T, E, k, n_shared):
    g = np.repeat(np.arange(E), r["counts"])
    return np.concatenate([g, np.full(T, E)]) if n_shared else g


def combine(rows, w, pos, n_shared):
    """(y, size of its terms); w None: weights of one."""
    T, k = pos.shape
    rows = rows.astype(np.float64)
    ww = np.ones((T, k)) if w is None else w.astype(np.float64)
    terms = rows[pos] * ww[:, :, None]
    y, size = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    if n_shared:
        y, size = y + rows[T * k:], size + np.abs(rows[T * k:])
    return y, size


def combine_backward(dy, rows, w, pos, n_shared):
    """(drows, dw, size of dw's terms)."""
    T, k = pos.shape
    dy, rows = dy.astype(np.float64), rows.astype(np.float64)
    drows = np.empty_like(rows)
    drows[pos] = dy[:, None] * w.astype(np.float64)[:, :, None]
    if n_shared:
        drows[T * k:] = dy
    terms = rows[pos] * dy[:, None]
    return drows, terms.sum(axis=2), np.abs(terms).sum(axis=2)
