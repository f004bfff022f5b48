"""Tokens sorted by expert and back with the gradient, the expert layer over
sorted tokens and low-rank adapters, in float64 numpy.  Test infrastructure only.

These are definitions of this project, not of the pages; the expert layer is that
of product.py, expert by expert.
"""
from __future__ import annotations

import numpy as np

from .product import silu


def moe_sort(ids, experts):
    """(order, place, offsets): choices token * top_k + s by (expert, choice)."""
    flat = np.asarray(ids).reshape(-1)
    rows = [c for e in range(experts) for c in np.flatnonzero(flat == e)]
    order = np.full(flat.size, -1, dtype=np.int32)
    place = np.full(flat.size, -1, dtype=np.int32)
    order[:len(rows)] = rows
    place[rows] = np.arange(len(rows))
    counts = [int((flat == e).sum()) for e in range(experts)]
    return order, place.reshape(np.shape(ids)), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def moe_dispatch(x, place, xs):
    """xs with xs[place[t, s]] = x[t]."""
    xs = xs.copy()
    for s in range(place.shape[1]):
        t = np.flatnonzero(place[:, s] >= 0)
        xs[place[t, s]] = x[t]
    return xs


def moe_combine(ys, place, weights=None):
    """(y, sum of magnitudes); y[t] = sum of weights[t, s] ys[place[t, s]]."""
    y = np.zeros((place.shape[0], ys.shape[1]))
    mag = np.zeros_like(y)
    for s in range(place.shape[1]):
        t = np.flatnonzero(place[:, s] >= 0)
        v = ys[place[t, s]] * (1.0 if weights is None else weights[t, s, None])
        y[t] += v
        mag[t] += np.abs(v)
    return y, mag


def moe_combine_grad(dy, ys, place, weights):
    """(dys, dweights, magnitudes of dweights' sums); rows without a choice are NaN in dys."""
    dys = np.full((place.size, dy.shape[1]), np.nan)
    dw, mag = np.zeros(place.shape), np.zeros(place.shape)
    for s in range(place.shape[1]):
        t = np.flatnonzero(place[:, s] >= 0)
        dys[place[t, s]] = weights[t, s, None] * dy[t]
        v = dy[t] * ys[place[t, s]]
        dw[t, s] = v.sum(1)
        mag[t, s] = np.abs(v).sum(1)
    return dys, dw, mag


def moe_forward_sorted(x, ids, weights, w13, w2, eps_sum, eps_h, eps_row):
    """(y, bound): product.moe_forward expert by expert, and how far off y may be
    before its own rounding where a sum of n products may be off by n eps_sum of
    the sum of their magnitudes, silu * up by eps_h of its value and an expert's
    row by eps_row of its own (and 2^-28 of that of the row's largest value).

    silu' lies in [-0.1, 1.1]: an error d of gate moves silu by at most 1.1 d."""
    y, off = np.zeros_like(x), np.zeros_like(x)
    hidden, inter = x.shape[1], w2.shape[2]
    for e in range(w13.shape[0]):
        t, s = np.nonzero(ids == e)
        if not t.size:
            continue
        xe, w = x[t], weights[t, s, None]
        gate, up = xe @ w13[e, 0].T, xe @ w13[e, 1].T
        d = (hidden + 3) * eps_sum
        dg, du = d * (np.abs(xe) @ np.abs(w13[e, 0]).T), d * (np.abs(xe) @ np.abs(w13[e, 1]).T)
        h = silu(gate) * up
        dh = (1.1 * dg * (np.abs(up) + du) + np.abs(silu(gate)) * du)
        dh += eps_h * (np.abs(h) + dh)
        row = h @ w2[e].T
        np.add.at(y, t, w * row)
        mag = (np.abs(h) + dh) @ np.abs(w2[e]).T
        d = dh @ np.abs(w2[e]).T + (inter + ids.shape[1] + 3) * eps_sum * mag
        d += eps_row * (np.abs(row) + d + 2.0 ** -28 * (np.abs(row) + d).max(1, keepdims=True))
        np.add.at(off, t, np.abs(w) * d)
    return y, off


def matmul_lora(x, w, ids, a, b, scale, eps_sum):
    """(y, bound before y's own rounding): x w^T + scale_a (x A_a^T) B_a^T."""
    k, rank = x.shape[1], a.shape[1]
    y = x @ w.T
    off = (k + 3) * eps_sum * (np.abs(x) @ np.abs(w).T)
    for j in range(a.shape[0]):
        t = np.flatnonzero(ids == j)
        u, mu = x[t] @ a[j].T, np.abs(x[t]) @ np.abs(a[j]).T
        y[t] += scale[j] * (u @ b[j].T)
        off[t] += abs(scale[j]) * (((k + 3) * eps_sum * mu) @ np.abs(b[j]).T
                                   + (3 * rank + 6) * eps_sum * (mu @ np.abs(b[j]).T))
    return y, off
