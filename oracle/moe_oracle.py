"""Float64 reference of the expert router and of a layer of experts."""
from __future__ import annotations

import numpy as np


def moe_route(logits, topk: int, renormalize: bool):
    """(ids, weights, offsets, order): by sorting (-logit, index) pairs."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    tokens, experts = l.shape
    ids = np.zeros((tokens, topk), dtype=np.int64)
    weights = np.zeros((tokens, topk))
    for t in range(tokens):
        order = sorted(range(experts), key=lambda e: (-l[t, e], e))
        ids[t] = order[:topk]
        top = l[t, order[0]]
        if top == -np.inf:
            continue
        p = np.array([1.0 if v == top else np.exp(v - top) for v in l[t]])
        chosen = p[ids[t]]
        weights[t] = chosen / (chosen.sum() if renormalize else p.sum())
    flat = ids.ravel()
    order = np.array(sorted(range(len(flat)), key=lambda i: (flat[i], i)), dtype=np.int64)
    offsets = np.array([int(np.sum(flat < e)) for e in range(experts + 1)], dtype=np.int64)
    return ids, weights, offsets, order


def moe_weight_bound(logits, ids, weights):
    """Bound on a weight's error: the difference to the largest logit rounds by half
    a unit (2^-24 of it, relative to the weight), the exponential, the sum of at
    most 16 lanes' (or of 1024 / 64 + 6) terms and the division by less than 8
    2^-23 together."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        gap = top - np.take_along_axis(l, ids, axis=1)
    gap = np.where(np.isfinite(gap), gap, 0.0)
    return (gap / 2 + 8) * 2.0 ** -23 * weights + 2.0 ** -126


def silu(a):
    return a / (1 + np.exp(-a))


def moe_layer(gate_up, down, X, ids, weights):
    """Y of the layer: gate_up (experts, 2 f, d), down (experts, d, f), float64."""
    return _layer(gate_up, down, X, ids, weights)[0]


def moe_layer_and_bound(gate_up, down, X, ids, weights, weight_err, up_units, down_units):
    """Y and a bound on the kernels' error before the rounding to Y's type.

    up_units, down_units: errors of the two products in units of 2^-23 of their
    terms' magnitudes.  silu's slope is below 1.1, so h moves by at most 1.1 dg
    (|u| + du) + |silu(g)| du; its own arithmetic (exponential, two divisions and a
    product) rounds by less than 8 2^-24.  Adding the experts' products (at most
    16), the waves' (8) and the splits' (16) sums rounds 40 times by 2^-24."""
    return _layer(gate_up, down, X, ids, weights, weight_err, up_units, down_units)


def _layer(gate_up, down, X, ids, weights, weight_err=None, up_units=0.0, down_units=0.0):
    X = np.asarray(X, dtype=np.float64)
    f = gate_up.shape[1] // 2
    Y = np.zeros((X.shape[0], down.shape[1]))
    bound = np.zeros_like(Y)
    unit = 2.0 ** -23
    for t in range(X.shape[0]):
        for j, e in enumerate(ids[t]):
            z, zm = gate_up[e] @ X[t], np.abs(gate_up[e]) @ np.abs(X[t])
            g, u = z[:f], z[f:]
            h = silu(g) * u
            v = down[e] @ h
            Y[t] += weights[t, j] * v
            if weight_err is None:
                continue
            dg, du = up_units * unit * zm[:f], up_units * unit * zm[f:]
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + 4 * unit * np.abs(h)
            a = np.abs(down[e])
            mags = a @ (np.abs(h) + dh)
            bound[t] += weights[t, j] * (a @ dh + (down_units + 20) * unit * mags) + weight_err[t, j] * mags
    return Y, bound + 2.0 ** -120
