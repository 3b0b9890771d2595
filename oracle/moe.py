"""A mixture-of-experts layer from the exported form, in float64, with the error that its fixed-point
activations and float32 steps may cost.

p = softmax(router x), the top_k largest (equal ones by index), weights p (/ their sum);
y = sum_j w_j D ( act(G x) * (U x) ), each matrix R^T (s z): a product is s sum z . x~ with x~ = R x =
kappa H (sign * x).  Matrices come as 2z [rows, cols] and scale [rows] of each expert.

Bounds (u = 2^-24): x~ of a block of b columns is off by (log2 b + 2) u times the block's sum of |x| kappa, and by
at most 2^-23 max |x~| for the fixed point (2^-22 is allowed); a product adds u of itself; act * up 16 u of itself
(and of |g| |u|: 1 + tanh cancels for negative g); its error passes through down; weights and their sum 40 u, the sum over
k places k u of its terms.
"""

import numpy as np

from .core import core_points

U = 2.0 ** -24


def exported_two_z(core_idx, records, counts, shape, bound):
    """2z [experts, rows, cols] (int64) of an exported form; a slot without a point is 0."""
    experts, rows, cols = shape
    pts = core_points(bound)
    idx = np.asarray(core_idx).astype(np.int64).reshape(experts, rows * cols // 8)
    z = np.where((idx < len(pts))[..., None], pts[np.minimum(idx, len(pts) - 1)], 0)
    first = 0
    for e in range(experts):
        rec = records[first:first + int(counts[e])]
        for r in rec:
            if idx[e, r["group"]] == 0xFFFF:
                z[e, r["group"]] = r["two_z"]
        first += int(counts[e])
    return z.reshape(experts, rows, cols)


def _fwht(v, b):
    """Sylvester transform of every block of b of the last axis, float64."""
    shape, width = v.shape, 1
    while width < b:
        v = v.reshape(-1, b // (2 * width), 2, width)
        v = np.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], axis=2)
        width *= 2
    return v.reshape(shape)


def _rotate(x, signs, had):
    """x~ and the blocks' kappa sum |x|, of the last axis."""
    x = np.asarray(x, np.float64)
    if signs is None:
        return x, np.zeros_like(x)
    v = _fwht(x * signs, had) / np.sqrt(had)
    size = np.abs(x).reshape(x.shape[:-1] + (-1, had)).sum(axis=-1, keepdims=True) / np.sqrt(had)
    return v, np.broadcast_to(size, size.shape[:-1] + (had,)).reshape(x.shape)


def _input_error(x, signs, had):
    v, size = _rotate(x, signs, had)
    steps = np.log2(had) + 2 if signs is not None else 0
    return v, steps * U * size + 2.0 ** -22 * 1.001 * np.abs(v).max(axis=-1, keepdims=True)


def _product(two_z, scale, v, err):
    """Product and its bound of one expert's matrix with the vectors v [n, cols]."""
    s = np.where((scale > 0) & np.isfinite(scale), scale, 0.0).astype(np.float64) / 2
    y = v @ two_z.T.astype(np.float64) * s
    return y, err @ np.abs(two_z).T.astype(np.float64) * s + U * np.abs(y)


def moe_route(x, router, top_k, normalize):
    """Places and weights [tokens, top_k]; a NaN logit counts as -inf."""
    with np.errstate(invalid="ignore"):
        logits = np.asarray(x, np.float64) @ np.asarray(router, np.float64).T
    logits = np.where(np.isnan(logits), -np.inf, logits)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    w = np.take_along_axis(p, idx, axis=1)
    return idx, w / (w if normalize else p).sum(axis=1, keepdims=True)


def moe_layer(x, gate, up, down, idx, weight, signs_in=None, had_in=0, signs_down=None, had_down=0, act="silu"):
    """y [tokens, hidden] and its bound; gate, up, down are (2z [experts, rows, cols], scale [experts, rows])."""
    x = np.asarray(x, np.float64)
    experts = gate[0].shape[0]
    y, tol = np.zeros(x.shape), np.zeros(x.shape)
    size = np.zeros(x.shape)
    for e in range(experts):
        tok, place = np.nonzero(np.asarray(idx) == e)
        if not len(tok):
            continue
        v, err = _input_error(x[tok], signs_in, had_in)
        g, eg = _product(gate[0][e], gate[1][e], v, err)
        u, eu = _product(up[0][e], up[1][e], v, err)
        with np.errstate(all="ignore"):
            if act == "silu":
                a = g / (1 + np.exp(-g))
            else:
                a = 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
        h = a * u
        eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 16 * U * np.abs(g * u)     # |act'| <= 1.13
        v2, err2 = _input_error(h, signs_down, had_down)
        err2 = err2 + (_rotate(eh, np.ones(h.shape[1]), had_down)[1] if signs_down is not None else eh)
        err2 = err2 + 2.0 ** -22 * (err2.max(axis=-1, keepdims=True))
        d, ed = _product(down[0][e], down[1][e], v2, err2)
        w = np.asarray(weight, np.float64)[tok, place][:, None]
        np.add.at(y, tok, w * d)
        np.add.at(tol, tok, np.abs(w) * (ed + 40 * U * np.abs(d)))
        np.add.at(size, tok, np.abs(w * d))
    return y, tol + idx.shape[1] * U * size
