"""Embedding lookup with scaling and its gradient in float64."""

import numpy as np


def embed(table, tokens, scale=1.0):
    t = np.asarray(tokens, np.int64).reshape(-1)
    live = (t >= 0) & (t < table.shape[0])
    rows = np.asarray(table, np.float64)[np.where(live, t, 0)] * float(scale)
    return np.where(live[:, None], rows, 0.0)


def embed_grad(grad_out, tokens, vocab, scale=1.0):
    """The table's gradient, and the sums of absolute values (for error bounds)."""
    t = np.asarray(tokens, np.int64).reshape(-1)
    g = np.asarray(grad_out, np.float64).reshape(t.size, -1) * float(scale)
    live = (t >= 0) & (t < vocab)
    out, mag = np.zeros((vocab, g.shape[1])), np.zeros((vocab, g.shape[1]))
    np.add.at(out, t[live], g[live])
    np.add.at(mag, t[live], np.abs(g[live]))
    return out, mag
