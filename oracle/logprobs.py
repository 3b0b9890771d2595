"""Token log probabilities, entropy, alternatives and their gradient in float64.

y = scale * x; lse = log sum exp y; logprob = y_t - lse; entropy = -sum p log p;
alternatives by value, equal values by index (NaN first).  A negative token, or
one past the vocabulary, is ignored (logprob 0, no gradient).  A row of -inf
only: lse and log probabilities -inf, entropy 0, gradient 0.
"""

import numpy as np


def _rows(x, scale):
    y = np.asarray(x, dtype=np.float64) * float(scale)
    with np.errstate(all="ignore"):
        m = y.max(axis=1, keepdims=True)
        empty = np.isneginf(m[:, 0])
        e = np.exp(y - np.where(np.isneginf(m), 0.0, m))
        s = e.sum(axis=1, keepdims=True)
        lse = m + np.log(np.where(empty[:, None], 1.0, s))
        lse = np.where(empty[:, None], -np.inf, lse)
        p = np.where(empty[:, None], 0.0, e / s)
        lp = np.where(empty[:, None], -np.inf, y - lse)
    return lse[:, 0], p, lp, empty


def _entropy(p, lp):
    with np.errstate(all="ignore"):
        return -np.where(p == 0, 0.0, p * lp).sum(axis=1)


def _tokens(tokens, rows, vocab):
    t = np.asarray(tokens, dtype=np.int64).reshape(rows, -1)
    return t, (t >= 0) & (t < vocab)


def logprobs(x, scale=1.0, tokens=None, top_k=0):
    rows, vocab = x.shape
    lse, p, lp, _ = _rows(x, scale)
    out = {"lse": lse, "entropy": _entropy(p, lp)}
    if tokens is not None:
        t, live = _tokens(tokens, rows, vocab)
        out["logprob"] = np.where(live, np.take_along_axis(lp, np.where(live, t, 0), axis=1), 0.0)
    if top_k:
        v = np.where(np.isnan(x), np.inf, np.asarray(x, np.float64))
        order = np.lexsort((np.broadcast_to(np.arange(vocab), x.shape), -v, ~np.isnan(x)), axis=1)[:, :top_k]
        out["top_idx"] = order
        out["top_logprob"] = np.take_along_axis(lp, order, axis=1)
    return out


def logprobs_grad(x, scale, tokens, grad_logprob, grad_entropy=None):
    """d/dx of sum(grad_logprob * logprob) + sum(grad_entropy * entropy)."""
    rows, vocab = x.shape
    _, p, lp, empty = _rows(x, scale)
    d = np.zeros(x.shape)
    if tokens is not None:
        t, live = _tokens(tokens, rows, vocab)
        g = np.where(live, np.asarray(grad_logprob, np.float64).reshape(rows, -1), 0.0)
        d -= g.sum(axis=1, keepdims=True) * p
        np.add.at(d, (np.arange(rows)[:, None], np.where(live, t, 0)), g)
    if grad_entropy is not None:
        h = _entropy(p, lp)
        with np.errstate(all="ignore"):
            d -= np.asarray(grad_entropy, np.float64)[:, None] * np.where(p == 0, 0.0, p * (lp + h[:, None]))
    d[empty] = 0.0
    return d * float(scale)
