"""The distillation loss against a teacher's top logits, and its gradient, in float64.

y = scale * x, q = softmax(y); places (i_j, l_j), p_j = exp(l_j) where i_j names
a token (0 <= i_j < vocab), else the place is not used.  w = p ("none"), p / sum p
("renorm"), or p with w_r = max(0, 1 - sum p) for all tokens that no place names
("rest"; 0 where their q is 0 because all are named or -inf).
loss = sum w_j (log w_j - log q_{i_j}) + w_r (log w_r - log q_r).
A row without a used place: loss 0, gradient 0, whatever its logits.
"""

import numpy as np


def distill(x, scale, idx, lp, tail, grad_loss=None):
    """Per row: loss, log q at the places (0: not used), the places' weights, the rest's weight and log q,
    log q of all tokens, each one's share of the rest, and with ``grad_loss`` the gradient of the logits."""
    x, lp = np.asarray(x, np.float64), np.asarray(lp, np.float64)
    idx = np.asarray(idx, np.int64)
    rows, vocab = x.shape
    out = {"loss": np.zeros(rows), "logprob": np.zeros(idx.shape), "w": np.zeros(idx.shape),
           "w_rest": np.zeros(rows), "log_rest": np.full(rows, -np.inf), "log_q": np.zeros(x.shape),
           "share": np.zeros(x.shape)}
    grad = np.zeros(x.shape)
    for r in range(rows):
        live = (idx[r] >= 0) & (idx[r] < vocab)
        if not live.any():
            continue
        i, l = idx[r][live], lp[r][live]
        y = x[r] * float(scale)
        with np.errstate(all="ignore"):
            m = y.max()
            empty = np.isneginf(m)
            lse = m if empty else m + np.log(np.exp(y - m).sum())
            lq = np.full(vocab, -np.inf) if empty else y - lse
            p = np.exp(l)
            mass = p.sum()
            w, lw = (p, l) if tail != "renorm" else (p / mass if mass != 0 else p, l - np.log(mass))
            terms = np.where((w == 0) & ~np.isnan(lse), 0.0, w * (lw - lq[i]))
            named = np.zeros(vocab, bool)
            named[i] = True
            w_r, lq_r, share = 0.0, -np.inf, np.zeros(vocab)
            if not named.all() and not np.isneginf(y[~named]).all():
                top = y[~named].max()                        # apart from lse: it may be far above
                ls = np.log(np.exp(y[~named] - top).sum())
                lq_r = (top - m) + ls - (lse - m)
                share = np.where(named, 0.0, np.exp(y - top - ls))
                if tail == "rest":
                    w_r = np.maximum(0.0, 1.0 - mass)
            out["loss"][r] = terms.sum() + (w_r * (np.log(w_r) - lq_r) if w_r > 0 else 0.0)
            out["logprob"][r, live], out["w"][r, live] = lq[i], w
            out["w_rest"][r], out["log_rest"][r], out["log_q"][r], out["share"][r] = w_r, lq_r, lq, share
            if grad_loss is not None and not empty:
                total = w.sum() + w_r
                at = np.zeros(vocab)
                np.add.at(at, i, w)
                outside = share * (total * np.exp(lq_r) - w_r) if w_r > 0 else total * np.exp(lq)
                grad[r] = np.where(named, total * np.exp(lq) - at, outside) * float(scale) * float(grad_loss[r])
    if grad_loss is not None:
        out["grad"] = grad
    return out
