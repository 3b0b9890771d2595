"""Newton-Schulz orthogonalization and the latents' step along it, in float64."""

import numpy as np


def orthogonalize(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315)):
    """X = G / |G|_F, then ``steps`` times X <- a X + (b A + c A^2) X, A = X X^T
    (on the smaller side), per matrix of ``g`` [batch, rows, cols]."""
    a, b, c = (float(np.float32(v)) for v in coeffs)
    out = np.empty(g.shape)
    for i, m in enumerate(np.asarray(g, np.float64)):
        with np.errstate(all="ignore"):
            norm = np.sqrt((m * m).sum())
            if not np.isfinite(norm):
                out[i] = np.nan
                continue
        x = m / norm if norm > 0 else m * 0.0
        tall = x.shape[0] > x.shape[1]
        x = x.T if tall else x
        for _ in range(steps):
            s = x @ x.T
            x = a * x + (b * s + c * (s @ s)) @ x
        out[i] = x.T if tall else x
    return out


def orthogonal_step(w, grad, momentum, mu, nesterov, lr, decay, gamma, steps=5, coeffs=(3.4445, -4.7750, 2.0315)):
    g, m = np.asarray(grad, np.float64), np.asarray(momentum, np.float64)
    m1 = mu * m + g
    u = g + mu * m1 if nesterov else m1
    o = orthogonalize(u, steps, coeffs)
    return np.asarray(w, np.float64) * (1.0 - lr * decay) - lr * gamma * o, m1, o
