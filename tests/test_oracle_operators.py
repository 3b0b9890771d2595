"""Pins of the float64 oracles of the operators around the projection: closed
forms, and gradients against central differences."""

import numpy as np
import pytest

import oracle


def test_logprobs_closed_forms():
    r = oracle.logprobs(np.zeros((1, 8)), 1.0, np.array([[3, -1, 8]]), top_k=3)
    assert np.allclose(r["lse"], np.log(8)) and np.allclose(r["entropy"], np.log(8))
    assert np.allclose(r["logprob"], [[-np.log(8), 0.0, 0.0]])
    assert r["top_idx"].tolist() == [[0, 1, 2]]                       # equal values by index
    x = np.array([[1.0, -np.inf, 3.0, -np.inf], [-np.inf] * 4])
    r = oracle.logprobs(x, 2.0, np.array([[2], [1]]), top_k=4)
    assert np.allclose(r["lse"][0], 6 + np.log1p(np.exp(-4.0))) and r["lse"][1] == -np.inf
    assert r["entropy"][1] == 0.0 and r["logprob"][1, 0] == -np.inf
    assert r["top_idx"].tolist() == [[2, 0, 1, 3], [0, 1, 2, 3]]
    r = oracle.logprobs(np.array([[1.0, np.nan, 5.0]]), 1.0, None, top_k=3)
    assert r["top_idx"].tolist() == [[1, 2, 0]] and np.isnan(r["lse"][0])


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_logprobs_gradient_against_differences(scale):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 7)) * 2
    x[1, 4] = -np.inf
    tok = np.array([[2, 2], [0, -1], [6, 9]])
    g, gh = rng.normal(size=(3, 2)), rng.normal(size=3)

    def loss(v):
        r = oracle.logprobs(v, scale, tok)
        return (r["logprob"] * g).sum() + (r["entropy"] * gh).sum()

    d = oracle.logprobs_grad(x, scale, tok, g, gh)
    for i in range(3):
        for j in range(7):
            if np.isinf(x[i, j]):
                assert d[i, j] == 0.0
                continue
            h = 1e-5
            a, b = x.copy(), x.copy()
            a[i, j] += h
            b[i, j] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - d[i, j]) < 1e-8


def test_embed_gradient_against_differences():
    rng = np.random.default_rng(2)
    tab, tok, g = rng.normal(size=(5, 3)), np.array([4, 0, 4, -1, 7, 4]), rng.normal(size=(6, 3))
    out = oracle.embed(tab, tok, 1.5)
    assert np.array_equal(out[3], np.zeros(3)) and np.array_equal(out[4], np.zeros(3))
    d, mag = oracle.embed_grad(g, tok, 5, 1.5)
    assert (mag >= np.abs(d)).all() and not d[1].any()
    for v in range(5):
        for c in range(3):
            t = tab.copy()
            t[v, c] += 1.0                                            # linear: differences are exact
            assert abs(((oracle.embed(t, tok, 1.5) - out) * g).sum() - d[v, c]) < 1e-12


@pytest.mark.parametrize("shape", [(1, 6, 9), (2, 9, 6), (1, 1, 4)])
def test_orthogonalize_is_the_polynomial_of_the_singular_values(shape):
    g = np.random.default_rng(3).normal(size=shape)
    got = oracle.orthogonalize(g, 5)
    a, b, c = (float(np.float32(v)) for v in (3.4445, -4.7750, 2.0315))
    for i in range(shape[0]):
        u, s, vt = np.linalg.svd(g[i], full_matrices=False)
        s = s / np.sqrt((s * s).sum())
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        assert np.allclose(got[i], (u * s) @ vt, atol=1e-10)
    assert not oracle.orthogonalize(np.zeros((1, 3, 8))).any()
    w, m, o = oracle.orthogonal_step(g, g, g, 0.5, True, 0.1, 0.01, 2.0)
    assert np.allclose(m, 1.5 * g) and np.allclose(o, oracle.orthogonalize(1.75 * g))
    assert np.allclose(w, g * (1 - 0.001) - 0.2 * o)
