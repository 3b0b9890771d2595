"""Pins of the float64 oracles of the distillation loss, the adjustment of logits and the
mixture-of-experts layer: closed forms, gradients against central differences, dense
matrices; and the LDS that the layer's kernels take against what its host side allows them."""

import os
import re
import subprocess

import numpy as np
import pytest

import oracle
from bit_e8_lattice_amd import build


def test_distill_closed_forms():
    x = np.log(np.array([[0.5, 0.25, 0.125, 0.125]]))
    idx, p = np.array([[0, 2]]), np.array([[0.4, 0.2]])
    lp = np.log(p)
    r = oracle.distill(x, 1.0, idx, lp, "none")
    assert np.allclose(r["loss"], 0.4 * np.log(0.4 / 0.5) + 0.2 * np.log(0.2 / 0.125))
    assert np.allclose(r["logprob"], np.log([[0.5, 0.125]]))
    r = oracle.distill(x, 1.0, idx, lp, "renorm")
    assert np.allclose(r["loss"], 2 / 3 * np.log(2 / 3 / 0.5) + 1 / 3 * np.log(1 / 3 / 0.125))
    r = oracle.distill(x, 1.0, idx, lp, "rest")
    assert np.allclose(r["loss"], 0.4 * np.log(0.4 / 0.5) + 0.2 * np.log(0.2 / 0.125) + 0.4 * np.log(0.4 / 0.375))
    same = oracle.distill(x, 1.0, np.array([[0, 1]]), np.log([[0.5, 0.25]]), "rest", np.ones(1))
    assert np.allclose(same["loss"], 0) and np.allclose(same["grad"], 0)          # the student is the teacher
    empty = oracle.distill(x, 1.0, np.array([[-1, 9]]), lp, "rest", np.ones(1))
    assert empty["loss"][0] == 0 and not empty["grad"].any()


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_distill_of_non_finite_logits(tail, value):
    """NaN loss and gradient, whatever the places weigh; 0 where no place is used."""
    lp = np.full((1, 2), -np.inf)
    for at in (0, 1):
        x = np.zeros((1, 4))
        x[0, at] = value
        r = oracle.distill(x, 1.0, np.array([[0, 2]]), lp, tail, np.ones(1))
        assert np.isnan(r["loss"]).all() and np.isnan(r["grad"]).all() and np.isnan(r["logprob"]).all()
        r = oracle.distill(x, 1.0, np.array([[-1, -1]]), lp, tail, np.ones(1))
        assert not r["loss"].any() and not r["grad"].any()


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
def test_distill_gradient_against_differences(tail):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(3, 9)) * 2
    x[1, 4] = -np.inf
    idx = np.array([[2, 2, 5], [0, -1, 8], [6, 9, 1]])
    lp = np.log(rng.dirichlet(np.ones(4), size=3)[:, :3])
    g = rng.normal(size=3)
    d = oracle.distill(x, 0.8, idx, lp, tail, g)["grad"]
    for i in range(3):
        for j in range(9):
            if np.isinf(x[i, j]):
                assert d[i, j] == 0
                continue
            a, b = x.copy(), x.copy()
            a[i, j] += 1e-5
            b[i, j] -= 1e-5
            diff = (oracle.distill(a, 0.8, idx, lp, tail)["loss"] - oracle.distill(b, 0.8, idx, lp, tail)["loss"])[i] / 2e-5
            assert abs(diff * g[i] - d[i, j]) < 1e-8


def test_adjust_closed_forms():
    x = np.array([[1.0, -2.0, 3.0, -4.0, 5.0]])
    a = dict(history=np.array([[0, 1, 1, 4, -1, 7]]), prompt_len=np.array([2]), repetition=np.array([2.0]),
             frequency=np.array([0.5]), presence=np.array([0.25]))
    # made: 1 once, 4 once; in the history: 0, 1, 4
    assert np.allclose(oracle.adjust_logits(x, **a), [[0.5, -4.75, 3.0, -4.0, 1.75]])
    a["history_len"] = np.array([3])
    assert np.allclose(oracle.adjust_logits(x, **a), [[0.5, -4.75, 3.0, -4.0, 5.0]])
    r = oracle.adjust_logits(x, bias_idx=np.array([[3, 3, -1]]), bias=np.array([[1.0, 2.0, 9.0]]),
                             mask=np.array([[0b01011]], np.int32))
    assert np.array_equal(r, [[1.0, -2.0, -np.inf, -1.0, -np.inf]])


def test_moe_against_dense_matrices():
    rng = np.random.default_rng(3)
    experts, hidden, inter, tokens = 3, 16, 8, 4
    two_z = [rng.integers(-4, 5, size=s) for s in ((experts, inter, hidden),) * 2 + ((experts, hidden, inter),)]
    scale = [rng.uniform(0.5, 1.5, size=t.shape[:2]) for t in two_z]
    sign = np.where(rng.random(hidden) < 0.5, -1.0, 1.0), np.where(rng.random(inter) < 0.5, -1.0, 1.0)
    had = np.ones((1, 1))
    while had.shape[0] < 8:
        had = np.block([[had, had], [had, -had]])
    rotation = [np.kron(np.eye(n // 8), had) / np.sqrt(8) * s for n, s in ((hidden, sign[0]), (inter, sign[1]))]
    w = [(t * (s[..., None] / 2)) @ rotation[0 if i < 2 else 1] for i, (t, s) in enumerate(zip(two_z, scale))]
    x, router = rng.normal(size=(tokens, hidden)), rng.normal(size=(experts, hidden))
    idx, weight = oracle.moe_route(x, router, 2, True)
    y, tol = oracle.moe_layer(x, *zip(two_z, scale), idx, weight, sign[0], 8, sign[1], 8)
    for t in range(tokens):
        p = np.exp(x[t] @ router.T)
        want = np.zeros(hidden)
        for e in np.argsort(-p)[:2]:
            g, u = w[0][e] @ x[t], w[1][e] @ x[t]
            want += p[e] / np.sort(p)[-2:].sum() * (w[2][e] @ (g / (1 + np.exp(-g)) * u))
        assert np.allclose(y[t], want) and (tol[t] > 0).all() and (tol[t] < 1e-3 * np.abs(y).max()).all()


def test_moe_route_counts_nan_as_minus_infinity():
    router = np.array([[np.nan, 1.0], [2.0, 0.0], [-np.inf, 0.0], [1.0, 0.0]])
    for normalize in (True, False):
        idx, w = oracle.moe_route(np.array([[1.0, 1.0]]), router, 4, normalize)
        assert idx.tolist() == [[1, 3, 0, 2]]
        assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1)), 0, 0]])


def test_lds_of_the_layers_kernels(tmp_path):
    """More LDS than a CU has, the kernel's own and what its launch asks for, ends the queue with an error that no
    call returns: the host side counts with kMoeOwn for the former, so the kernels may not have more."""
    source = "e8q_moe.hip"
    text = open(os.path.join(build.CSRC, source)).read()
    own, small = (eval(re.search(rf"constexpr uint32_t {n} = ([0-9 *]+);", text).group(1)) for n in ("kMoeOwn", "kMoeSmall"))
    out = tmp_path / "device.s"
    res = subprocess.run([build.hipcc()] + build.FLAGS + build.SOURCE_FLAGS.get(source, []) +
                         ["-I", build.INCLUDE, "-I", build.CSRC, "-S", "--cuda-device-only",
                          os.path.join(build.CSRC, source), "-o", str(out)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    seen = 0
    for lds, name in re.findall(r"\.group_segment_fixed_size: (\d+).*?\.name: +(\S+)", out.read_text(), re.S):
        m = re.search(r"moe_(product|direct)_kernelI(?:Lb[01]E)?Li([012])E", name)
        if m:
            seen += 1
            assert int(lds) <= own + (small * 4 if m.group(2) == "1" else 0), name
    assert seen == 15
