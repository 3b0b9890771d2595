"""Rows whose logits lie far from zero: masked everywhere by the type's lowest
value, or with a common offset.  Only the differences from the row's maximum
count, so outputs and gradients are held to bounds in which the offset does not
occur.

Bounds.  With d = scale (x - max), an exponent is off by 2^-22 |d|, v_exp_f32
and v_log_f32 add a few units in the last place, and a thread adds at most
V / 256 terms one after another: ln sum and entropy are within
u (16 + 4 log2 V + V / 256), u = 2^-23, times (4 + H + log V) for the entropy
(its terms weigh up to |log p|); a log probability adds u (|d| + |its value|).
p is within the same of itself, plus u |2 d|, plus 2^-20: e8q_token_logprobs_backward
takes the rounded lse of a row while |lse| <= 32.  lse itself is one rounding of
its own size."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rel(x, scale):
    """d, the logits' part of every bound, and the sums' relative bound."""
    vocab = x.shape[1]
    m = x.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        d = np.where(np.isneginf(m), 0.0, (x - m) * scale)
    return d, U * (16 + 4 * np.log2(max(vocab, 2)) + vocab / 256)


def _reference(x, scale, tok, g, gh):
    """Outputs and gradient in float64, from the differences d; and the gradient's bound."""
    rows, vocab = x.shape
    d, rel = _rel(x, scale)
    s = np.exp(d).sum(axis=1, keepdims=True)
    lp = d - np.log(s)
    p = np.exp(lp)
    ent = -np.where(p > 0, p * lp, 0.0).sum(axis=1)
    live = (tok >= 0) & (tok < vocab)
    take = np.where(live, tok, 0)
    lpt = np.where(live, np.take_along_axis(lp, take, axis=1), 0.0)
    gg = np.where(live, g, 0.0)
    mag = np.abs(gg).sum(axis=1, keepdims=True) * p
    dx = -gg.sum(axis=1, keepdims=True) * p
    np.add.at(dx, (np.arange(rows)[:, None], take), gg)
    at = np.zeros((rows, vocab))
    np.add.at(at, (np.arange(rows)[:, None], take), np.abs(gg))
    if gh is not None:
        dx -= gh[:, None] * np.where(p > 0, p * (lp + ent[:, None]), 0.0)
        mag += np.abs(gh)[:, None] * p * (np.abs(np.where(p > 0, lp, 0.0)) + ent[:, None] + 4 + np.log(vocab))
    with np.errstate(all="ignore"):
        off = np.where(p > 0, 8 * rel + 2 * U * np.abs(d) + 2.0 ** -20, 0.0)
    return {"logprob": lpt, "entropy": ent, "ln_s": np.log(s)[:, 0], "dx": dx * scale, "p": p,
            "lim": scale * (mag * off + 2.0 ** -22 * at), "rel": rel, "d": np.where(live, np.take_along_axis(d, take, axis=1), 0.0)}


def _rows(kind, rows, vocab, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, vocab), generator=g) * 3
    if kind == "lowest":
        x[:] = torch.finfo(dtype).min
    elif kind == "lowest but few":
        x[:, 3:] = torch.finfo(dtype).min
    else:
        x = x + float(kind)
    return x.to(dtype).to(device())


def _check(x, scale, seed, in_place):
    """Both forms of the gradient, and the outputs, of one batch."""
    d, (rows, vocab) = x.device, x.shape
    rg = torch.Generator().manual_seed(seed)
    tok = torch.randint(-1, vocab, (rows, 2), generator=rg).to(d)
    tok[:, 0] = torch.arange(rows, device=d) % vocab
    g, gh = torch.randn((rows, 2), generator=rg).to(d), torch.randn((rows,), generator=rg).to(d)
    sc = float(np.float32(scale))
    want = _reference(_f64(x), sc, tok.cpu().numpy(), _f64(g), _f64(gh))
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab), dtype=torch.uint8, device=d)
    out = {n: torch.empty((rows, 2) if n == "logprob" else (rows,), device=d) for n in ("logprob", "lse", "entropy")}
    e8q.e8q_token_logprobs(x, ws, st, tokens=tok, scale=scale, logprob_out=out["logprob"], lse_out=out["lse"],
                           entropy_out=out["entropy"])
    last = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -22
    lim = want["lim"] + last * np.abs(want["dx"]) + 1e-37

    def outputs(o, what):
        tol = want["rel"]
        assert (np.abs(_f64(o["logprob"]) - want["logprob"]) <= tol + U * (np.abs(want["d"]) + np.abs(want["logprob"]))).all(), what
        assert (np.abs(_f64(o["entropy"]) - want["entropy"]) <= tol * (4 + want["entropy"] + np.log(vocab))).all(), what
        lse = _f64(x).max(axis=1) * sc + want["ln_s"]
        fits = np.abs(lse) < np.finfo(np.float32).max
        assert (np.abs(_f64(o["lse"]) - lse)[fits] <= (tol + 2 * U * np.abs(lse))[fits]).all(), what

    def gradient(t, what):
        off = np.abs(_f64(t) - want["dx"])
        assert (off <= lim).all(), (what, float((off / lim).max()), float(off.max()))

    outputs(out, "outputs")
    dx = x.clone() if in_place else torch.empty_like(x)
    e8q.e8q_token_logprobs_backward(dx if in_place else x, out["lse"], dx, st, tokens=tok, grad_logprob=g, scale=scale,
                                    entropy=out["entropy"], grad_entropy=gh)
    gradient(dx, "backward")
    dy = x.clone() if in_place else torch.empty_like(x)
    one = {n: torch.empty_like(v) for n, v in out.items()}
    e8q.e8q_token_logprobs_grad(dy if in_place else x, tok, g, dy, ws, st, grad_entropy=gh, scale=scale,
                                logprob_out=one["logprob"], lse_out=one["lse"], entropy_out=one["entropy"])
    gradient(dy, "one call")
    outputs(one, "outputs of the one call")
    assert int(st.item()) == 0
    return out, dx, dy


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 700), (2, 9000), (1, 40001), (1100, 515)])
@pytest.mark.parametrize("kind", ["lowest", "lowest but few", "1e4", "-1e4", "1e6", "60"])
def test_offsets(kind, rows, vocab, dtype, in_place):
    _check(_rows(kind, rows, vocab, dtype, rows + vocab), 1.0, 3, in_place)


@pytest.mark.parametrize("scale", [0.7, 1.25])
def test_offsets_with_a_scale(scale):
    for kind in ("1e4", "-1e6"):
        _check(_rows(kind, 3, 5000, torch.float32, 4), scale, 5, False)


@pytest.mark.parametrize("rows", [2, 1100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_row_of_lowest_values_is_uniform(rows, dtype):
    """logprob = -ln V, entropy = ln V, gradient g ([i = t] - 1 / V) and no gradient of the entropy."""
    d, vocab = device(), 4100
    x = torch.full((rows, vocab), torch.finfo(dtype).min, dtype=dtype, device=d)
    tok = torch.full((rows, 1), 7, device=d)
    one, st = torch.ones((rows, 1), device=d), torch.zeros(1, dtype=torch.int32, device=d)
    lp, h, lse = torch.empty((rows, 1), device=d), torch.empty(rows, device=d), torch.empty(rows, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs(x, ws, st, tokens=tok, logprob_out=lp, entropy_out=h, lse_out=lse)
    ln_v = np.log(vocab)
    assert (np.abs(_f64(lp) + ln_v) <= 8 * U * ln_v).all() and (np.abs(_f64(h) - ln_v) <= 8 * U * ln_v).all()
    two, both = torch.empty_like(x), torch.empty_like(x)
    e8q.e8q_token_logprobs_backward(x, lse, two, st, tokens=tok, grad_logprob=one, entropy=h, grad_entropy=100 * one[:, 0])
    e8q.e8q_token_logprobs_grad(x, tok, one, both, ws, st, grad_entropy=100 * one[:, 0])
    last = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    want = np.full(vocab, -1.0 / vocab)
    want[7] += 1.0
    for got in (two, both):
        # the entropy's gradient is 0, but for rounding of log p + H: 100 / V * 16 u ln V
        assert (np.abs(_f64(got) - want) <= last * np.abs(want) + 100 / vocab * 16 * U * ln_v).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 40001), (5, 9000), (301, 20011), (1100, 515)])
def test_in_place_gives_the_same_bits(rows, vocab, dtype):
    """Rows of moderate and of large lse in one call: the same gradient into another buffer and in place."""
    d = device()
    x = _rows("0", rows, vocab, dtype, 9)
    x[::2] += 1000
    x[rows - 1] = torch.finfo(dtype).min
    if rows > 4:
        x[3] = -float("inf")
    tok = (torch.arange(rows * 3, device=d) * 997 % vocab).view(rows, 3)
    g, gh = torch.randn((rows, 3), device=d), torch.randn(rows, device=d)
    st, lse, h = torch.zeros(1, dtype=torch.int32, device=d), torch.empty(rows, device=d), torch.empty(rows, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs(x, ws, st, lse_out=lse, entropy_out=h)
    other, own = torch.empty_like(x), x.clone()
    e8q.e8q_token_logprobs_backward(x, lse, other, st, tokens=tok, grad_logprob=g, entropy=h, grad_entropy=gh)
    for _ in range(3):
        own.copy_(x)
        e8q.e8q_token_logprobs_backward(own, lse, own, st, tokens=tok, grad_logprob=g, entropy=h, grad_entropy=gh)
        assert torch.equal(own, other)
    assert int(st.item()) == 0 and bool(torch.isfinite(other).all())
