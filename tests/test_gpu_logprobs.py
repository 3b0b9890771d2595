"""e8q_token_logprobs, its gradient, and both in one call, against float64.

Bounds.  Every exponent is a difference of float32 logits times a constant
(relative error 2^-22 of the exponent d, so at most 2^-22 |d| of its term,
which weighs p |log2 p| <= log2 V in the sum), v_exp_f32 and v_log_f32 add a
few units in the last place, and a thread adds at most V / 256 terms one after
another: |lse error| <= u (16 + 4 log2 V + V / 256 + |lse| + |m|), u = 2^-23.
The entropy weighs the same errors with up to |log p|: (4 + H + log V) times
as much.  A gradient is p (G + gH (log p + H)): the relative error of p times
that, and its last rounding."""

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


def _logits(rows, vocab, dtype, seed, pad=0, banned=False, ties=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, vocab + pad), generator=g) * 3
    if ties:
        x = torch.round(x)
    if banned:
        x[:, vocab // 3: vocab // 3 + vocab // 5] = -float("inf")
    return x.to(dtype).to(device())[:, :vocab]


def _bound(ref, x, scale):
    vocab = x.shape[1]
    m = np.where(np.isneginf(x), -np.inf, np.abs(x) * scale)
    m = np.where(np.isfinite(m), m, 0.0).max(axis=1)
    lse = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0.0)
    return U * (16 + 4 * np.log2(max(vocab, 2)) + vocab / 256 + lse + m)


def _close(got, want, tol, what):
    with np.errstate(all="ignore"):                     # a value past float32's range is an infinity there
        want = np.where(np.isinf(np.asarray(want).astype(np.float32)), np.sign(want) * np.inf, want)
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what
    off = np.abs(got[fin] - want[fin])
    assert (off <= np.broadcast_to(tol, want.shape)[fin]).all(), (what, off.max())


def _forward(x, tok, scale, k, stream=None):
    d, (rows, vocab) = x.device, x.shape
    n = 0 if tok is None else (tok.shape[1] if tok.dim() == 2 else 1)
    o = {"logprob": torch.full((rows, n), 9.0, device=d) if n else None,
         "lse": torch.full((rows,), 9.0, device=d), "entropy": torch.full((rows,), 9.0, device=d),
         "top_idx": torch.full((rows, k), -7, dtype=torch.int32, device=d) if k else None,
         "top_logprob": torch.full((rows, k), 9.0, device=d) if k else None}
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab, k), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs(x, ws, st, tokens=tok, scale=scale, logprob_out=o["logprob"], lse_out=o["lse"],
                           entropy_out=o["entropy"], top_idx_out=o["top_idx"], top_logprob_out=o["top_logprob"],
                           stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def _check_forward(x, tok, scale, k, status=0):
    o, st = _forward(x, tok, scale, k)
    xn = _f64(x)
    sc = float(np.float32(scale))
    ref = oracle.logprobs(xn, sc, None if tok is None else tok.cpu().numpy(), k)
    tol = _bound(ref, xn, sc)
    assert st == status
    _close(_f64(o["lse"]), ref["lse"], tol, "lse")
    _close(_f64(o["entropy"]), ref["entropy"], tol * (4 + ref["entropy"] + np.log(x.shape[1])), "entropy")
    if tok is not None:
        lim = tol[:, None] + U * np.where(np.isfinite(ref["logprob"]), np.abs(ref["logprob"]), 0)
        _close(_f64(o["logprob"]).reshape(ref["logprob"].shape), ref["logprob"], lim, "logprob")
    if k:
        assert np.array_equal(o["top_idx"].cpu().numpy(), ref["top_idx"])
        lim = tol[:, None] + U * np.where(np.isfinite(ref["top_logprob"]), np.abs(ref["top_logprob"]), 0)
        _close(_f64(o["top_logprob"]), ref["top_logprob"], lim, "top_logprob")
    return o, ref


CASES = [(1, 1, 0, 1), (1, 2, 0, 2), (3, 7, 5, 7), (2, 63, 0, 1), (5, 64, 3, 64), (4, 65, 0, 8), (2, 255, 0, 50),
         (3, 2049, 1, 20), (2, 4097, 0, 64), (1, 32003, 13, 5), (1, 131072, 0, 8), (9, 50001, 0, 33),
         (1100, 515, 0, 3), (2, 8192, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,pad,k", CASES)
def test_forward(rows, vocab, pad, k, dtype):
    x = _logits(rows, vocab, dtype, rows + vocab, pad)
    g = torch.Generator().manual_seed(5)
    tok = torch.randint(-1, vocab, (rows, 3), generator=g).to(device())
    _check_forward(x, tok, 1.0, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(2, 1000), (1, 40000), (3, 131), (1030, 300)])
def test_ties_masks_and_order(rows, vocab, dtype):
    d = device()
    x = _logits(rows, vocab, dtype, 3, banned=True, ties=True)                 # many equal logits
    _check_forward(x, torch.zeros((rows,), dtype=torch.int32, device=d), 0.7, 50)
    same = torch.full((rows, vocab), 2.5, dtype=dtype, device=d)               # one value
    _check_forward(same, None, 1.0, 64)
    up = (torch.arange(vocab, device=d, dtype=torch.float32) / 512).to(dtype).expand(rows, vocab).contiguous()
    _check_forward(up, None, 1.0, 17)                                          # every element a candidate
    _check_forward(up.flip(1).contiguous(), None, 1.0, 17)
    few = torch.full((rows, vocab), -float("inf"), dtype=dtype, device=d)      # fewer live logits than k
    few[:, vocab // 2] = 1.0
    few[:, vocab - 1] = 2.0
    _check_forward(few, torch.full((rows, 1), vocab - 1, device=d), 1.0, 5)
    low = torch.full((rows, vocab), torch.finfo(dtype).min, dtype=dtype, device=d)
    _check_forward(low, None, 1.0, 4)                                          # the type's lowest value everywhere
    low[:, 5] = -3.0
    _check_forward(low, torch.full((rows, 2), 5, device=d), 1.25, 4)
    zero = torch.zeros((rows, vocab), dtype=dtype, device=d)
    zero[:, ::2] = -0.0                                                        # equal to +0
    _check_forward(zero, None, 1.0, 9)


@pytest.mark.parametrize("vocab", [9, 5000, 131072])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_live_logit_and_nonfinite_rows(vocab, dtype):
    d = device()
    x = _logits(6, vocab, dtype, 8)
    x[1] = -float("inf")
    x[3, vocab // 2] = float("nan")
    x[4, 1] = float("inf")
    x[5, 2] = -float("nan")
    tok = torch.tensor([2, 2, 0, 1, 0, -1], device=d)
    o, ref = _check_forward(x, tok, 1.0, 6, status=e8q.STATUS_BITS["NONFINITE"])
    assert ref["lse"][1] == -np.inf and ref["entropy"][1] == 0.0 and np.isnan(ref["lse"][3:]).all()
    gl = torch.ones((6, 1), device=d)
    dx = torch.full_like(x, 9.0)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    e8q.e8q_token_logprobs_backward(x, o["lse"], dx, st, tokens=tok, grad_logprob=gl, entropy=o["entropy"],
                                    grad_entropy=torch.ones(6, device=d))
    dy = torch.full_like(x, 9.0)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(6, vocab), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs_grad(x, tok, gl, dy, ws, st, grad_entropy=torch.ones(6, device=d))
    torch.cuda.synchronize()
    for t in (dx, dy):
        assert not _f64(t)[1].any()                       # nothing left by the mask: gradient 0
        assert np.isnan(_f64(t)[3]).all() and np.isnan(_f64(t)[4]).all()
        assert np.isfinite(_f64(t)[:3]).all()


def test_ignored_and_out_of_range_tokens():
    d = device()
    x = _logits(4, 100, torch.float32, 4)
    tok = torch.tensor([[-100, 3], [100, 2 ** 40], [5, 5], [-1, -1]], device=d)
    o, _ = _check_forward(x, tok, 1.0, 0, status=e8q.STATUS_BITS["BAD_INDEX"])
    assert not _f64(o["logprob"])[[0, 1, 1, 3, 3], [0, 0, 1, 0, 1]].any()


def _grad_bound(xn, scale, tok, g, gh, ref, dtype):
    rows, vocab = xn.shape
    tol = _bound(ref, xn, scale)
    with np.errstate(all="ignore"):
        lp = xn * scale - ref["lse"][:, None]
        p = np.exp(lp)
        mag = np.zeros(xn.shape)
        if tok is not None:
            live = (tok >= 0) & (tok < vocab)
            gg = np.abs(np.where(live, g.reshape(rows, -1), 0.0))
            mag += gg.sum(axis=1, keepdims=True) * p
            np.add.at(mag, (np.arange(rows)[:, None], np.where(live, tok, 0)), gg)
        if gh is not None:
            mag += np.abs(gh)[:, None] * np.where(p > 0, p * (np.abs(lp) + ref["entropy"][:, None] + 4 + np.log(vocab)), 0.0)
    last = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    # below 1e-37 float32 is subnormal
    return scale * mag * (8 * tol[:, None] + last) + 1e-37


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,pad,n,ent,scale", [
    (1, 1, 0, 1, True, 1.0), (3, 5, 2, 1, False, 1.0), (2, 4096, 0, 4, True, 0.7), (7, 1001, 3, 2, True, 1.3),
    (1, 131072, 0, 1, True, 1.0), (3, 32003, 0, 1, False, 1.0), (1100, 520, 0, 1, True, 1.0),
    (1100, 131, 0, 3, False, 0.5), (2, 9000, 0, 0, True, 1.0), (2, 700, 0, 1024, False, 1.0)])
def test_gradient(rows, vocab, pad, n, ent, scale, dtype):
    d = device()
    x = _logits(rows, vocab, dtype, 77 + vocab, pad, banned=vocab > 1000)
    rg = torch.Generator().manual_seed(6)
    tok = torch.randint(-1, vocab, (rows, n), generator=rg).to(d) if n else None
    g = torch.randn((rows, n), generator=rg).to(d) if n else None
    gh = torch.randn((rows,), generator=rg).to(d) if ent else None
    o, st = _forward(x, tok, scale, 0)
    assert st == 0
    xn, sc = _f64(x), float(np.float32(scale))
    tn = None if tok is None else tok.cpu().numpy()
    gn, hn = None if g is None else _f64(g), None if gh is None else _f64(gh)
    want = oracle.logprobs_grad(xn, sc, tn, gn, hn)
    ref = oracle.logprobs(xn, sc, tn)
    lim = _grad_bound(xn, sc, tn, gn, hn, ref, dtype)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    buf = torch.full((rows, vocab + pad + 1), 9.0, dtype=dtype, device=d)

    dx = buf[:, :vocab]                          # rows aligned otherwise than the logits'
    e8q.e8q_token_logprobs_backward(x, o["lse"], dx, status, tokens=tok, grad_logprob=g, scale=scale,
                                    entropy=o["entropy"] if ent else None, grad_entropy=gh)
    _close(_f64(dx), want, lim, "backward")
    assert (buf[:, vocab:] == 9.0).all()
    inplace = x.clone()
    e8q.e8q_token_logprobs_backward(inplace, o["lse"], inplace, status, tokens=tok, grad_logprob=g, scale=scale,
                                    entropy=o["entropy"] if ent else None, grad_entropy=gh)
    assert torch.equal(inplace, dx)

    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab), dtype=torch.uint8, device=d)
    lse, h = torch.empty(rows, device=d), torch.empty(rows, device=d)
    lp = torch.empty((rows, n), device=d) if n else None
    one = torch.full_like(buf, 9.0)
    e8q.e8q_token_logprobs_grad(x, tok, g, one[:, :vocab], ws, status, grad_entropy=gh, scale=scale,
                                logprob_out=lp, lse_out=lse, entropy_out=h)
    _close(_f64(one[:, :vocab]), want, lim, "one call")
    assert (one[:, vocab:] == 9.0).all()
    tol = _bound(ref, xn, sc)
    _close(_f64(lse), ref["lse"], tol, "lse of the one call")
    _close(_f64(h), ref["entropy"], tol * (4 + ref["entropy"] + np.log(vocab)), "entropy of the one call")
    if n:
        _close(_f64(lp), ref["logprob"], tol[:, None] + U * np.abs(ref["logprob"]), "logprob of the one call")
    inplace = x.clone()
    e8q.e8q_token_logprobs_grad(inplace, tok, g, inplace, ws, status, grad_entropy=gh, scale=scale)
    assert torch.equal(inplace, one[:, :vocab].contiguous())
    assert int(status.item()) == 0


def test_gradient_against_differences():
    """Central differences of the GPU's own float32 outputs."""
    d = device()
    x = _logits(2, 40, torch.float32, 12) / 3
    tok = torch.tensor([[3, 7], [0, 39]], device=d)
    g, gh = torch.tensor([[1.0, -2.0], [0.5, 0.25]], device=d), torch.tensor([0.5, -1.0], device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    dx = torch.empty_like(x)
    o, _ = _forward(x, tok, 1.0, 0)
    e8q.e8q_token_logprobs_backward(x, o["lse"], dx, st, tokens=tok, grad_logprob=g, entropy=o["entropy"],
                                    grad_entropy=gh)
    h = 2.0 ** -6                                     # truncation h^2 |f'''| / 6, rounding 2^-20 / h

    def loss(v):
        r, _ = _forward(v, tok, 1.0, 0)
        return (_f64(r["logprob"]) * _f64(g)).sum() + (_f64(r["entropy"]) * _f64(gh)).sum()

    for i, j in ((0, 3), (0, 7), (0, 20), (1, 0), (1, 5)):
        a, b = x.clone(), x.clone()
        a[i, j] += h
        b[i, j] -= h
        assert abs((loss(a) - loss(b)) / (2 * h) - float(dx[i, j])) < 2e-3


def test_other_stream_and_repeated_calls_give_the_same_bits():
    d = device()
    x = _logits(5, 50001, torch.bfloat16, 21)
    tok = torch.arange(5, device=d)
    a, _ = _forward(x, tok, 1.0, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = _forward(x, tok, 1.0, 12, stream=s)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_offsets_past_32_bits():
    """Rows that start past 2^32 elements."""
    d = device()
    stride, vocab = (1 << 31) + 24, 1000
    buf = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device=d)
    x = buf.as_strided((3, vocab), (stride, 1))
    src = _logits(3, vocab, torch.bfloat16, 30)
    x.copy_(src)
    tok = torch.tensor([1, 999, 5], device=d)
    a, _ = _forward(x, tok, 1.0, 4)
    b, _ = _forward(src, tok, 1.0, 4)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    st = torch.zeros(1, dtype=torch.int32, device=d)
    g = torch.ones((3, 1), device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(3, vocab), dtype=torch.uint8, device=d)
    want = torch.empty_like(src)
    e8q.e8q_token_logprobs_grad(src, tok, g, want, ws, st)
    e8q.e8q_token_logprobs_grad(x, tok, g, x, ws, st)
    assert torch.equal(x.contiguous(), want)


def test_refusals():
    d = device()
    x = _logits(2, 64, torch.float32, 1)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=d)
    lse = torch.empty(2, device=d)
    with pytest.raises(ValueError):
        e8q.e8q_token_logprobs(x.t(), ws, st, lse_out=torch.empty(64, device=d))     # columns not contiguous
    with pytest.raises(TypeError):
        e8q.e8q_token_logprobs(x.half(), ws, st, lse_out=lse)
    with pytest.raises(TypeError):
        e8q.e8q_token_logprobs(x, ws, st, tokens=torch.zeros(2, device=d), lse_out=lse)
    with pytest.raises(ValueError):
        e8q.e8q_token_logprobs(x, ws, st, tokens=torch.zeros(3, dtype=torch.int64, device=d), lse_out=lse)
    with pytest.raises(ValueError):
        e8q.e8q_token_logprobs(x, ws, st, lse_out=torch.empty(3, device=d))
    with pytest.raises(e8q.E8QError):
        e8q.e8q_token_logprobs(x, ws, st, scale=-1.0, lse_out=lse)
    with pytest.raises(e8q.E8QError):
        e8q.e8q_token_logprobs(x, ws, st)                                            # no output
    with pytest.raises(e8q.E8QError):
        e8q.e8q_token_logprobs(x, ws, st, top_idx_out=torch.empty((2, 65), dtype=torch.int32, device=d))
    with pytest.raises(e8q.E8QError):
        e8q.e8q_token_logprobs(_logits(1, 131072, torch.float32, 1), ws[:16], st, lse_out=lse[:1])   # workspace
    with pytest.raises(ValueError):
        e8q.e8q_token_logprobs_backward(x, lse, torch.empty((2, 63), device=d), st)
    assert int(st.item()) == 0
