"""e8q_embed and e8q_embed_backward against float64.

The lookup is one float32 product and one rounding: bit for bit.  The gradient
adds c rows of a token in float32 (error at most (c + 1) 2^-24 of the sum of
absolute values), times scale (2^-24), and rounds once to its type."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tokens(n, vocab, seed, kind="text"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        t = np.full(n, vocab // 2)
    elif kind == "distinct":
        t = rng.permutation(vocab)[:n]
    else:
        t = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1.0)).astype(np.int64) - 1, vocab - 1)
        t[rng.random(n) < 0.05] = -1
    return torch.from_numpy(np.asarray(t, np.int64)).to(device())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,dim,scale", [(1, 1, 1, 1.0), (1, 7, 4096, 64.0), (5, 100, 33, 0.37), (64, 1000, 768, 1.0),
                                               (1001, 300, 1001, 2.5), (3, 50, 6, 1.0), (2, 9, 4100, 1.0)])
def test_lookup_bit_for_bit(n, vocab, dim, scale, dtype, out_dtype):
    d = device()
    tab = torch.randn((vocab, dim), generator=torch.Generator().manual_seed(n + dim)).to(dtype).to(d)
    for idx in (torch.int64, torch.int32):
        tok = _tokens(n, vocab, dim).to(idx)
        out = torch.full((n, dim), 9.0, dtype=out_dtype, device=d)
        st = torch.zeros(1, dtype=torch.int32, device=d)
        e8q.e8q_embed(tab, tok, out, st, scale=scale)
        live = (tok >= 0)[:, None]
        want = tab[tok.clamp(min=0).long()].float() * torch.tensor(scale, dtype=torch.float32, device=d)
        want = torch.where(live, want, torch.zeros_like(want)).to(out_dtype)
        assert torch.equal(out, want) and int(st.item()) == 0


def test_lookup_padded_and_out_of_range_ids():
    d = device()
    tab = torch.randn((4, 24), device=d)
    tok = torch.tensor([-1, 4, 3, 2 ** 40, -2 ** 40], device=d)
    out = torch.full((5, 24), 9.0, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    e8q.e8q_embed(tab, tok, out, st)
    assert int(st.item()) == e8q.STATUS_BITS["BAD_INDEX"]
    assert torch.equal(out[2], tab[3]) and not out[[0, 1, 3, 4]].any()
    # unaligned table and output rows
    buf = torch.randn(4 * 24 + 1, device=d)
    tab = buf[1:].view(4, 24)
    o = torch.empty(3 * 24 + 3, dtype=torch.bfloat16, device=d)[3:].view(3, 24)
    e8q.e8q_embed(tab, torch.tensor([2, 0, 2], device=d), o, st)
    assert torch.equal(o, tab[[2, 0, 2]].to(torch.bfloat16))


def _backward(g, tok, vocab, dtype, scale, latents=None, lr=1.0, stream=None):
    d, dim = g.device, g.shape[1]
    out = None if dtype is None else torch.full((vocab, dim), 9.0, dtype=dtype, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.full((e8q.e8q_embed_backward_workspace_size(tok.numel(), vocab, dim),), 0xA5, dtype=torch.uint8, device=d)
    e8q.e8q_embed_backward(g, tok, vocab, ws, st, scale=scale, grad_table=out, w_latent=latents, lr=lr, stream=stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def _check(got, g, tok, vocab, scale, dtype):
    sc = float(np.float32(scale))
    want, mag = oracle.embed_grad(_f64(g), tok.cpu().numpy(), vocab, sc)
    t = tok.cpu().numpy()
    cnt = np.bincount(t[(t >= 0) & (t < vocab)], minlength=vocab)[:, None]
    lim = (cnt + 2) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0) + 1e-38
    assert (np.abs(_f64(got) - want) <= lim).all()


@pytest.mark.parametrize("gdtype", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,dim,kind", [
    (1, 1, 1, "text"), (1, 5, 8, "one"), (31, 40, 17, "text"), (32, 40, 64, "one"), (33, 64, 6, "one"),
    (64, 64, 12, "distinct"), (65, 3, 4, "text"), (999, 501, 101, "text"), (4096, 1023, 40, "text"),
    (4097, 1024, 40, "text"), (5000, 1025, 24, "one"), (10000, 131072, 8, "text"), (9000, 70000, 1, "distinct"),
    (300, 20, 2100, "text")])
def test_gradient(n, vocab, dim, kind, dtype, gdtype):
    d = device()
    g = torch.randn((n, dim), generator=torch.Generator().manual_seed(n)).to(gdtype).to(d)
    tok = _tokens(n, vocab, n + dim, kind)
    tok = tok.to(torch.int32) if n % 2 else tok
    got, st = _backward(g, tok, vocab, dtype, 1.75)
    assert st == 0
    _check(got, g, tok, vocab, 1.75, dtype)
    again, _ = _backward(g, tok, vocab, dtype, 1.75)
    assert torch.equal(got, again)


@pytest.mark.parametrize("n,vocab,dim", [(700, 90, 48), (6000, 5000, 33)])
def test_latents_step(n, vocab, dim):
    """w <- bf16(w - lr g) on the rows that occur; the others keep their bits."""
    d = device()
    g = torch.randn((n, dim), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(d)
    tok = _tokens(n, vocab, 4)
    w0 = (torch.randn((vocab, dim), generator=torch.Generator().manual_seed(5))).to(torch.bfloat16).to(d)
    w = w0.clone()
    grad, _ = _backward(g, tok, vocab, torch.float32, 0.5, w, 0.25)
    only = w0.clone()
    _backward(g, tok, vocab, None, 0.5, only, 0.25)
    assert torch.equal(w, only)
    lr = torch.tensor(0.25, device=d)
    want = (w0.float() - lr * grad).to(torch.bfloat16)
    there = torch.zeros(vocab, dtype=torch.bool, device=d)
    there[tok[tok >= 0]] = True
    assert torch.equal(w[there], want[there]) and torch.equal(w[~there], w0[~there])


def test_ids_that_do_not_count():
    d = device()
    g = torch.ones((5, 16), device=d)
    tok = torch.tensor([-1, 9, -5, 2 ** 33, -1], device=d)
    got, st = _backward(g, tok, 9, torch.float32, 1.0)
    assert st == e8q.STATUS_BITS["BAD_INDEX"] and not got.any()
    got, st = _backward(g, torch.full((5,), -1, device=d), 9, torch.bfloat16, 1.0)
    assert st == 0 and not got.any()
    nan = g.clone()
    nan[0] = float("nan")                                  # a padded position's gradient does not leak
    got, _ = _backward(nan, torch.tensor([-1, 2, 2, 3, 2], device=d), 9, torch.float32, 1.0)
    assert torch.isfinite(got).all() and (got[2] == 3).all() and (got[3] == 1).all()


def test_gradient_against_differences():
    """The lookup is linear in the table: <grad_out, E(T + D) - E(T)> = <grad, D>."""
    d = device()
    tok = _tokens(200, 37, 8)
    tab = torch.randint(-8, 8, (37, 20), generator=torch.Generator().manual_seed(1)).float().to(d)
    step = torch.randint(-4, 4, (37, 20), generator=torch.Generator().manual_seed(2)).float().to(d)
    g = torch.randint(-4, 4, (200, 20), generator=torch.Generator().manual_seed(3)).float().to(d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    a, b = torch.empty((200, 20), device=d), torch.empty((200, 20), device=d)
    e8q.e8q_embed(tab + step, tok, a, st, scale=2.0)
    e8q.e8q_embed(tab, tok, b, st, scale=2.0)
    grad, _ = _backward(g, tok, 37, torch.float32, 2.0)
    assert (_f64(g) * (_f64(a) - _f64(b))).sum() == (_f64(grad) * _f64(step)).sum()     # small integers: exact


def test_other_stream():
    d = device()
    g = torch.randn((5000, 64), device=d)
    tok = _tokens(5000, 999, 1)
    a, _ = _backward(g, tok, 999, torch.float32, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = _backward(g, tok, 999, torch.float32, 1.0, stream=s)
    assert torch.equal(a, b)


def test_refusals():
    d = device()
    st = torch.zeros(1, dtype=torch.int32, device=d)
    tab, tok = torch.zeros((4, 8), device=d), torch.zeros(3, dtype=torch.int64, device=d)
    with pytest.raises(ValueError):
        e8q.e8q_embed(tab, tok, torch.empty((3, 9), device=d), st)
    with pytest.raises(TypeError):
        e8q.e8q_embed(tab, tok.float(), torch.empty((3, 8), device=d), st)
    with pytest.raises(ValueError):
        e8q.e8q_embed(tab.t(), tok, torch.empty((3, 4), device=d), st)
    ws = torch.empty(e8q.e8q_embed_backward_workspace_size(3, 4, 8), dtype=torch.uint8, device=d)
    g = torch.zeros((3, 8), device=d)
    with pytest.raises(e8q.E8QError):
        e8q.e8q_embed_backward(g, tok, 4, ws, st)                                     # no output
    with pytest.raises(e8q.E8QError):
        e8q.e8q_embed_backward(g, tok, 4, ws[:256], st, grad_table=tab)
    with pytest.raises(ValueError):
        e8q.e8q_embed_backward(g, tok, 5, ws, st, grad_table=tab)
    with pytest.raises(TypeError):
        e8q.e8q_embed_backward(g, tok, 4, ws, st, w_latent=tab)
    assert int(st.item()) == 0
