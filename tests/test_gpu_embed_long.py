"""e8q_embed_backward on long batches: both sides of the switch at 65536 ids, past
which the sort's counts are summed by a kernel of their own, for keys of one, two and three
digits; and one workspace for batches of several lengths.

Bound as in test_gpu_embed: c rows of a token add up to (c + 1) 2^-24 of the sum of
absolute values, times scale 2^-24 more, and one rounding to the result's type."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tokens(n, vocab, kind):
    rng = np.random.default_rng(n + vocab)
    if kind == "one":
        t = np.full(n, vocab - 1)
    elif kind == "descending":
        t = (np.arange(n) * 7 // 5)[::-1] % vocab
    else:
        t = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1.0)).astype(np.int64) - 1, vocab - 1)
        t = t * 40503 % vocab
        t[rng.random(n) < 0.05] = -1
    return torch.from_numpy(np.ascontiguousarray(t, np.int64)).to(device())


def _backward(g, tok, vocab, ws=None, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=g.device)
    if ws is None:
        size = e8q.e8q_embed_backward_workspace_size(tok.numel(), vocab, g.shape[1])
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=g.device)
    e8q.e8q_embed_backward(g, tok, vocab, ws, st, **kw)
    return int(st.item())


@pytest.mark.parametrize("kind", ["text", "one", "descending"])
@pytest.mark.parametrize("vocab,dim", [(900, 8), (50001, 6), (1500007, 2)])
@pytest.mark.parametrize("n", [65536, 65537, 200003])
def test_gradient(n, vocab, dim, kind):
    d = device()
    dtype = torch.bfloat16 if n % 2 else torch.float32
    g = torch.randn((n, dim), generator=torch.Generator().manual_seed(n)).to(dtype).to(d)
    tok = _tokens(n, vocab, kind)
    tok = tok.to(torch.int32) if kind == "text" else tok
    got = torch.full((vocab, dim), 9.0, device=d)
    assert _backward(g, tok, vocab, scale=1.75, grad_table=got) == 0
    t = tok.cpu().numpy()
    want, mag = oracle.embed_grad(_f64(g), t, vocab, 1.75)
    cnt = np.bincount(t[t >= 0], minlength=vocab)[:, None]
    assert (np.abs(_f64(got) - want) <= (cnt + 2) * 2.0 ** -24 * mag + 1e-38).all()
    again = torch.full((vocab, dim), 7.0, device=d)
    w0 = torch.randn((vocab, dim), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(d)
    w = w0.clone()
    assert _backward(g, tok, vocab, scale=1.75, grad_table=again, w_latent=w, lr=0.25) == 0
    assert torch.equal(got, again)
    there = torch.zeros(vocab, dtype=torch.bool, device=d)
    there[tok[tok >= 0].long()] = True
    step = (w0.float() - 0.25 * got).to(torch.bfloat16)
    assert torch.equal(w, torch.where(there[:, None], step, w0))


def test_ids_out_of_range():
    d, n, vocab = device(), 70000, 3000
    tok = _tokens(n, vocab, "text")
    tok[60000:60010] = vocab
    tok[69999] = 2 ** 40
    g = torch.ones((n, 4), device=d)
    got = torch.empty((vocab, 4), device=d)
    assert _backward(g, tok, vocab, grad_table=got) == e8q.STATUS_BITS["BAD_INDEX"]
    t = tok.cpu().numpy()
    assert (got[:, 0].cpu().numpy() == np.bincount(t[(t >= 0) & (t < vocab)], minlength=vocab)).all()


def test_other_stream():
    d, n, vocab = device(), 100000, 5000
    g, tok = torch.randn((n, 16), device=d), _tokens(n, vocab, "text")
    a, b = torch.empty((vocab, 16), device=d), torch.empty((vocab, 16), device=d)
    _backward(g, tok, vocab, grad_table=a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    size = e8q.e8q_embed_backward_workspace_size(n, vocab, 16)
    ws, st = torch.empty(size, dtype=torch.uint8, device=d), torch.zeros(1, dtype=torch.int32, device=d)
    s.wait_stream(torch.cuda.current_stream())
    e8q.e8q_embed_backward(g, tok, vocab, ws, st, grad_table=b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_one_workspace_for_smaller_batches():
    d, vocab, dim = device(), 700, 40
    ws = torch.full((e8q.e8q_embed_backward_workspace_size(4104, vocab, dim),), 0xA5, dtype=torch.uint8, device=d)
    g, tok = torch.randn((4104, dim), device=d), _tokens(4104, vocab, "text")
    for n in (4104, 4096, 3000, 1):
        a, b = torch.empty((vocab, dim), device=d), torch.empty((vocab, dim), device=d)
        _backward(g[:n], tok[:n], vocab, ws, grad_table=a)
        _backward(g[:n], tok[:n], vocab, grad_table=b)
        assert torch.equal(a, b)
