"""Batches that give every row one block: the loop of the forward pass past its
first round, with and without alternatives, and the gradient's kernel for every
length of row, with masked, lowest-value, NaN and infinite rows among them.

Against float64 on the GPU.  Bounds as in test_gpu_logprobs_offsets: with
d = scale (x - max), u = 2^-23 and r = u (16 + 4 log2 V + V / 64) (a thread adds at
most V / 64 terms one after another), ln sum and p are within r, p also within
u |2 d| of itself, the entropy within r (4 + H + log V), a log probability within
r + u (|d| + |its value|)."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
from gpu_util import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NONFINITE = e8q.STATUS_BITS["NONFINITE"]


def _splits(rows, vocab, dtype):
    """Blocks per row: the library's rule."""
    ve = 8 if dtype == torch.bfloat16 else 4
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    nvec = (vocab + ve - 1) // ve
    return max(1, min((4 * cus + rows - 1) // rows, (nvec + 1023) // 1024, 256)), nvec


def _logits(rows, vocab, dtype, pad, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, vocab + pad), generator=g, device=device()) * 3
    x[rows // 3, vocab // 3:] = -float("inf")
    x[5] = -float("inf")                                      # nothing left
    x[6] = torch.finfo(dtype).min                             # the lowest value everywhere
    x[7] = -float("inf")
    x[7, vocab - 1] = 2.0                                     # one logit left, the last
    x = x.to(dtype)
    x[8] = torch.finfo(dtype).min
    x[8, vocab // 2] = -3.0
    return x[:, :vocab]


BAD = {9: float("nan"), 10: float("inf"), 11: -float("nan")}


class Reference:
    """Of rows in float64, in parts that fit."""

    def __init__(self, x, scale, tok, g=None, gh=None):
        rows, vocab = x.shape
        self.r = U * (16 + 4 * np.log2(max(vocab, 2)) + vocab / 64)
        y = x.double()
        m = y.amax(dim=1, keepdim=True)
        d = torch.where(torch.isneginf(m), torch.full_like(y, -float("inf")), (y - m) * scale)
        s = d.exp().sum(dim=1, keepdim=True)
        empty = torch.isneginf(m)
        self.d = d
        self.lp = torch.where(empty, torch.full_like(d, -float("inf")), d - s.log())
        self.p = torch.where(empty, torch.zeros_like(d), self.lp.exp())
        plp = torch.where(self.p == 0, torch.zeros_like(d), self.p * self.lp)
        self.entropy = -plp.sum(dim=1)
        self.lse = torch.where(empty, m, m * scale + s.log())[:, 0]
        live = (tok >= 0) & (tok < vocab)
        self.live, self.take = live, tok.clamp(0, vocab - 1).long()
        self.logprob = torch.where(live, self.lp.gather(1, self.take), torch.zeros_like(tok, dtype=torch.float64))
        self.tok_d = torch.where(live, d.gather(1, self.take), torch.zeros_like(self.logprob))
        if g is None:
            return
        gg = torch.where(live, g.double(), torch.zeros_like(self.logprob))
        dx = -gg.sum(dim=1, keepdim=True) * self.p
        mag = gg.abs().sum(dim=1, keepdim=True) * self.p
        at = torch.zeros_like(d).scatter_add_(1, self.take, gg.abs())
        dx.scatter_add_(1, self.take, gg)
        if gh is not None:
            h = self.entropy[:, None]
            dx -= gh.double()[:, None] * torch.where(self.p == 0, torch.zeros_like(d), plp + self.p * h)
            mag += gh.double().abs()[:, None] * (plp.abs() + self.p * (h + 4 + np.log(vocab)))
        dx = torch.where(empty, torch.zeros_like(dx), dx)
        off = torch.where(self.p == 0, torch.zeros_like(d), 8 * self.r + 2 * U * d.abs())
        last = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -22
        self.dx = dx * scale
        self.lim = scale * (torch.where(self.p == 0, torch.zeros_like(d), mag * off) + 2.0 ** -22 * at) + last * self.dx.abs() + 1e-37


def _close(got, want, lim, what):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), what
    fin = want.isfinite()
    assert torch.equal(got[~fin & ~want.isnan()], want[~fin & ~want.isnan()]), what
    lim = lim.expand_as(want) if torch.is_tensor(lim) else torch.full_like(want, lim)
    off = (got - want).abs()[fin]
    assert bool((off <= lim[fin]).all()), (what, float((off / lim[fin]).max()))


def _check_outputs(o, ref, vocab, rows=slice(None)):
    _close(o["lse"][rows], torch.where(ref.lse.abs() > 3.4e38, ref.lse.float().double(), ref.lse),
           ref.r + 2 * U * torch.where(ref.lse.isfinite(), ref.lse.abs(), torch.zeros_like(ref.lse)), "lse")
    _close(o["entropy"][rows], ref.entropy, ref.r * (4 + ref.entropy + np.log(vocab)), "entropy")
    fin = torch.where(ref.logprob.isfinite(), ref.logprob.abs() + ref.tok_d.abs(), torch.zeros_like(ref.logprob))
    want = torch.where(ref.logprob < -3.4e38, torch.full_like(ref.logprob, -float("inf")), ref.logprob)
    _close(o["logprob"][rows], want, ref.r + U * fin, "logprob")


GRAD = [(torch.bfloat16, 2048), (torch.bfloat16, 4090), (torch.bfloat16, 8191), (torch.bfloat16, 8193),
        (torch.bfloat16, 16384), (torch.bfloat16, 16390), (torch.bfloat16, 32768), (torch.bfloat16, 32769),
        (torch.bfloat16, 50001), (torch.float32, 1000), (torch.float32, 2048), (torch.float32, 4096),
        (torch.float32, 4097), (torch.float32, 8191), (torch.float32, 8200), (torch.float32, 16384),
        (torch.float32, 16385), (torch.float32, 32003), (torch.float32, 32769), (torch.float32, 40000)]


@pytest.mark.parametrize("dtype,vocab", GRAD)
@pytest.mark.parametrize("pad,ntok,ent,scale", [(0, 1, True, 1.0), (13, 3, False, 0.7)])
def test_gradient_of_batches(dtype, vocab, pad, ntok, ent, scale):
    d, rows = device(), 1030
    assert _splits(rows, vocab, dtype)[0] == 1
    x = _logits(rows, vocab, dtype, pad, vocab)
    g0 = torch.Generator(device="cuda").manual_seed(1)
    tok = torch.randint(-1, vocab, (rows, ntok), generator=g0, device=d)
    tok[:, 0] = (torch.arange(rows, device=d) * 37) % vocab
    tok[7, 0], tok[8, 0] = vocab - 1, vocab // 2
    g = torch.randn((rows, ntok), generator=g0, device=d)
    gh = torch.randn(rows, generator=g0, device=d) if ent else None
    for row, v in BAD.items():
        x[row, vocab - 2 if row == 10 else vocab // 5] = v
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab), dtype=torch.uint8, device=d)
    o = {"logprob": torch.empty((rows, ntok), device=d), "lse": torch.empty(rows, device=d), "entropy": torch.empty(rows, device=d)}
    buf = torch.full((rows, vocab + 5), 9.0, dtype=dtype, device=d)
    dx = buf[:, 1:vocab + 1]
    e8q.e8q_token_logprobs_grad(x, tok, g, dx, ws, st, grad_entropy=gh, scale=scale, logprob_out=o["logprob"],
                                lse_out=o["lse"], entropy_out=o["entropy"])
    assert int(st.item()) == NONFINITE and bool((buf[:, 0] == 9).all()) and bool((buf[:, vocab + 1:] == 9).all())
    sc = float(np.float32(scale))
    good = [r for r in range(rows) if r not in BAD]
    for part in torch.tensor(good, device=d).split(128):
        ref = Reference(x[part], sc, tok[part], g[part], None if gh is None else gh[part])
        _close(dx[part], ref.dx, ref.lim, "gradient")
        _check_outputs({k: v[part] for k, v in o.items()}, ref, vocab)
    bad = list(BAD)
    assert bool(dx[bad].isnan().all()) and bool(o["lse"][bad].isnan().all()) and bool(o["entropy"][bad].isnan().all())
    assert not bool(dx[5].any())
    # the same from the stored lse: p within 2^-20 more
    two = torch.full_like(buf, 9.0)[:, 1:vocab + 1]
    e8q.e8q_token_logprobs_backward(x, o["lse"], two, st, tokens=tok, grad_logprob=g, scale=scale,
                                    entropy=o["entropy"] if ent else None, grad_entropy=gh)
    for part in torch.tensor(good, device=d).split(128):
        ref = Reference(x[part], sc, tok[part], g[part], None if gh is None else gh[part])
        more = (ref.p * (g[part].abs().sum(dim=1, keepdim=True) + (0 if gh is None else gh[part].abs()[:, None])) * sc
                * 2.0 ** -20 * (8 + np.log(vocab) + torch.where(ref.p == 0, torch.zeros_like(ref.d), ref.d.abs())))
        _close(two[part], ref.dx, ref.lim + more, "backward")
    # in place: the same bits
    own = x.clone()
    e8q.e8q_token_logprobs_grad(own, tok, g, own, ws, st, grad_entropy=gh, scale=scale)
    assert torch.equal(own[good], dx[good]) and bool(own[bad].isnan().all())
    own = x.clone()
    e8q.e8q_token_logprobs_backward(own, o["lse"], own, st, tokens=tok, grad_logprob=g, scale=scale,
                                    entropy=o["entropy"] if ent else None, grad_entropy=gh)
    assert torch.equal(own[good], two[good])


def _order(x, k):
    """Indices by value, equal values by index, NaN first."""
    v = x.float() + 0.0
    v = torch.where(v.isnan(), torch.full_like(v, float("inf")), v)
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]


def _kinds(rows, vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    d = device()
    yield "random", _logits(rows, vocab, dtype, 3, vocab)
    ties = torch.round(torch.randn((rows, vocab), generator=g, device=d) * 2).to(dtype)
    ties[:, ::2] *= -1
    yield "ties", ties
    up = (torch.arange(vocab, device=d, dtype=torch.float32) / 512).to(dtype).expand(rows, vocab).contiguous()
    yield "ascending", up
    yield "descending", up.flip(1).contiguous()
    late = torch.full((rows, vocab), -float("inf"), dtype=dtype, device=d)
    late[:, -70:] = torch.randn((rows, 70), generator=g, device=d).to(dtype)
    yield "late", late                                        # the first rounds hold nothing
    yield "equal", torch.full((rows, vocab), 2.5, dtype=dtype, device=d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,k", [(1030, 20000, 0), (1030, 20000, 20), (1027, 33001, 64), (1100, 9001, 1), (600, 40001, 7),
                                          (1025, 8192, 5)])
def test_forward_past_the_first_round(rows, vocab, k, dtype):
    d = device()
    splits, nvec = _splits(rows, vocab, dtype)
    per = (nvec + splits - 1) // splits
    assert per > 1024 or vocab == 8192                        # one block reads more than a round of its part
    g0 = torch.Generator(device="cuda").manual_seed(2)
    tok = torch.randint(-1, vocab, (rows, 2), generator=g0, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab, k), dtype=torch.uint8, device=d)
    for name, x in _kinds(rows, vocab, dtype):
        o = {"logprob": torch.empty((rows, 2), device=d), "lse": torch.empty(rows, device=d), "entropy": torch.empty(rows, device=d)}
        idx = torch.full((rows, k), -7, dtype=torch.int32, device=d) if k else None
        top = torch.full((rows, k), 9.0, device=d) if k else None
        e8q.e8q_token_logprobs(x, ws, st, tokens=tok, scale=0.8, logprob_out=o["logprob"], lse_out=o["lse"],
                               entropy_out=o["entropy"], top_idx_out=idx, top_logprob_out=top)
        assert int(st.item()) == 0, name
        for lo in range(0, rows, 128):
            part = slice(lo, min(lo + 128, rows))
            ref = Reference(x[part], float(np.float32(0.8)), tok[part])
            _check_outputs(o, ref, vocab, part)
            if k:
                order = _order(x[part], k)
                assert torch.equal(idx[part].long(), order), name
                want, off = ref.lp.gather(1, order), ref.d.gather(1, order)
                fin = torch.where(want.isfinite(), want.abs() + off.abs(), torch.zeros_like(want))
                want = torch.where(want < -3.4e38, torch.full_like(want, -float("inf")), want)
                _close(top[part], want, ref.r + U * fin, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity_past_the_first_round(dtype):
    d, rows, vocab, k = device(), 1030, 30000, 9
    x = _logits(rows, vocab, dtype, 0, 4)
    where = {20: (25000, "nan"), 21: (29999, "inf"), 22: (9000, "-nan"), 23: (24001, "nan")}
    for row, (at, v) in where.items():
        x[row, at] = float(v)
    x[23, 3] = float("nan")
    idx, lse = torch.empty((rows, k), dtype=torch.int32, device=d), torch.empty(rows, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(rows, vocab, k), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs(x, ws, st, lse_out=lse, top_idx_out=idx)
    assert int(st.item()) == NONFINITE
    bad = list(where)
    assert bool(lse[bad].isnan().all()) and int(lse.isnan().sum()) == len(bad)
    assert torch.equal(idx.long(), _order(x, k)) and idx[23, 0] == 3 and idx[23, 1] == 24001
