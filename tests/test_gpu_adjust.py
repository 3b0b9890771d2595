"""e8q_adjust_logits against float64.

Bounds, u = 2^-24: the penalty's division or product is off by u |y| (a subnormal
quotient by 2^-148), f c + p by u (2 |f c| + |p|), each difference and sum by u of its result; m biases by
u m sum |b|; one rounding to the type.  All of it: u (4 |x'| + 4 |f c| + 4 |p| + (m + 2) sum |b|)."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ALL = ("repetition", "frequency", "presence")


def make(rows, vocab, dtype, cols, n_bias, mask, seed, index=torch.int64, pad=0, penalties=ALL):
    d = device()
    g = torch.Generator(device=d).manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device=d)  # noqa: E731
    x = (torch.randn((rows, vocab + pad), generator=g, device=d) * 3).to(dtype)[:, :vocab]
    a = {}
    if cols:
        a["history"] = (rand(rows, cols) ** 3 * vocab).to(index)        # low ids often
        a["history_len"] = (rand(rows) * (cols + 1)).to(torch.int32)
        a["prompt_len"] = (rand(rows) * (a["history_len"] + 1)).to(torch.int32)
        for n, lo, hi in (("repetition", 0.8, 1.4), ("frequency", -0.2, 0.9), ("presence", -0.5, 0.9)):
            if n in penalties:
                a[n] = lo + (hi - lo) * rand(rows)
    if n_bias:
        a["bias_idx"] = (rand(rows, n_bias) ** 2 * vocab).to(index)
        a["bias"] = torch.randn((rows, n_bias), generator=g, device=d) * 4
    if mask:
        words = (vocab + 31) // 32
        bits = rand(rows, words, 32) < torch.where(rand(rows) < 0.5, 0.02, 0.98)[:, None, None]
        v = (bits.long() << torch.arange(32, device=d)).sum(dim=2)
        a["mask"] = torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)
    return x, a


def run(x, a, out=None, stream=None):
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device=x.device) if out is None else out
    st = torch.zeros(1, dtype=torch.int32, device=x.device)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    e8q.e8q_adjust_logits(x, out, st, stream=stream, **a)
    torch.cuda.synchronize()
    return out, int(st.item())


def check(out, x, a, rows=None):
    sel = np.arange(x.shape[0]) if rows is None else np.asarray(rows)
    t = torch.from_numpy(sel).to(x.device)
    pick = {}
    for n, v in a.items():
        v = v if v.dim() == 1 and n not in ("bias_idx", "bias", "mask") else (v.expand(x.shape[0], -1) if v.dim() == 1 or v.shape[0] == 1 else v)
        pick[n] = v[t].cpu().numpy()
    xs = x[t].float().cpu().numpy().astype(np.float64)
    vocab = x.shape[1]
    want = oracle.adjust_logits(xs, **pick)
    with np.errstate(all="ignore"):                        # past float32's range: an infinity there
        want = np.where(np.isinf(want.astype(np.float32)), np.sign(want) * np.inf, want)
    # the size of what is added up: the penalized logit, f c, p and the biases
    size = np.abs(oracle.adjust_logits(xs, **{n: v for n, v in pick.items() if n in (
        "history", "history_len", "prompt_len", "repetition")}))
    zero = {n: v for n, v in pick.items() if n not in ("bias_idx", "bias", "mask", "repetition")}
    for n in ("frequency", "presence"):
        if n in zero:
            zero[n] = -np.abs(zero[n])
    size = 4 * size + 4 * np.abs(oracle.adjust_logits(np.zeros_like(xs), **zero))
    if "bias" in pick:
        size += (2 + pick["bias"].shape[1]) * oracle.adjust_logits(np.zeros_like(xs), bias_idx=pick["bias_idx"],
                                                                   bias=np.abs(pick["bias"]))
    got = out[t].float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fin = np.isfinite(want)
    tol = U * size[fin] + HALF[x.dtype] * np.abs(want[fin]) * (1 + 2.0 ** -20) + 2.0 ** -133
    off = np.abs(got[fin] - want[fin])
    assert (off <= tol).all(), (off.max(), (off / tol).max())
    return want


@pytest.mark.parametrize("rows,vocab,dtype,cols,n_bias,mask,index,pad", [
    (1, 1, torch.float32, 1, 1, True, torch.int64, 0),
    (3, 31, torch.bfloat16, 5, 2, True, torch.int32, 0),
    (2, 33, torch.float32, 0, 40, False, torch.int32, 3),
    (4, 500, torch.bfloat16, 300, 0, False, torch.int64, 1),
    (5, 2051, torch.bfloat16, 1000, 30, True, torch.int64, 0),
    (1, 40001, torch.float32, 3000, 1024, True, torch.int32, 7),
    (7, 12345, torch.bfloat16, 64, 0, True, torch.int64, 0),
    (3, 5000, torch.float32, 0, 0, True, torch.int64, 0),
    (3, 4999, torch.bfloat16, 0, 0, False, torch.int64, 2),          # a copy
    (2100, 300, torch.float32, 20, 3, True, torch.int32, 0),
    (700, 33001, torch.bfloat16, 200, 20, True, torch.int64, 0),     # parts of 16384
    (600, 17000, torch.float32, 2000, 5, False, torch.int32, 1),
])
def test_sizes(rows, vocab, dtype, cols, n_bias, mask, index, pad):
    x, a = make(rows, vocab, dtype, cols, n_bias, mask, rows + vocab, index, pad)
    out, st = run(x, a)
    assert st == 0
    check(out, x, a, rows=None if rows * vocab < 1 << 20 else [0, 1, rows // 2, rows - 1])
    same, _ = run(x, a, stream=torch.cuda.Stream())
    assert torch.equal(out, same)
    y = x.clone()
    wide = torch.zeros((rows, vocab + 9), dtype=dtype, device=x.device)
    run(x, a, out=wide[:, 4:4 + vocab])                    # unaligned rows, nothing written beside them
    assert torch.equal(wide[:, 4:4 + vocab], out) and not wide[:, :4].any() and not wide[:, 4 + vocab:].any()
    run(y, a, out=y)
    assert torch.equal(y, out)


@pytest.mark.parametrize("which", [("repetition",), ("frequency",), ("presence",), ("frequency", "presence")])
def test_each_penalty(which):
    x, a = make(3, 5000, torch.float32, 700, 0, False, 4, penalties=which)
    out, _ = run(x, a)
    check(out, x, a)
    for n in ("history_len", "prompt_len"):
        b = {k: v for k, v in a.items() if k != n}
        if n == "history_len":
            b["history"] = torch.where(torch.arange(700, device=x.device) < a["history_len"][:, None], a["history"], -1)
        out2, _ = run(x, b)
        check(out2, x, b)


def test_shared_lists_views_and_odd_ids():
    x, a = make(5, 9000, torch.float32, 50, 12, True, 6, torch.int32)
    a["bias_idx"], a["bias"] = a["bias_idx"][0].contiguous(), a["bias"][0].contiguous()
    a["mask"] = a["mask"][1].contiguous()
    a["bias_idx"][3] = a["bias_idx"][7]                    # the same token three times
    a["bias_idx"][5] = a["bias_idx"][7]
    a["bias_idx"][1] = -4
    a["history"][0, :7] = -1
    a["history_len"][1] = 0
    a["history_len"][2] = -3
    a["history_len"][3] = 5000                             # more than there are
    a["prompt_len"][3] = 6000
    a["prompt_len"][4] = -1
    out, st = run(x, a)
    assert st == 0
    check(out, x, a)
    # rows of wider tensors
    wide = {"history": torch.nn.functional.pad(a["history"], (0, 9), value=1)[:, :50],
            "mask": torch.nn.functional.pad(a["mask"].expand(5, -1), (0, 3))[:, :282],
            "bias_idx": torch.nn.functional.pad(a["bias_idx"].expand(5, -1), (0, 2))[:, :12],
            "bias": torch.nn.functional.pad(a["bias"].expand(5, -1), (0, 2))[:, :12]}
    again, _ = run(x, {**a, **wide})
    assert torch.equal(out, again)
    a["history"][4, 0] = 9000
    a["history_len"][4] = 3
    out, st = run(x, a)
    assert st == e8q.STATUS_BITS["BAD_INDEX"]
    check(out, x, a)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_values(dtype):
    """Infinities, NaN, zeros, the type's lowest value and subnormals in touched and masked places; a row that the mask
    empties."""
    x, a = make(3, 64, dtype, 64, 0, True, 7)
    x = x.contiguous()
    special = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, torch.finfo(dtype).min,
                            torch.finfo(dtype).max, 1e-39], device=x.device).to(dtype)
    x[:, :8] = special
    x[:, 8:16] = special
    a["history"][:, :8] = torch.arange(8, device=x.device)
    a["history_len"][:] = 8
    a["prompt_len"][:] = 4
    a["presence"][:] = 0.5
    a["frequency"][:] = 0.25
    a["repetition"][:] = 1.25
    a["mask"][0] = -1
    a["mask"][1] = 0
    out, st = run(x, a)
    assert st == 0
    check(out, x, a)
    assert torch.isneginf(out[1]).all() and torch.isnan(out[0, 2]) and torch.isinf(out[0, 0])


def test_counts_past_16_bits():
    """One token made 70000 times."""
    x, a = make(1, 3000, torch.float32, 70001, 0, False, 8)
    a["history"][:] = 17
    a["history_len"][:] = 70001
    a["prompt_len"][:] = 1
    out, _ = run(x, a)
    check(out, x, a)


@pytest.mark.parametrize("vocab,n_bias,same", [(930, 300, 0), (930, 300, 40), (20000, 1024, 1024), (17, 1024, 0),
                                               (300000, 1024, 12)])
def test_many_biases_of_a_token(vocab, n_bias, same):
    """More biases than tokens, one token named more often than a lane looks it up by itself, ids that share their low
    bits."""
    x, a = make(300 if vocab < 1000 else 2, vocab, torch.float32, 20, n_bias, False, vocab + same)
    a["bias_idx"][:, :same] = vocab // 2
    if same == 12:
        a["bias_idx"][:, 12:] = torch.arange(n_bias - 12, device=x.device) % 290 * 1024 + 5
    out, st = run(x, a)
    assert st == 0
    check(out, x, a)
    again, _ = run(x, a)
    assert torch.equal(out, again)


def test_expanded_history_is_refused():
    """Rows of one history in common (a stride of 0) cannot be passed on; biases and masks in common can."""
    x, a = make(3, 500, torch.float32, 9, 4, True, 5)
    for h in (a["history"][:1].expand(3, -1), torch.arange(40, device=x.device).as_strided((3, 9), (4, 1))):
        with pytest.raises(ValueError):
            run(x, {**a, "history": h})
    wide = {**a, "bias_idx": a["bias_idx"][:1].expand(3, -1), "bias": a["bias"][:1].expand(3, -1),
            "mask": a["mask"][:1].expand(3, -1)}
    out, _ = run(x, wide)
    same, _ = run(x, {n: v.contiguous() for n, v in wide.items()})
    assert torch.equal(out, same)


def test_offsets_past_32_bits():
    """Rows of logits that start past 2^32 elements, in place and out of it."""
    x, a = make(3, 1000, torch.bfloat16, 30, 5, True, 9)
    stride = (1 << 31) + 24
    far = torch.empty(2 * stride + 1000, dtype=torch.bfloat16, device=x.device).as_strided((3, 1000), (stride, 1))
    far.copy_(x)
    want, _ = run(x, a)
    got, _ = run(far, a)
    assert torch.equal(got, want)
    run(far, a, out=far)
    assert torch.equal(far.contiguous(), want)


@pytest.mark.parametrize("penalties", [("frequency",), ("presence",), ("repetition",), ALL])
@pytest.mark.parametrize("vocab", [40, 20000])
def test_prompt_ids_past_the_vocabulary(vocab, penalties):
    """An id past the vocabulary is flagged in the prompt too, also where no penalty is for the prompt."""
    x, a = make(2, vocab, torch.float32, 700, 0, False, 13, penalties=penalties)
    a["history_len"][:] = 690
    a["prompt_len"][:] = 600
    out, st = run(x, a)
    assert st == 0
    for at in (0, 599):
        b = {**a, "history": a["history"].clone()}
        b["history"][1, at] = vocab + at
        out, st = run(x, b)
        assert st == e8q.STATUS_BITS["BAD_INDEX"]
        check(out, x, b)
    b["history"][1, 599] = -1
    b["history"][1, 690] = vocab                           # behind the history's end: not read as an id
    out, st = run(x, b)
    assert st == 0


@pytest.mark.parametrize("value", [float("inf"), 3.4028234663852886e38, 2.0 ** 127, 2.0 ** 126, 2.0 ** -126, 1e-38, 1e-40,
                                   2.0 ** -149, float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_extreme_repetition(dtype, value):
    """Penalties whose reciprocal is not a normal number: x / r all the same, as x r."""
    x, a = make(2, 100, dtype, 100, 0, False, 14, penalties=("repetition",))
    x = x.contiguous()
    x[0, :12] = torch.tensor([1e-30, 1e-38, 1e-41, 1.0, 3e38, -1e-30, -1e-38, -3e38, 2.0 ** -126, 2.0 ** 127, 1.7e38, 0.0],
                             device=x.device).to(dtype)
    if value == float("inf"):
        x[0, 11] = 1.0                                     # (0 * inf is a NaN)
    a["history"][:] = torch.arange(100, device=x.device)
    a["history_len"][:] = 100
    a["repetition"][:] = value
    out, st = run(x, a)
    assert st == 0
    check(out, x, a)


def test_the_longest_row():
    """2^31 - 17 logits: ids, biases and the mask's last words at both ends and in the middle, in place and out of it."""
    vocab, d = (1 << 31) - 17, device()
    x = torch.ones((1, vocab), dtype=torch.bfloat16, device=d)
    at = torch.tensor([0, vocab // 2, vocab - 1], device=d)
    mask = torch.full(((vocab + 31) // 32,), -1, dtype=torch.int32, device=d)
    mask[(vocab - 2) // 32] &= ~(1 << (vocab - 2) % 32)
    a = {"history": at[None].contiguous(), "frequency": torch.full((1,), 0.5, device=d), "bias_idx": at[1:] - 1,
         "bias": torch.tensor([2.0, 4.0], device=d), "mask": mask}
    for got in (None, x):
        got, st = run(x, a, out=got)
        assert st == 0
        assert got[0, at].tolist() == [0.5, 0.5, 0.5] and float(got[0, vocab // 2 - 1]) == 3.0
        assert float(got[0, vocab - 2]) == -float("inf")
        got[0, at] = 1.0
        got[0, at[1:] - 1] = 1.0
        assert bool((got == 1.0).all())
