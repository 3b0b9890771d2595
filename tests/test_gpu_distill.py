"""e8q_distill, its gradient, and both in one call, against float64.

Bounds, u = 2^-23.  An exponent (x - m) k is off by at most 2^-22 of itself, its
term weighs p |log2 p| <= log2 V in a sum, exp2 and log2 add a few units in the last place and a
thread adds at most V / 64 terms one after another: a log-sum is off by
b = u (16 + 4 log2 V + V / 64).  log q = (x - m) scale - ln s: off by t = b + 2 u |log q|
+ u log V.  The weights: exp is good to 2 u, their sum over k places to n u, n = 8 + k / 64;
the rest's weight so to e = n u max(1, sum p).
loss: each term w (log w - log q) is off by w (t + n u (|l| + |log q| + 2)), the rest's
by w_r (2 b + 4 u |log q_r|) + e (|log max(w_r, e)| + |log q_r| + 2).
Gradient: relative 4 u for the factors, t in every q (log q_r in place of log q for the
rest's: its own bound 2 b + 4 u |log q_r|), e in w_r; one rounding to the type."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
TAIL = {"none": e8q.TAIL_NONE, "renorm": e8q.TAIL_RENORM, "rest": e8q.TAIL_REST}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(rows, vocab, dtype, k, seed, pad=0, index=torch.int64, full=1.0):
    """Logits on the device, places and log probabilities (a teacher near the student; sum p < full)."""
    g = torch.Generator(device=device()).manual_seed(seed)
    x = (torch.randn((rows, vocab + pad), generator=g, device=device()) * 2).to(dtype)[:, :vocab]
    idx = torch.argsort(torch.rand((rows, min(vocab, 4 * k)), generator=g, device=device()), dim=1)[:, :k]
    idx = (idx * max(1, vocab // min(vocab, 4 * k))).contiguous()
    z = torch.gather(x.float(), 1, idx) + torch.randn((rows, k), generator=g, device=device())
    rest = full * (0.02 + 0.5 * torch.rand((rows, 1), generator=g, device=device()))
    lp = torch.log_softmax(z, dim=1) + torch.log1p(-rest)
    w = torch.rand(rows, generator=g, device=device()) + 0.5
    return x, idx.to(index), lp, w


def calls(x, idx, lp, tail, scale, w, stream=None):
    """All three entry points: forward and backward outputs, and the one-call form's."""
    d, (rows, vocab), k = x.device, x.shape, idx.shape[1]
    new = lambda *s: torch.full(s, 7.0, device=d)  # noqa: E731
    ws = torch.full((e8q.e8q_distill_workspace_size(rows, vocab, k),), 0xFF, dtype=torch.uint8, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    o = {"loss": new(rows), "logprob": new(rows, k), "stats": new(rows, 4), "grad": torch.full_like(x, 7.0),
         "loss1": new(rows), "logprob1": new(rows, k), "grad1": torch.full_like(x, 7.0)}
    t = TAIL[tail]
    e8q.e8q_distill(x, idx, lp, ws, st, scale=scale, tail=t, loss_out=o["loss"], logprob_out=o["logprob"],
                    stats_out=o["stats"], stream=stream)
    e8q.e8q_distill_backward(x, idx, lp, o["stats"], w, o["grad"], st, scale=scale, tail=t, stream=stream)
    e8q.e8q_distill_grad(x, idx, lp, w, o["grad1"], ws, st, scale=scale, tail=t, loss_out=o["loss1"],
                         logprob_out=o["logprob1"], stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    fin = np.isfinite(want)
    off, tol = np.abs(got[fin] - want[fin]), np.broadcast_to(tol, want.shape)[fin]
    assert (off <= tol).all(), (what, off.max(), (off / np.maximum(tol, 1e-300)).max())


def check(o, x, idx, lp, tail, scale, w, rows=None):
    """The outputs of these rows (all) against the oracle."""
    sel = np.arange(x.shape[0]) if rows is None else np.asarray(rows)
    f64 = lambda t: t.detach()[torch.from_numpy(sel).to(t.device)].float().cpu().numpy().astype(np.float64)  # noqa: E731
    xs, ls, gs = f64(x), f64(lp), f64(w)
    ids = idx[torch.from_numpy(sel).to(idx.device)].cpu().numpy()
    vocab, k = x.shape[1], idx.shape[1]
    ref = oracle.distill(xs, float(np.float32(scale)), ids, ls, tail, gs)
    with np.errstate(all="ignore"):
        fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0.0)  # noqa: E731
        b = U * (16 + 4 * np.log2(max(vocab, 2)) + vocab / 64)
        n = 8 + k / 64
        t_at = lambda lq: b + 2 * U * fin(lq) + U * np.log(max(vocab, 2))  # noqa: E731
        live = (ids >= 0) & (ids < vocab)
        p = np.where(live, np.exp(ls), 0.0)
        e = (n * U * np.maximum(1.0, p.sum(axis=1)) if tail == "rest" else np.zeros(len(sel)))
        t_rest = 2 * b + 4 * U * fin(ref["log_rest"])
        tol_loss = (ref["w"] * (t_at(ref["logprob"]) + n * U * (fin(ls) + fin(ref["logprob"]) + 2))).sum(axis=1)
        log_w = np.abs(np.log(np.maximum(np.maximum(ref["w_rest"], e), 1e-300)))
        tol_loss += ref["w_rest"] * t_rest + e * (np.where(e > 0, log_w, 0.0) + fin(ref["log_rest"]) + 2)
        lq = ref["log_q"]
        named = np.zeros(lq.shape, bool)
        for r in range(len(sel)):
            named[r, ids[r][live[r]]] = True
        total = (ref["w"].sum(axis=1) + ref["w_rest"])[:, None]
        at = np.zeros(lq.shape)
        for r in range(len(sel)):
            np.add.at(at[r], ids[r][live[r]], ref["w"][r][live[r]])
        q = np.exp(lq)
        tol_in = total * q * (t_at(lq) + 4 * U) + q * e[:, None] + at * (n + 4) * U
        r_i = ref["share"]
        q_r = np.exp(ref["log_rest"])[:, None]
        coef = np.abs(total * q_r - ref["w_rest"][:, None])
        tol_out = r_i * (coef * (b + 2 * U * (fin(lq) + fin(ref["log_rest"])[:, None]) + 8 * U) +
                         total * q_r * t_rest[:, None] + e[:, None] * (1 + q_r) + 4 * U * ref["w_rest"][:, None])
        tol_plain = total * q * (t_at(lq) + (n + 8) * U)
        has = (ref["w_rest"] > 0)[:, None]
        tol = np.where(named, tol_in, np.where(has, tol_out, tol_plain + (r_i * e[:, None] if tail == "rest" else 0.0)))
        tol = tol * np.abs(gs)[:, None] * scale + np.abs(ref["grad"]) * (HALF[x.dtype] + 4 * U) + 1e-37
    for form in ("", "1"):
        close(f64(o["loss" + form]), ref["loss"], tol_loss + 1e-37, "loss" + form)
        close(f64(o["logprob" + form]), ref["logprob"], t_at(ref["logprob"]), "logprob" + form)
        close(f64(o["grad" + form]), ref["grad"], tol, "grad" + form)
    return ref


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("rows,vocab,dtype,k,pad,index,scale", [
    (1, 1, torch.float32, 1, 0, torch.int64, 1.0),
    (3, 2, torch.bfloat16, 1, 1, torch.int32, 1.0),
    (2, 7, torch.float32, 7, 0, torch.int32, 0.5),           # all tokens named
    (5, 100, torch.bfloat16, 9, 3, torch.int64, 2.0),
    (9, 1024, torch.float32, 64, 0, torch.int32, 1.0),       # one block of 64, whole vectors
    (4, 2047, torch.float32, 65, 5, torch.int64, 0.7),
    (4, 4100, torch.bfloat16, 130, 0, torch.int64, 1.0),
    (3, 8191, torch.bfloat16, 1024, 1, torch.int32, 1.0),
    (1, 40001, torch.bfloat16, 20, 0, torch.int32, 1.25),    # split rows
    (5, 33000, torch.float32, 16, 11, torch.int64, 0.5),
    (48, 50001, torch.float32, 20, 175, torch.int32, 1.0),
])
def test_sizes(rows, vocab, dtype, k, pad, index, scale, tail):
    x, idx, lp, w = make(rows, vocab, dtype, k, 11 * rows + vocab, pad, index)
    o, st = calls(x, idx, lp, tail, scale, w)
    assert st == 0
    check(o, x, idx, lp, tail, scale, w)


@pytest.mark.parametrize("vocab,dtype,tail", [
    (9001, torch.bfloat16, "rest"), (16384, torch.bfloat16, "none"), (30001, torch.bfloat16, "rest"),
    (40000, torch.bfloat16, "renorm"), (5000, torch.float32, "rest"), (16000, torch.float32, "renorm"),
    (20001, torch.float32, "rest"), (36001, torch.float32, "rest"), (140001, torch.float32, "rest")])
def test_whole_rows(vocab, dtype, tail):
    """One block a row: each kernel that keeps a row, the one that reads it twice, and rows whose marks come in
    several parts."""
    rows = 1024
    x, idx, lp, w = make(rows, vocab, dtype, 24, vocab, 1)
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == 0
    check(o, x, idx, lp, tail, 1.0, w, rows=[0, 1, 511, 777, 1023])
    # in place, in both forms
    t = TAIL[tail]
    status = torch.zeros(1, dtype=torch.int32, device=x.device)
    ws = torch.empty(e8q.e8q_distill_workspace_size(rows, vocab, 24), dtype=torch.uint8, device=x.device)
    y = x.clone()
    e8q.e8q_distill_grad(y, idx, lp, w, y, ws, status, tail=t)
    assert torch.equal(y, o["grad1"])
    y = x.clone()
    e8q.e8q_distill_backward(y, idx, lp, o["stats"], w, y, status, tail=t)
    assert torch.equal(y, o["grad"])


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("rows,vocab", [(6, 300), (6, 30000), (1100, 9000)])
def test_odd_places(rows, vocab, tail):
    """Unused places, tokens named twice, p = 0, no used place, ids past the vocabulary, banned and emptied rows, the
    type's lowest value."""
    k = 12
    x, idx, lp, w = make(rows, vocab, torch.float32, k, 5)
    x = x.contiguous()
    idx[0, 4:] = -1
    idx[1, 3] = idx[1, 2]
    idx[1, 5] = idx[1, 2]
    lp[2, 1:4] = -float("inf")
    idx[3] = -1
    x[3, 5] = float("nan")                                   # a padded position may hold anything
    x[4, :] = -float("inf")
    x[5, :] = -3.4028234663852886e38
    x[5, idx[5, 0]] = 1.0
    idx[0, 6] = vocab
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == e8q.STATUS_BITS["BAD_INDEX"]
    check(o, x, idx, lp, tail, 1.0, w, rows=range(6))
    assert float(o["loss"][3]) == 0.0 and not o["grad"][3].any() and not o["grad1"][3].any()
    assert float(o["loss"][4]) == float("inf") and not o["grad"][4].any() and not o["grad1"][4].any()
    if tail == "rest":
        # everything outside K banned: the rest has no term
        x[2] = -float("inf")
        x[2].scatter_(0, idx[2].long(), 1.0)
        o, _ = calls(x, idx, lp, tail, 1.0, w)
        check(o, x, idx, lp, tail, 1.0, w, rows=[2])
        assert torch.isfinite(o["loss"][2])


@pytest.mark.parametrize("rows,vocab", [(3, 500), (3, 20000)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite(rows, vocab, value):
    for where in ("named", "other", "teacher"):
        x, idx, lp, w = make(rows, vocab, torch.bfloat16, 8, 9)
        x = x.contiguous()
        if where == "teacher":
            lp[1, 3] = value
        else:
            x[1, idx[1, 2] if where == "named" else (set(range(20)) - set(idx[1].tolist())).pop()] = value
        o, st = calls(x, idx, lp, "rest", 1.0, w)
        assert st == e8q.STATUS_BITS["NONFINITE"], where
        assert torch.isnan(o["loss"][1]) and torch.isnan(o["grad"][1]).any() and torch.isnan(o["grad1"][1]).any()
        if where != "teacher":
            assert torch.isnan(o["grad"][1]).all() and torch.isnan(o["grad1"][1]).all()
        check({n: t[[0, 2]] for n, t in o.items()}, x[[0, 2]], idx[[0, 2]], lp[[0, 2]], "rest", 1.0, w[[0, 2]])


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
def test_gradient_against_differences(tail):
    """Central differences of the oracle's loss (float64, step 1e-5: error about 1e-9) against the gradient."""
    x, idx, lp, w = make(2, 40, torch.float32, 5, 3)
    o, _ = calls(x, idx, lp, tail, 0.7, w)
    xs, ids, ls = x.cpu().numpy().astype(np.float64), idx.cpu().numpy(), lp.cpu().numpy()
    s = float(np.float32(0.7))
    for j in range(40):
        up, down = xs.copy(), xs.copy()
        up[:, j] += 1e-5
        down[:, j] -= 1e-5
        d = (oracle.distill(up, s, ids, ls, tail)["loss"] - oracle.distill(down, s, ids, ls, tail)["loss"]) / 2e-5
        assert np.abs(d * w.cpu().numpy() - o["grad"][:, j].cpu().numpy()).max() < 1e-5


def test_confident_student_keeps_the_rest():
    """The student gives K all but 1e-12 of its mass: q_r does not come out of 1 - sum."""
    x, idx, lp, w = make(3, 5000, torch.float32, 6, 2)
    x = x.contiguous()
    x.scatter_(1, idx, torch.gather(x, 1, idx) + 40.0)
    o, _ = calls(x, idx, lp, "rest", 1.0, w)
    ref = check(o, x, idx, lp, "rest", 1.0, w)
    assert (ref["log_rest"] < -20).all()


def test_the_same_for_any_stream_and_run():
    x, idx, lp, w = make(7, 30011, torch.bfloat16, 40, 8, pad=3)
    first, _ = calls(x, idx, lp, "rest", 1.0, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again, _ = calls(x, idx, lp, "rest", 1.0, w, stream=side)
        for n in first:
            assert torch.equal(first[n], again[n]), n


@pytest.mark.parametrize("tail", ["renorm", "rest"])
@pytest.mark.parametrize("rows,vocab,dtype", [(3, 600, torch.float32), (2, 30000, torch.bfloat16),
                                              (1100, 5000, torch.bfloat16), (1100, 70000, torch.bfloat16)])
def test_places_that_share_tokens(rows, vocab, dtype, tail):
    """300 places for 40 tokens, the first and the last of the vocabulary among them."""
    x, idx, lp, w = make(rows, vocab, dtype, 300 if vocab >= 1200 else 150, rows + vocab)
    idx = idx % 40 * (vocab // 40)
    idx[:, 7] = idx[:, 50] = vocab - 1
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == 0
    check(o, x, idx, lp, tail, 1.0, w, rows=None if rows < 10 else [0, 500, rows - 1])


@pytest.mark.parametrize("rows,vocab", [(5, 9000), (1100, 9000), (1030, 40000)])
def test_gradient_over_the_logits(rows, vocab):
    """The gradient may take the logits' place."""
    x, idx, lp, w = make(rows, vocab, torch.bfloat16, 20, 12, pad=4)
    o, _ = calls(x, idx, lp, "rest", 1.0, w)
    ws = torch.zeros(e8q.e8q_distill_workspace_size(rows, vocab, 20), dtype=torch.uint8, device=x.device)
    st = torch.zeros(1, dtype=torch.int32, device=x.device)
    y = x.clone()
    e8q.e8q_distill_grad(y, idx, lp, w, y, ws, st, tail=e8q.TAIL_REST)
    assert torch.equal(y, o["grad1"])
    y = x.clone()
    e8q.e8q_distill_backward(y, idx, lp, o["stats"], w, y, st, tail=e8q.TAIL_REST)
    assert torch.equal(y, o["grad"]) and int(st.item()) == 0


@pytest.mark.parametrize("vocab", [900, 300001])
def test_offsets_past_32_bits(vocab):
    """Rows of logits and gradients that start past 2^32 elements."""
    x, idx, lp, w = make(3, vocab, torch.bfloat16, 9, 21)
    stride = (1 << 31) + 24
    far = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device=x.device).as_strided((3, vocab), (stride, 1))
    far.copy_(x)
    want, _ = calls(x, idx, lp, "rest", 1.0, w)
    got = {}
    st = torch.zeros(1, dtype=torch.int32, device=x.device)
    ws = torch.zeros(e8q.e8q_distill_workspace_size(3, vocab, 9), dtype=torch.uint8, device=x.device)
    got["loss"], got["stats"] = torch.zeros(3, device=x.device), torch.zeros((3, 4), device=x.device)
    e8q.e8q_distill(far, idx, lp, ws, st, tail=TAIL["rest"], loss_out=got["loss"], stats_out=got["stats"])
    e8q.e8q_distill_grad(far, idx, lp, w, far, ws, st, tail=TAIL["rest"])
    torch.cuda.synchronize()
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(far.contiguous(), want["grad1"])
    far.copy_(x)
    e8q.e8q_distill_backward(far, idx, lp, got["stats"], w, far, st, tail=TAIL["rest"])
    torch.cuda.synchronize()
    assert torch.equal(far.contiguous(), want["grad"]) and int(st.item()) == 0


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("rows,vocab,dtype,k", [(1, 131072, torch.bfloat16, 20), (3, 40001, torch.float32, 200),
                                                (7, 70001, torch.bfloat16, 1), (300, 33001, torch.float32, 16),
                                                (1, 600001, torch.float32, 64)])
def test_few_long_rows(rows, vocab, dtype, k, tail):
    """Rows that are split over blocks and joined, and the gradient from the stored statistics."""
    x, idx, lp, w = make(rows, vocab, dtype, k, rows + vocab, pad=rows % 2)
    idx[:, -1] = vocab - 1
    if k > 4:
        idx[0, 1] = idx[0, 0]
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == 0
    check(o, x, idx, lp, tail, 1.0, w, rows=None if rows < 10 else [0, 7, rows - 1])


def test_graph_of_split_rows():
    """Few long rows in a graph, replayed with other inputs and eager calls between."""
    x, idx, lp, w = make(4, 90001, torch.bfloat16, 12, 3)
    x = x.contiguous()
    ws = torch.zeros(e8q.e8q_distill_workspace_size(4, 90001, 12), dtype=torch.uint8, device=x.device)
    st = torch.zeros(1, dtype=torch.int32, device=x.device)
    outs = [torch.zeros(4, device=x.device), torch.zeros((4, 4), device=x.device), torch.zeros_like(x), torch.zeros_like(x)]

    def work(loss, stats, grad, both):
        e8q.e8q_distill(x, idx, lp, ws, st, tail=e8q.TAIL_REST, loss_out=loss, stats_out=stats)
        e8q.e8q_distill_backward(x, idx, lp, stats, w, grad, st, tail=e8q.TAIL_REST)
        e8q.e8q_distill_grad(x, idx, lp, w, both, ws, st, tail=e8q.TAIL_REST)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(*outs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(*outs)
    for seed in (1, 2, 3):
        x.normal_(generator=torch.Generator(device=x.device).manual_seed(seed))
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.zeros_like(t) for t in outs]
        work(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)) and int(st.item()) == 0


@pytest.mark.parametrize("rows,vocab", [(8, 300), (8, 30000), (1100, 9000), (1030, 40000)])
def test_renorm_of_far_log_probabilities(rows, vocab):
    """A shift of a row's log probabilities leaves p / sum p as it is: sums below float32's least number and above its largest
    are no limit.  Weights too small beside the row's largest are 0."""
    x, idx, lp, w = make(rows, vocab, torch.float32, 12, 31)
    for row, shift in enumerate((-90.0, -101.0, -120.0, -5000.0, 95.0, 300.0, -700.0)):
        lp[row] += shift
    lp[6, 3:] -= 200.0
    lp[7, :4] = -float("inf")
    lp[7, 4:] -= 95.0
    idx[5, 4:] = -1
    lp[5, 4:] = 1000.0                                       # (places that are not used)
    o, st = calls(x, idx, lp, "renorm", 1.0, w)
    assert st == 0
    shifted = lp.clone()
    shifted[3] += 5000.0                                     # (exact; the float64 oracle's exp(-5000) is 0)
    ref = check(o, x, idx, shifted, "renorm", 1.0, w, rows=range(8))
    assert (ref["loss"] > 0).all() and (np.abs(ref["w"].sum(axis=1) - 1) < 1e-12).all()


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("rows,vocab", [(4, 300), (4, 30000), (1100, 9000), (1030, 40000)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_logits_where_no_place_weighs(rows, vocab, value, tail):
    """NaN outputs where a logit is a NaN or infinite, though all places have p = 0; loss 0 where the logits are finite."""
    x, idx, lp, w = make(rows, vocab, torch.float32, 8, 9)
    x = x.contiguous()
    lp[:3] = -float("inf")
    x[0, idx[0, 2]] = value
    x[1, (set(range(20)) - set(idx[1].tolist())).pop()] = value
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == e8q.STATUS_BITS["NONFINITE"]
    for n in ("loss", "loss1", "logprob", "logprob1", "grad", "grad1"):
        assert torch.isnan(o[n][:2]).all(), n
    check(o, x, idx, lp, tail, 1.0, w, rows=[2, 3])
    if tail != "rest":
        assert float(o["loss"][2]) == 0.0 and not o["grad"][2].any()


@pytest.mark.parametrize("tail", ["none", "renorm", "rest"])
@pytest.mark.parametrize("rows,vocab", [(6, 300), (6, 30000), (1100, 9000), (1030, 40000)])
def test_non_finite_rows_without_another_token(rows, vocab, tail):
    """All tokens that no place names are -inf: a NaN or an infinity among the named ones, or a teacher's, reaches the
    gradient of every token all the same."""
    x, idx, lp, w = make(rows, vocab, torch.float32, 8, 10)
    x = x.contiguous()
    named = torch.gather(x, 1, idx)
    x[:5] = -float("inf")
    x[:5] = x[:5].scatter(1, idx[:5], named[:5])
    x[0, idx[0, 1]] = float("nan")
    x[1, idx[1, 1]] = float("inf")
    lp[2, 3] = float("nan")
    lp[3, 3] = float("inf")
    o, st = calls(x, idx, lp, tail, 1.0, w)
    assert st == e8q.STATUS_BITS["NONFINITE"]
    for n in ("loss", "loss1", "grad", "grad1"):
        assert torch.isnan(o[n][:4]).all(), n
    check(o, x, idx, lp, tail, 1.0, w, rows=[4, 5])


def parts(rows, vocab, dtype):
    """Elements of a block's part of a row, where few rows are split (as the host side splits them)."""
    ve = 8 if dtype == torch.bfloat16 else 4
    vectors = -(-vocab // ve)
    n = max(1, min(-(-torch.cuda.get_device_properties(0).multi_processor_count * 4 // rows), -(-vectors // 1024), 256))
    return -(-vectors // n) * ve


@pytest.mark.parametrize("tail", ["none", "rest"])
@pytest.mark.parametrize("rows,vocab,dtype", [
    (1, 131071, torch.bfloat16), (3, 300001, torch.float32), (40, 50003, torch.float32),     # split
    (1100, 70003, torch.bfloat16), (1100, 140005, torch.float32),                            # two passes, two segments of marks
    (1030, 263007, torch.bfloat16),
    (7, 2043, torch.bfloat16), (1100, 9001, torch.bfloat16), (5, 16381, torch.float32)])     # in registers
def test_no_element_is_left_out(rows, vocab, dtype, tail):
    """A logit far above all others, that no place names, at the row's ends and at the borders of vectors, parts and segments: without
    it the loss would be 40 less."""
    x, idx, lp, w = make(rows, vocab, dtype, 6, vocab)
    x, ve = x.contiguous(), 8 if dtype == torch.bfloat16 else 4
    part = parts(rows, vocab, dtype)
    at = {0, 1, ve, vocab - 1, vocab - 2, vocab - vocab % ve, vocab - vocab % ve - 1, 32768 * ve - 1, 32768 * ve, 32768 * ve + 1}
    for p in range(part, vocab, max(part, part * (vocab // part // 6))):
        at |= {p - 1, p}
    for block in (64, 128, 256, 1024):
        at |= {block * ve - 1, block * ve, 4 * block * ve - 1, 4 * block * ve}
    at = sorted(p for p in at if 0 <= p < vocab)
    base = x.clone()
    for i in range(0, len(at), rows):
        x.copy_(base)
        here = at[i:i + rows]
        for r, p in enumerate(here):
            idx[r][idx[r] == p] = -1
            x[r, p] = float(base[r].float().max()) + 40.0
        o, st = calls(x, idx, lp, tail, 1.0, w)
        assert st == 0
        ref = check(o, x, idx, lp, tail, 1.0, w, rows=range(len(here)))
        live = (idx[:len(ref["loss"])] >= 0).cpu().numpy()
        assert (ref["logprob"][live] < -38).all()


@pytest.mark.parametrize("rows,vocab,dtype", [(1, 131072, torch.bfloat16), (2, 600001, torch.float32), (1100, 40001, torch.bfloat16),
                                              (1100, 30001, torch.float32), (1030, 140001, torch.float32)])
def test_log_probabilities_of_long_rows(rows, vocab, dtype):
    """log q within what a thread really adds one after the other: pairs of vectors, of which a block of 256 threads or more has
    V / (512 VE) a thread, each pair's elements in two chains; then the lanes, waves and parts (at most 256 of them).
    b = u (16 + 4 log2 V + V / (512 VE) + VE): below a left-out vector's share of the sum, but for the longest row."""
    x, idx, lp, w = make(rows, vocab, dtype, 16, 5)
    o, st = calls(x, idx, lp, "none", 1.0, w)
    assert st == 0
    sel = sorted({0, rows // 2, rows - 1})
    ref = oracle.distill(x[sel].float().cpu().numpy(), 1.0, idx[sel].cpu().numpy(), lp[sel].cpu().numpy(), "none")
    ve = 8 if dtype == torch.bfloat16 else 4
    b = U * (16 + 4 * np.log2(vocab) + vocab / (512 * ve) + ve)
    assert b < ve / vocab or vocab > 200000
    tol = b + 2 * U * np.abs(ref["logprob"]) + U * np.log(vocab)
    for form in ("", "1"):
        off = np.abs(o["logprob" + form][sel].cpu().numpy() - ref["logprob"])
        assert (off <= tol).all(), (off.max(), tol.min())


def test_the_longest_row():
    """2^31 - 17 logits, all 0 but the last one: sums of ones, which float32 adds without loss up to 2^24 in a thread, then join by
    rounding to 2^-24 each: eight lane and part levels, 16 u of the sum."""
    vocab = (1 << 31) - 17
    x = torch.zeros((1, vocab), dtype=torch.bfloat16, device=device())
    x[0, -1] = 20.0
    idx = torch.tensor([[0, vocab // 2, vocab - 2]], device=x.device)
    lp = torch.log(torch.tensor([[0.25, 0.5, 0.125]], device=x.device))
    w = torch.full((1,), 2.0 ** 20, device=x.device)
    o, st = calls(x, idx, lp, "rest", 1.0, w)
    assert st == 0
    total, p = vocab - 1 + np.exp(20.0), np.exp(lp.cpu().numpy().astype(np.float64))[0]
    lse, rest, w_rest = np.log(total), (total - 3) / total, 1 - p.sum()
    loss = (p * (np.log(p) + lse)).sum() + w_rest * (np.log(w_rest) - np.log(rest))
    plain, last = (1 - w_rest / rest) / total * 2.0 ** 20, (1 - w_rest / rest) * np.exp(20.0) / total * 2.0 ** 20
    for form in ("", "1"):
        assert abs(float(o["loss" + form][0]) - loss) < 64 * U * (lse + 1)
        assert np.abs(o["logprob" + form][0].cpu().numpy() + lse).max() < 32 * U * lse
        g = o["grad" + form][0]
        named = (1 / total - p) * 2.0 ** 20
        assert np.abs(g[idx[0]].float().cpu().numpy() - named).max() < 2.0 ** -8 * np.abs(named).max()
        assert abs(float(g[-1]) - last) < 1.01 * 2.0 ** -8 * last
        g[idx[0]] = g[1].clone()
        g[-1] = g[1]
        assert abs(float(g[1]) - plain) < 1.01 * 2.0 ** -8 * plain and bool((g == g[1]).all())
