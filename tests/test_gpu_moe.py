"""e8q_moe_core_escape against float64, within the bounds of oracle/moe.py."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device
from moe_cases import Layer

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


def inputs(layer, tokens, x_dtype, router_dtype, seed):
    e, h, _ = layer.shape
    g = torch.Generator(device=layer.device).manual_seed(seed)
    x = torch.randn((tokens, h), generator=g, device=layer.device)
    x[:, torch.randint(0, h, (max(1, h // 100),), generator=g, device=layer.device)] *= 20.0
    router = torch.randn((e, h), generator=g, device=layer.device) / h ** 0.5
    return x.to(x_dtype), router.to(router_dtype)


def close(y, want, tol):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = tol + HALF[y.dtype] * np.abs(want) * (1 + 2.0 ** -10) + 1e-30
    off = np.abs(got - want)
    assert (off <= tol).all(), (off.max(), (off / tol).max())


def check(layer, tokens, k, seed, normalize=True, act="silu", x_dtype=torch.bfloat16, router_dtype=torch.bfloat16,
          y_dtype=torch.float32):
    x, router = inputs(layer, tokens, x_dtype, router_dtype, seed)
    y, idx, weight, st = layer.run(x, k, router, normalize, act, y_dtype)
    assert st == 0
    want_idx, want_w = oracle.moe_route(x.float().cpu().numpy(), router.float().cpu().numpy(), k, normalize)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    assert np.abs(weight.cpu().numpy() - want_w).max() <= 40 * U
    want, tol = layer.expect(x, want_idx, want_w, act)
    close(y, want, tol)
    return x, router, y, idx, weight


@pytest.mark.parametrize("experts,hidden,inter,bound,alpha,had_in,had_down,k,act", [
    (2, 8, 8, 8, 3.0, 8, 8, 1, "silu"),
    (1, 64, 24, 16, 3.0, 0, 0, 1, "gelu_tanh"),
    (9, 520, 328, 24, 2.5, 8, 8, 2, "gelu_tanh"),
    (5, 768, 256, 8, 1.0, 128, 64, 3, "silu"),              # most groups escape
    (70, 256, 128, 16, 3.0, 32, 16, 8, "silu"),             # more than a wave of experts
    (4, 2560, 144, 16, 2.0, 512, 16, 2, "silu"),            # digits in two parts
    (3, 4096, 1024, 40, 3.0, 4096, 1024, 2, "silu"),        # wide rotations; the table in memory
    (2, 8200, 72, 32, 2.0, 8, 0, 1, "silu"),                # more than 8192 columns
    (2, 40, 8200, 16, 2.0, 8, 8, 2, "silu"),
])
@pytest.mark.parametrize("tokens", [1, 6, 23])
def test_sizes(experts, hidden, inter, bound, alpha, had_in, had_down, k, act, tokens):
    layer = Layer(experts, hidden, inter, bound, alpha, had_in, had_down, experts + hidden, device())
    check(layer, tokens, k, tokens, normalize=tokens != 6, act=act, x_dtype=torch.float32 if tokens == 6 else torch.bfloat16,
          router_dtype=torch.float32 if tokens == 23 else torch.bfloat16,
          y_dtype=torch.bfloat16 if tokens == 23 else torch.float32)


def test_expert_workload():
    """The gate, up and down sizes of the expert workload."""
    layer = Layer(8, 2048, 768, 16, 3.0, 128, 128, 5, device())
    for tokens in (1, 2, 16):
        check(layer, tokens, 4, tokens, y_dtype=torch.bfloat16)


def test_many_tokens():
    layer = Layer(3, 128, 64, 16, 3.0, 128, 64, 5, device())
    check(layer, 700, 2, 1)
    check(layer, 1365, 3, 2)


def test_wide_escapes():
    """Escaped points of more than eight bits, beside ordinary ones."""
    layer = Layer(3, 256, 160, 16, 3.0, 32, 32, 8, device(), outliers=400)
    assert all(np.abs(m[0]).max() > 2000 for m in layer.oracle)
    check(layer, 7, 2, 3)


def test_given_places():
    """Routes of the caller: unused places, an expert named twice, ids out of range, a token without a place."""
    layer = Layer(6, 256, 128, 16, 3.0, 128, 128, 9, device())
    x, _ = inputs(layer, 9, torch.float32, torch.float32, 2)
    idx = torch.randint(0, 6, (9, 4), dtype=torch.int32, device=x.device)
    idx[0] = -1
    idx[1] = 3
    idx[2, 1:] = -5
    weight = torch.randn((9, 4), device=x.device)
    keep, keep_w = idx.clone(), weight.clone()
    y, _, _, st = layer.run(x, 4, idx=idx, weight=weight)
    assert st == 0 and torch.equal(idx, keep) and torch.equal(weight, keep_w)
    want, tol = layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy())
    close(y, want, tol)
    assert not y[0].any()
    idx[4, 2] = 6
    y, _, _, st = layer.run(x, 4, idx=idx, weight=weight)
    assert st == e8q.STATUS_BITS["BAD_INDEX"]
    want, tol = layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy())
    close(y, want, tol)


def test_ties_take_the_lowest_index():
    layer = Layer(5, 64, 16, 8, 3.0, 0, 0, 9, device())
    x, router = inputs(layer, 3, torch.float32, torch.float32, 2)
    router[3] = router[1]
    router[4] = router[1]
    x[2] = 0                                               # every logit 0
    y, idx, weight, st = layer.run(x, 4, router)
    want_idx, want_w = oracle.moe_route(x.cpu().numpy(), router.cpu().numpy(), 4, True)
    assert st == 0 and np.array_equal(idx.cpu().numpy(), want_idx) and not y[2].any()
    assert idx[2].tolist() == [0, 1, 2, 3]


def test_malformed_data():
    """Non-finite tokens, bad scales, indices past the core, missing and impossible records."""
    layer = Layer(4, 256, 64, 16, 1.5, 128, 64, 10, device())
    x, router = inputs(layer, 5, torch.float32, torch.float32, 3)
    clean, idx, weight, _ = layer.run(x, 2, router)
    bad = x.clone()
    bad[1, 3] = float("nan")
    bad[3, 5] = float("inf")
    y, idx2, _, st = layer.run(bad, 2, router)
    assert st == e8q.STATUS_BITS["NONFINITE"]
    assert torch.isnan(y[[1, 3]]).all() and torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
    assert ((idx2 >= 0) & (idx2 < 4)).all()
    # a scale that is no positive number: the row is 0
    core, esc, cnt, scale = layer.down.tensors
    keep = scale.clone()
    scale[int(idx[0, 0]) * 256 + 7] = float("nan")
    scale[int(idx[0, 0]) * 256 + 9] = -1.0
    layer.oracle[2] = (layer.oracle[2][0], scale.cpu().numpy().reshape(4, 256))
    y, _, _, st = layer.run(x, 2, router)
    assert st == e8q.STATUS_BITS["BAD_SCALE"]
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))
    scale.copy_(keep)
    layer.oracle[2] = (layer.oracle[2][0], scale.cpu().numpy().reshape(4, 256))
    # an index past the core and an escaped slot without its record decode to 0; so does an impossible record
    used = int(idx[0, 0])
    groups = 256 * 64 // 8
    slots = core.view(4, groups)
    z = layer.oracle[2][0].reshape(4, groups, 8)
    plain = (slots[used] != -1).nonzero()[:2, 0].tolist()
    keep = core.clone()
    for value, flag in ((oracle.core_size(16), "BAD_INDEX"), (-1, "ESC_MISSING")):
        slots[used, plain[0]] = value
        was = z[used, plain[0]].copy()
        z[used, plain[0]] = 0
        y, _, _, st = layer.run(x, 2, router)
        assert st == e8q.STATUS_BITS[flag]
        close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))
        z[used, plain[0]] = was
        core.copy_(keep)
    first = int(cnt[:used].sum())
    rec = esc.view(-1, 20)[first].view(torch.int16)
    kept = rec.clone()
    rec[2 + 3] = 32767
    group = int(esc.view(-1, 20)[first].view(torch.int32)[0])
    z[used, group] = 0
    y, _, _, st = layer.run(x, 2, router)
    assert st == e8q.STATUS_BITS["X_RANGE"]
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))
    rec.copy_(kept)


def test_streams_workspaces_and_smaller_batches():
    layer = Layer(7, 512, 96, 16, 3.0, 128, 32, 11, device())
    e, h, f = layer.shape
    ws = torch.zeros(e8q.e8q_moe_workspace_size(e, h, f, 12, 3), dtype=torch.uint8, device=layer.device)
    x, router = inputs(layer, 12, torch.bfloat16, torch.bfloat16, 4)
    first = layer.run(x, 3, router, ws=ws)
    for t in (12, 5, 1):
        for stream in (None, torch.cuda.Stream()):
            y, idx, weight, st = layer.run(x[:t].contiguous(), 3, router, ws=ws, stream=stream)
            assert st == 0 and torch.equal(y, first[0][:t]) and torch.equal(idx, first[1][:t])
            assert torch.equal(weight, first[2][:t])


@pytest.mark.parametrize("experts,tokens,k", [(1024, 900, 4), (300, 40, 7), (40, 64, 8)])
def test_sweeps_of_several_turns(experts, tokens, k):
    """More sweeps than the chip has blocks, and some in between; experts that no token chose, and one that all did."""
    layer = Layer(experts, 64, 48, 16, 3.0, 32, 16, experts, device())
    x, router = inputs(layer, tokens, torch.bfloat16, torch.float32, 7)
    router[5] = x.float().mean(dim=0) * 3 + 0.2 * x[0].float()
    router[6] = 0
    y, idx, weight, st = layer.run(x, k, router)
    want_idx, want_w = oracle.moe_route(x.float().cpu().numpy(), router.cpu().numpy(), k, True)
    assert st == 0 and np.array_equal(idx.cpu().numpy(), want_idx)
    close(y, *layer.expect(x, want_idx, want_w))


@pytest.mark.parametrize("tokens", [1, 3])
def test_given_places_of_few_tokens(tokens):
    """At most 16 places, whose sum is formed with the products: unused ones, one expert twice, ids out of range."""
    layer = Layer(6, 256, 128, 16, 3.0, 128, 128, 9, device())
    x, _ = inputs(layer, tokens, torch.float32, torch.float32, 2)
    idx = torch.tensor([[2, 2, -1, 4], [-7, -1, -2, -3], [5, 0, 0, 0]][:tokens], dtype=torch.int32, device=x.device)
    weight = torch.randn((tokens, 4), device=x.device)
    y, _, _, st = layer.run(x, 4, idx=idx, weight=weight)
    assert st == 0
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))
    idx[0, 3] = 100
    y, _, _, st = layer.run(x, 4, idx=idx, weight=weight)
    assert st == e8q.STATUS_BITS["BAD_INDEX"]
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("tokens,k", [(1, 5), (3, 4), (5, 5), (6, 5), (40, 4)])
def test_router_logits_that_are_no_numbers(tokens, k, normalize):
    """A NaN logit counts as -inf: p = 0, and among equal ones the lowest index first.  Few tokens, whose experts the products'
    blocks choose, and more."""
    layer = Layer(5, 64, 40, 16, 3.0, 32, 8, 12, device())
    x, router = inputs(layer, tokens, torch.float32, torch.float32, 5)
    x[:, 0] = x[:, 0].abs() + 0.5
    router[1, 7] = float("nan")
    router[3, :] = 0
    router[3, 0] = -float("inf")
    router[4, 63] = float("nan")
    y, idx, weight, st = layer.run(x, k, router, normalize)
    assert st == e8q.STATUS_BITS["NONFINITE"]
    want_idx, want_w = oracle.moe_route(x.cpu().numpy(), router.cpu().numpy(), k, normalize)
    assert (want_idx[:, 2:] == [1, 3, 4][:k - 2]).all() and not want_w[:, 2:].any() and np.isfinite(want_w).all()
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    assert np.abs(weight.cpu().numpy() - want_w).max() <= 40 * U
    close(y, *layer.expect(x, want_idx, want_w))


@pytest.mark.parametrize("tokens", [3, 20])
def test_counts_whose_sum_passes_64_bits(tokens):
    """Counts past the records, up to the type's largest: an expert before them is served, those behind have no records."""
    layer = Layer(4, 256, 128, 16, 1.5, 32, 16, 13, device())
    x, _ = inputs(layer, tokens, torch.float32, torch.float32, 6)
    for i, m in enumerate((layer.gate, layer.up, layer.down)):
        core, _, counts, _ = m.tensors
        first = int(counts[0])
        assert first > 2 and int(counts[1:].min()) > 0
        counts[1:3] = 2 ** 63 - 1                          # the second sum is 2 below the first count, modulo 2^64
        escaped = core.view(4, -1).cpu().numpy() == -1
        two_z = layer.oracle[i][0].reshape(4, -1, 8)
        two_z[2:][escaped[2:]] = 0
    idx = torch.tensor([[0, 2], [3, 0], [2, 3]], dtype=torch.int32, device=x.device).repeat(tokens, 1)[:tokens]
    weight = torch.rand((tokens, 2), device=x.device) + 0.5
    y, _, _, st = layer.run(x, 2, idx=idx, weight=weight)
    assert st == e8q.STATUS_BITS["ESC_MISSING"]
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))


def wide_layer(experts, hidden, inter, bound, had_in, had_down):
    layer = Layer(experts, hidden, inter, bound, 3.0, had_in, had_down, 21, device(), outliers=400)
    assert all(np.abs(m[0]).max() > 200 for m in layer.oracle)      # (a wide rotation spreads them)
    return layer


@pytest.mark.parametrize("experts,hidden,inter,bound,had_in,had_down", [
    (3, 256, 160, 16, 32, 32),
    (3, 264, 1040, 24, 8, 16),                              # a table of changing place; down's columns in several chunks
    (2, 2600, 2200, 16, 8, 8),                              # digits of every product in two parts, ready before down
    (2, 600, 2048, 40, 8, 2048),                            # the table in memory
])
@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_wide_escapes_of_all_sweeps(experts, hidden, inter, bound, had_in, had_down, tokens):
    """Escaped points of more than eight bits in gate, up and down: the direct sum, planned sweeps of one and two products, whole
    rows and parts of them."""
    layer = wide_layer(experts, hidden, inter, bound, had_in, had_down)
    check(layer, tokens, 2, tokens)


@pytest.mark.parametrize("hidden,inter", [(2600, 2200), (1104, 1600)])
def test_wide_escapes_of_whole_rounds(hidden, inter):
    """One expert's 1400 tokens in 140 sweeps and more: jobs of full rounds and a shared one behind them."""
    layer = wide_layer(2, hidden, inter, 16, 8, 8)
    x, _ = inputs(layer, 1400, torch.bfloat16, torch.float32, 8)
    idx = torch.zeros((1400, 2), dtype=torch.int32, device=x.device)
    idx[:, 1] = 1
    weight = torch.rand((1400, 2), device=x.device)
    y, _, _, st = layer.run(x, 2, idx=idx, weight=weight)
    assert st == 0
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("tokens", [5, 23])
def test_malformed_matrices(which, tokens):
    """Bad scales and indices, missing and impossible records of gate, up and down in turn; the direct sum and planned sweeps."""
    layer = Layer(4, 256, 64, 16, 1.5, 128, 64, 10, device())
    m = (layer.gate, layer.up, layer.down)[which]
    rows, cols = m.shape[1:]
    x, router = inputs(layer, tokens, torch.float32, torch.float32, 3)
    _, idx, weight, _ = layer.run(x, 2, router)
    used = int(idx[0, 0])
    core, esc, cnt, scale = m.tensors
    two_z = layer.oracle[which][0]
    slots, z = core.view(4, -1), two_z.reshape(4, -1, 8)

    def expect(flag):
        layer.oracle[which] = (two_z, scale.cpu().numpy().reshape(4, rows))
        y, _, _, st = layer.run(x, 2, router)
        assert st == e8q.STATUS_BITS[flag], flag
        close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))

    for value in (float("nan"), -1.0, float("inf"), 0.0):
        keep = scale.clone()
        scale[used * rows + 7] = value
        expect("BAD_SCALE")
        scale.copy_(keep)
    plain = (slots[used] != -1).nonzero()[:, 0].tolist()
    for at in (plain[0], plain[-1]):
        for value, flag in ((oracle.core_size(16), "BAD_INDEX"), (-1, "ESC_MISSING")):
            keep, was = core.clone(), z[used, at].copy()
            slots[used, at] = value
            z[used, at] = 0
            expect(flag)
            z[used, at] = was
            core.copy_(keep)
    first = int(cnt[:used].sum())
    for at in (first, first + int(cnt[used]) - 1):
        rec = esc.view(-1, 20)[at].view(torch.int16)
        group = int(esc.view(-1, 20)[at].view(torch.int32)[0])
        kept, was = rec.clone(), z[used, group].copy()
        for value, flag in ((32767, "X_RANGE"), (-32768, "X_RANGE")):
            rec[2 + 3] = value
            z[used, group] = 0
            expect(flag)
        rec.copy_(kept)
        z[used, group] = was
    # no records from this expert on
    cnt[used:] = 0
    assert (slots[used] == -1).any()
    z[used:][slots[used:].cpu().numpy() == -1] = 0
    expect("ESC_MISSING")


@pytest.mark.parametrize("tokens", [2, 30])
def test_one_channel_far_above_the_others(tokens):
    """Without a rotation, a channel of 10^5 times the others: the step of the fixed point is the largest one's, 2^-23 of it."""
    layer = Layer(4, 256, 96, 16, 3.0, 0, 0, 22, device())
    x, router = inputs(layer, tokens, torch.float32, torch.float32, 9)
    x[:, 17] = 1e5
    idx = (torch.arange(2 * tokens, device=x.device).view(tokens, 2) % 4).to(torch.int32)
    weight = torch.full((tokens, 2), 0.5, device=x.device)
    y, _, _, st = layer.run(x, 2, idx=idx, weight=weight)
    assert st == 0
    close(y, *layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy()))


@pytest.mark.parametrize("hidden,inter,had_in,had_down", [(32768, 64, 0, 8), (64, 32768, 8, 0), (20480, 40, 4096, 8),
                                                          (24, 20480, 8, 4096)])
@pytest.mark.parametrize("tokens", [1, 12])
def test_the_widest_matrices(hidden, inter, had_in, had_down, tokens):
    layer = Layer(2, hidden, inter, 16, 3.0, had_in, had_down, 23, device())
    check(layer, tokens, 2, tokens)
