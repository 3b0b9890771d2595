"""The mixture-of-experts layer, the adjustment of logits and the distillation loss as they are
used together, and in HIP graphs."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
import test_gpu_adjust
import test_gpu_distill
from gpu_util import device
from moe_cases import ACT, Layer

pytestmark = pytest.mark.gpu

VOCAB = 5003


def test_a_teacher_step_and_a_students_loss():
    """A teacher of one exported layer: its logits are adjusted, its top ones taken; a student learns from them.
    Each operator against float64 on what the one before it gave."""
    d, tokens, k = device(), 6, 12
    layer = Layer(9, 256, 128, 16, 3.0, 128, 64, 3, d)
    g = torch.Generator(device=d).manual_seed(4)
    x = torch.randn((tokens, 256), generator=g, device=d)
    router = torch.randn((9, 256), generator=g, device=d) / 16
    head = torch.randn((VOCAB, 256), generator=g, device=d) / 8
    y, idx, weight, st = layer.run(x, 2, router)
    assert st == 0
    want, tol = layer.expect(x, idx.cpu().numpy(), weight.cpu().numpy())
    assert (np.abs(y.cpu().numpy() - want) <= tol + 2.0 ** -24 * np.abs(want)).all()

    logits = (x + y) @ head.T
    _, a = test_gpu_adjust.make(tokens, VOCAB, torch.float32, 40, 5, False, 6)
    banned = torch.randint(0, VOCAB, (400,), generator=g, device=d)
    bits = torch.ones((VOCAB + 31) // 32 * 32, dtype=torch.int64, device=d)
    bits[banned] = 0
    words = (bits.view(-1, 32) << torch.arange(32, device=d)).sum(dim=1)
    a["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    before = logits.clone()
    out, st = test_gpu_adjust.run(logits, a, out=logits)                     # in place
    assert st == 0
    test_gpu_adjust.check(out, before, a)

    status = torch.zeros(1, dtype=torch.int32, device=d)
    top = torch.empty((tokens, k), dtype=torch.int32, device=d)
    lp = torch.empty((tokens, k), device=d)
    ws = torch.empty(e8q.e8q_token_logprobs_workspace_size(tokens, VOCAB, k), dtype=torch.uint8, device=d)
    e8q.e8q_token_logprobs(out, ws, status, top_idx_out=top, top_logprob_out=lp)
    torch.cuda.synchronize()
    assert not torch.isin(top.long(), banned).any()
    best = oracle.logprobs(out.cpu().numpy().astype(np.float64), 1.0, None, top_k=k)
    assert np.array_equal(top.cpu().numpy(), best["top_idx"])

    student = torch.randn((tokens, VOCAB + 5), generator=g, device=d).to(torch.bfloat16)[:, :VOCAB]
    w = torch.full((tokens,), 1 / tokens, device=d)
    for tail in ("none", "renorm", "rest"):
        o, st = test_gpu_distill.calls(student, top, lp, tail, 1.0, w)
        assert st == 0
        test_gpu_distill.check(o, student, top, lp, tail, 1.0, w)


@pytest.mark.parametrize("tokens,k", [(1, 2), (5, 3), (9, 4), (40, 4)])
def test_graph_replays_equal_eager_calls(tokens, k):
    """Two graphs that share their workspaces, replayed in turn with eager work between; one token, an inline choice of
    experts, and planned sweeps."""
    d, places = device(), 7
    layer = Layer(12, 256, 136, 16, 3.0, 128, 8, 5, d)
    e, h, f = layer.shape
    router = torch.randn((e, h), device=d) / 16
    x = torch.empty((tokens, h), dtype=torch.bfloat16, device=d)
    logits, teacher = torch.empty((tokens, VOCAB), device=d), torch.empty((tokens, places), device=d)
    ids = torch.empty((tokens, places), dtype=torch.int64, device=d)
    _, a = test_gpu_adjust.make(tokens, VOCAB, torch.float32, 300, 20, True, 6)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    one = torch.ones(tokens, device=d)
    byte = lambda size: torch.full((max(1, size),), 0xFF, dtype=torch.uint8, device=d)  # noqa: E731
    ws = byte(e8q.e8q_moe_workspace_size(e, h, f, tokens, k)), byte(e8q.e8q_distill_workspace_size(tokens, VOCAB, places))
    outs = [{"idx": torch.empty((tokens, k), dtype=torch.int32, device=d), "weight": torch.empty((tokens, k), device=d),
             "y": torch.empty_like(x), "adjusted": torch.empty_like(logits), "loss": torch.empty(tokens, device=d),
             "stats": torch.empty((tokens, 4), device=d), "grad": torch.empty_like(logits), "both": torch.empty_like(logits)}
            for _ in range(2)]

    def work(o):
        e8q.e8q_moe_core_escape(layer.gate, layer.up, layer.down, layer.bound, x, o["idx"], o["weight"], o["y"], ws[0], status,
                                router=router, signs_in=layer.signs_in, had_block_in=layer.had_in,
                                signs_down=layer.signs_down, had_block_down=layer.had_down, activation=ACT["silu"])
        e8q.e8q_adjust_logits(logits, o["adjusted"], status, **a)
        e8q.e8q_distill(o["adjusted"], ids, teacher, ws[1], status, tail=e8q.TAIL_REST, loss_out=o["loss"],
                        stats_out=o["stats"])
        e8q.e8q_distill_backward(o["adjusted"], ids, teacher, o["stats"], one, o["grad"], status, tail=e8q.TAIL_REST)
        e8q.e8q_distill_grad(logits, ids, teacher, one, o["both"], ws[1], status, tail=e8q.TAIL_RENORM)

    def fill(seed):
        gen = torch.Generator(device=d).manual_seed(seed)
        x.normal_(generator=gen)
        logits.normal_(0.0, 3.0, generator=gen)
        ids.copy_(torch.randint(-1, VOCAB, ids.shape, generator=gen, device=d))
        teacher.uniform_(-6.0, -2.5, generator=gen)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(outs[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            work(o)
    same = lambda p, q: torch.equal(torch.nan_to_num(p.float()), torch.nan_to_num(q.float()))  # noqa: E731
    for seed in (1, 2, 3):
        fill(seed)
        for o in outs:
            for t in o.values():
                t.zero_()
        graphs[seed % 2].replay()
        graphs[1 - seed % 2].replay()
        torch.cuda.synchronize()
        got = [{n: t.clone() for n, t in o.items()} for o in outs]
        eager = {n: torch.zeros_like(t) for n, t in outs[0].items()}
        work(eager)
        torch.cuda.synchronize()
        for o in got:
            for n in o:
                assert same(o[n], eager[n]), (seed, n)
    assert int(status.item()) & ~e8q.STATUS_BITS["NONFINITE"] == 0


@pytest.mark.parametrize("tokens,k", [(1, 2), (5, 3), (6, 4), (33, 4)])
def test_graph_writes_every_output(tokens, k):
    """A graph's outputs bit for bit as the eager calls', over marks of their own: what a call leaves unwritten differs, and so does
    a NaN.  No status bit."""
    d, places = device(), 9
    layer = Layer(10, 256, 136, 16, 3.0, 128, 8, 15, d)
    e, h, f = layer.shape
    gen = torch.Generator(device=d).manual_seed(16)
    router = torch.randn((e, h), generator=gen, device=d) / 16
    x = torch.empty((tokens, h), dtype=torch.bfloat16, device=d)
    logits, teacher = torch.empty((tokens, VOCAB), device=d), torch.empty((tokens, places), device=d)
    ids = torch.empty((tokens, places), dtype=torch.int64, device=d)
    _, a = test_gpu_adjust.make(tokens, VOCAB, torch.float32, 300, 20, False, 6)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    one = torch.ones(tokens, device=d)
    ws = [torch.full((max(1, size),), 0xFF, dtype=torch.uint8, device=d) for size in
          (e8q.e8q_moe_workspace_size(e, h, f, tokens, k), e8q.e8q_distill_workspace_size(tokens, VOCAB, places))]
    shapes = {"idx": ((tokens, k), torch.int32), "weight": ((tokens, k), torch.float32), "y": ((tokens, h), torch.bfloat16),
              "adjusted": ((tokens, VOCAB), torch.float32), "loss": ((tokens,), torch.float32),
              "logprob": ((tokens, places), torch.float32), "stats": ((tokens, 4), torch.float32),
              "grad": ((tokens, VOCAB), torch.float32), "both": ((tokens, VOCAB), torch.float32), "loss1": ((tokens,), torch.float32)}
    make = lambda mark: {n: torch.full(s, mark, dtype=t, device=d) for n, (s, t) in shapes.items()}  # noqa: E731

    def work(o):
        e8q.e8q_moe_core_escape(layer.gate, layer.up, layer.down, layer.bound, x, o["idx"], o["weight"], o["y"], ws[0], status,
                                router=router, signs_in=layer.signs_in, had_block_in=layer.had_in,
                                signs_down=layer.signs_down, had_block_down=layer.had_down, activation=ACT["silu"])
        e8q.e8q_adjust_logits(logits, o["adjusted"], status, **a)
        e8q.e8q_distill(o["adjusted"], ids, teacher, ws[1], status, tail=e8q.TAIL_REST, loss_out=o["loss"],
                        logprob_out=o["logprob"], stats_out=o["stats"])
        e8q.e8q_distill_backward(o["adjusted"], ids, teacher, o["stats"], one, o["grad"], status, tail=e8q.TAIL_REST)
        e8q.e8q_distill_grad(logits, ids, teacher, one, o["both"], ws[1], status, tail=e8q.TAIL_RENORM, loss_out=o["loss1"])

    def fill(seed):
        g = torch.Generator(device=d).manual_seed(seed)
        x.normal_(generator=g)
        logits.normal_(0.0, 3.0, generator=g)
        ids.copy_(torch.randint(-1, VOCAB, ids.shape, generator=g, device=d))
        teacher.uniform_(-6.0, -2.5, generator=g)

    fill(0)
    out = make(-77)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(out)
    for seed in (1, 2, 3):
        fill(seed)
        for t in out.values():
            t.fill_(-77)
        graph.replay()
        torch.cuda.synchronize()
        eager = make(-99)
        work(eager)
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], eager[n]), (seed, n)
    assert int(status.item()) == 0
