"""The operators in a HIP graph: captured once, replayed with the program's own
work in between, each replay equal to the eager calls."""

import pytest
import torch

import bit_e8_lattice_amd as e8q
from gpu_util import device

pytestmark = pytest.mark.gpu


def test_graph_replays_equal_eager_calls():
    d = device()
    rows, vocab, dim, n = 6, 40000, 136, 5000
    x = torch.empty((rows, vocab), dtype=torch.bfloat16, device=d)
    tok = torch.randint(0, vocab, (rows,), device=d)
    ids = torch.empty(n, dtype=torch.int64, device=d)
    g, w = torch.empty((n, dim), device=d), torch.empty((3, 200, 328), device=d)
    lp, idx = torch.empty((rows, 1), device=d), torch.empty((rows, 7), dtype=torch.int32, device=d)
    dx, up = torch.empty_like(x), torch.empty(w.shape, dtype=torch.bfloat16, device=d)
    out, grad = torch.empty((n, dim), device=d), torch.empty((999, dim), device=d)
    table = torch.randn((999, dim), device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    byte = lambda size: torch.full((max(1, size),), 0xFF, dtype=torch.uint8, device=d)  # noqa: E731
    ws = [byte(e8q.e8q_token_logprobs_workspace_size(rows, vocab, 7)), byte(e8q.e8q_token_logprobs_workspace_size(rows, vocab)),
          byte(e8q.e8q_embed_backward_workspace_size(n, 999, dim)), byte(e8q.e8q_orthogonalize_workspace_size(*w.shape))]
    one = torch.ones((rows, 1), device=d)

    def work():
        e8q.e8q_token_logprobs(x, ws[0], st, tokens=tok, logprob_out=lp, top_idx_out=idx)
        e8q.e8q_token_logprobs_grad(x, tok, one, dx, ws[1], st)
        e8q.e8q_embed(table, ids, out, st, scale=2.0)
        e8q.e8q_embed_backward(g, ids, 999, ws[2], st, grad_table=grad)
        e8q.e8q_orthogonalize(w, up, ws[3], st)

    def fill(seed):
        gen = torch.Generator(device=d)
        gen.manual_seed(seed)
        x.normal_(0.0, 3.0, generator=gen)
        g.normal_(generator=gen)
        w.normal_(generator=gen)
        ids.copy_(torch.randint(-1, 999, (n,), generator=gen, device=d))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    outs = (lp, idx, dx, out, grad, up)
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        work()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
    assert int(st.item()) == 0
