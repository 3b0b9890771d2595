"""One training step of the example from the same state on two streams: equal losses and latents, bit for bit."""

import os
import sys

import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_another_stream_gives_the_same_step():
    import qat_language_model as ex
    d = device()
    tokens, targets = ex.MarkovChain(d).sample(ex.TOKENS)

    def steps():
        model = ex.Model(d)
        losses = [model.train_step(tokens, targets) for _ in range(3)]
        return model, losses

    here, losses = steps()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        there, other = steps()
    s.synchronize()
    assert [float(v) for v in losses] == [float(v) for v in other] and float(losses[2]) < float(losses[0])
    for a, b in ((here.table, there.table), (here.inner.w, there.inner.w), (here.outer.w, there.outer.w),
                 (here.inner.momentum, there.inner.momentum), (here.outer.momentum, there.outer.momentum)):
        assert torch.equal(a, b)
    assert int(here.status.item()) == 0 and int(there.status.item()) == 0
