"""The example's training step runs the operators together, and learns: from
ln(512) = 6.24 the loss comes closer to the chain's entropy (1.04)."""

import os
import sys

import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_learns_the_chain():
    import qat_language_model as ex
    device()
    losses, model, chain = ex.train(120)
    assert losses[0] > 5.0
    assert sum(losses[-10:]) / 10 < 3.0, losses[::10]
    assert int(model.status.item()) == 0
    idx, lp, ent = model.likely_next(3)
    assert len(idx) == 5 and lp == sorted(lp, reverse=True) and 0.0 <= ent <= 6.25
    # another stream gives the same result as the current one
    t, n = chain.sample(ex.TOKENS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss = model.train_step(t, n)
    torch.cuda.current_stream().wait_stream(s)
    assert float(loss) == float(loss)
