#!/usr/bin/env python3
"""Quantization-aware training of a small next-token model, every step on the library's operators.

The model: embedding (bf16 latents, scaled lookup) -> linear -> ReLU -> linear
to the vocabulary.  Both linear layers multiply by the E8 projection of their
bf16 latents (``e8q_project_hadamard_restore``); the identity straight-through
estimator hands their gradients to the latents.  One step:

1. ``e8q_embed``                         h = scale * E[tokens]
2. ``e8q_project_hadamard_restore``      W_hat of both layers; plain products
3. ``e8q_token_logprobs_grad``           loss terms and the logits' gradient
4. plain products                        gradients of W_hat (= of the latents) and of h
5. ``e8q_orthogonal_step``               the linear layers' latents
6. ``e8q_embed_backward``                SGD on the embedding rows that occurred

At the end ``e8q_token_logprobs`` lists the likely next tokens of a prompt token.
The data is a random Markov chain, so the loss has a known floor (its entropy).

Run: ``python examples/qat_language_model.py [--steps N]`` (needs an MI355X).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_e8_lattice_amd as e8q  # noqa: E402
from bit_e8_lattice_amd import workloads  # noqa: E402

VOCAB, DIM, HIDDEN, TOKENS = 512, 256, 512, 4096
EMBED_SCALE = 16.0
HAD_BLOCK = 128


class ProjectedLinear:
    """bf16 latents [rows, cols] used through their E8 projection."""

    def __init__(self, rows, cols, seed, device):
        self.w = workloads.normal((rows, cols), seed, device, std=cols ** -0.5)
        self.signs = workloads.signs(cols, seed + 1, device)
        self.w_hat = torch.empty_like(self.w)
        self.momentum = torch.zeros((rows, cols), dtype=torch.float32, device=device)
        self.ws = torch.empty(e8q.e8q_orthogonalize_workspace_size(1, rows, cols), dtype=torch.uint8, device=device)

    def project(self, status):
        scale = workloads.rms_scale(self.w, 0.7)
        e8q.e8q_project_hadamard_restore(self.w, scale, self.signs, HAD_BLOCK, self.w_hat, status)
        return self.w_hat

    def step(self, grad, status, lr):
        rows, cols = self.w.shape
        e8q.e8q_orthogonal_step(self.w, grad, self.momentum, self.ws, status, lr=lr,
                                gamma=max(1.0, rows / cols) ** 0.5)


class Model:
    def __init__(self, device, seed=1):
        self.device = device
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.table = workloads.normal((VOCAB, DIM), seed, device, std=1.0 / EMBED_SCALE)
        self.inner = ProjectedLinear(HIDDEN, DIM, seed + 10, device)
        self.outer = ProjectedLinear(VOCAB, HIDDEN, seed + 20, device)
        new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        self.h, self.dlogits = new(TOKENS, DIM), new(TOKENS, VOCAB)
        self.logprob = new(TOKENS, 1, dtype=torch.float32)
        self.weight = torch.full((TOKENS, 1), -1.0 / TOKENS, device=device)
        self.lp_ws = new(max(1, e8q.e8q_token_logprobs_workspace_size(TOKENS, VOCAB)), dtype=torch.uint8)
        self.embed_ws = new(e8q.e8q_embed_backward_workspace_size(TOKENS, VOCAB, DIM), dtype=torch.uint8)

    def logits(self, tokens, h):
        e8q.e8q_embed(self.table, tokens, h, self.status, scale=EMBED_SCALE)
        a = torch.relu(h @ self.inner.project(self.status).t())
        return a, a @ self.outer.project(self.status).t()

    def train_step(self, tokens, targets, lr=0.02, embed_lr=2.0):
        """One step on ``tokens`` -> ``targets``; returns the mean loss (a device tensor)."""
        a, logits = self.logits(tokens, self.h)
        e8q.e8q_token_logprobs_grad(logits, targets, self.weight, self.dlogits, self.lp_ws, self.status,
                                    logprob_out=self.logprob)
        d_outer = self.dlogits.t() @ a
        da = torch.where(a > 0, self.dlogits @ self.outer.w_hat, 0)
        d_inner = da.t() @ self.h
        dh = da @ self.inner.w_hat
        self.outer.step(d_outer, self.status, lr)
        self.inner.step(d_inner, self.status, lr)
        e8q.e8q_embed_backward(dh, tokens, VOCAB, self.embed_ws, self.status, scale=EMBED_SCALE,
                               w_latent=self.table, lr=embed_lr)
        return -self.logprob.mean()

    def likely_next(self, token, k=5):
        """The ``k`` most likely next tokens, their log probabilities, and the entropy."""
        tokens = torch.tensor([token], device=self.device)
        _, logits = self.logits(tokens, torch.empty((1, DIM), dtype=torch.bfloat16, device=self.device))
        idx = torch.empty((1, k), dtype=torch.int32, device=self.device)
        lp, ent = torch.empty((1, k), device=self.device), torch.empty(1, device=self.device)
        size = e8q.e8q_token_logprobs_workspace_size(1, VOCAB, k)
        ws = torch.empty(max(1, size), dtype=torch.uint8, device=self.device)
        e8q.e8q_token_logprobs(logits, ws, self.status, entropy_out=ent, top_idx_out=idx, top_logprob_out=lp)
        return idx[0].tolist(), lp[0].tolist(), float(ent)


class MarkovChain:
    """Four successors per token with fixed probabilities."""

    def __init__(self, device, seed=7):
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        self.next = torch.randint(0, VOCAB, (VOCAB, 4), generator=self.g, device=device)
        self.p = torch.tensor([0.6, 0.25, 0.1, 0.05], device=device)
        self.entropy = float(-(self.p * self.p.log()).sum())

    def sample(self, n):
        tokens = torch.randint(0, VOCAB, (n,), generator=self.g, device=self.p.device)
        pick = torch.multinomial(self.p, n, replacement=True, generator=self.g)
        return tokens, self.next[tokens, pick]


def train(steps, device="cuda", report=None):
    """Trains for ``steps`` steps; returns the losses and the model and chain."""
    model, chain = Model(device), MarkovChain(device)
    losses = []
    for i in range(steps):
        loss = model.train_step(*chain.sample(TOKENS))
        if report and i % report == 0:
            print(f"step {i:4d}  loss {float(loss):.4f}  (floor {chain.entropy:.4f})", flush=True)
        losses.append(loss)
    return [float(v) for v in losses], model, chain


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    losses, model, chain = train(args.steps, report=max(1, args.steps // 10))
    idx, lp, ent = model.likely_next(3)
    print(f"last loss {losses[-1]:.4f}, floor {chain.entropy:.4f}, status {int(model.status.item())}")
    print("after token 3:", ", ".join(f"{i} ({v:.2f})" for i, v in zip(idx, lp)), f"entropy {ent:.3f};",
          "the chain's successors:", chain.next[3].tolist())


if __name__ == "__main__":
    main()
