"""Exported experts for the tests of the mixture-of-experts layer."""

import numpy as np
import torch

import bit_e8_lattice_amd as e8q
import oracle
from bit_e8_lattice_amd import workloads
from gpu_util import run_encode

ACT = {"silu": e8q.ACT_SILU, "gelu_tanh": e8q.ACT_GELU_TANH}


def export(shape, bound, alpha, signs, had, seed, device, outliers=0):
    """``Experts`` of random weights, and (2z, scale) for the oracle."""
    experts, rows, cols = shape
    w = workloads.normal(shape, seed, device, dtype=torch.float32)
    scale = workloads.rms_scale(w, alpha)
    if outliers:
        # some groups far out: 2z of up to 14 bits
        g = torch.Generator(device=device).manual_seed(seed)
        at = torch.randint(0, w.numel() // 8, (outliers,), generator=g, device=device)
        w.view(-1, 8)[at] *= 10.0 ** (4 * torch.rand((outliers, 1), generator=g, device=device))
    enc = run_encode(w, scale, bound, signs=signs, hb=had, keep_device=True)
    core, esc, cnt = enc["dev"]
    two_z = oracle.exported_two_z(enc["core_idx"], enc["records"], enc["counts"], shape, bound)
    m = e8q.Experts(core, esc, cnt, scale, shape, esc_records=len(enc["records"]))
    return m, (two_z, scale.cpu().numpy().reshape(experts, rows)), enc


class Layer:
    def __init__(self, experts, hidden, inter, bound, alpha, had_in, had_down, seed, device, outliers=0):
        self.shape, self.bound, self.device = (experts, hidden, inter), bound, device
        self.had_in, self.had_down = had_in, had_down
        self.signs_in = workloads.signs(hidden, seed + 1, device) if had_in else None
        self.signs_down = workloads.signs(inter, seed + 2, device) if had_down else None
        made = [export((experts, r, c), bound, alpha, s, hb, seed + 3 + i, device, outliers) for i, (r, c, s, hb) in
                enumerate(((inter, hidden, self.signs_in, had_in), (inter, hidden, self.signs_in, had_in),
                           (hidden, inter, self.signs_down, had_down)))]
        self.gate, self.up, self.down = (m[0] for m in made)
        self.oracle = [m[1] for m in made]
        self.encoded = [m[2] for m in made]

    def run(self, x, k, router=None, normalize=True, act="silu", y_dtype=torch.float32, idx=None, weight=None, stream=None,
            ws=None):
        d, t = self.device, x.shape[0]
        idx = torch.full((t, k), -9, dtype=torch.int32, device=d) if idx is None else idx
        weight = torch.full((t, k), 9.0, device=d) if weight is None else weight
        y = torch.full(x.shape, 7.0, dtype=y_dtype, device=d)
        st = torch.zeros(1, dtype=torch.int32, device=d)
        e, h, f = self.shape
        if ws is None:
            ws = torch.full((e8q.e8q_moe_workspace_size(e, h, f, t, k),), 0xFF, dtype=torch.uint8, device=d)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        e8q.e8q_moe_core_escape(self.gate, self.up, self.down, self.bound, x, idx, weight, y, ws, st, router=router,
                                signs_in=self.signs_in, had_block_in=self.had_in, signs_down=self.signs_down,
                                had_block_down=self.had_down, activation=ACT[act], normalize=normalize, stream=stream)
        torch.cuda.synchronize()
        return y, idx, weight, int(st.item())

    def expect(self, x, idx, weight, act="silu"):
        signs = [None if s is None else s.cpu().numpy().astype(np.float64) for s in (self.signs_in, self.signs_down)]
        return oracle.moe_layer(x.float().cpu().numpy(), *self.oracle, idx, weight, signs[0], self.had_in, signs[1],
                                self.had_down, act)
