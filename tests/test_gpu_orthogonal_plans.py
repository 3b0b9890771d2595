"""e8q_orthogonalize and e8q_orthogonal_step in every plan of tiles and steps,
on spectra where rounding shows, against float64.

The plan follows from the sizes alone; `plan` repeats the library's rule, so that
a test says which plan it means and fails if it does not get it.

Bound.  Five default steps of float16 operands: 3.7e-3 of |O|_F (per step 3.5, 3.5
and 4.8 times 2^-12 / sqrt(3) for the roundings of M, X and A, in quadrature).
|error|^2 is a sum over n singular directions, so few of them scatter around
that: times 1 + 2 / sqrt(n).  In pairs the square A' = M A M is rounded in two
products where a single step rounds once, and its error meets the same factors:
twice the bound.  Steps beyond five add in quadrature.  The result's own rounding
to bf16 adds 2^-9 of it (root mean square), 2^-8 of an entry at most; no entry is
further off than six times the root mean square."""

import math

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu
REL = 3.7e-3


def plan(batch, rows, cols, growth=485.0):
    """(width of the square products' tiles, of the products with X, steps in pairs)"""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    n, m = min(rows, cols), max(rows, cols)

    def up(v, t):
        return (v + t - 1) // t

    def squares(t):
        return batch * (up(n, t) * (up(n, t) + 1) // 2)

    def rects(t):
        return batch * up(n, t) * up(m, t)

    def tile(of):
        small = 0.33 if of(128) <= cus else 0.75 * up(of(128), 2 * cus)
        return 256 if up(of(256), cus) <= small else 128

    rect = 64 if rects(128) < cus else tile(rects)
    square = rect if rect < 256 else tile(squares)
    return square, rect, rect != 64 and n >= 640 and m >= 2 * n and growth <= 512


def _matrix(n, m, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(n * 7 + m + seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float64)

    if kind == "flat":
        x = normal(n, m)
    elif kind == "fall":
        k = max(1, n // 8)
        x = (normal(n, k) * torch.linspace(1.0, 0.1, k, device="cuda", dtype=torch.float64)) @ normal(k, m) + 0.1 * normal(n, m)
    elif kind.startswith("rank"):
        k = max(1, n // int(kind[4:]))
        x = normal(n, k) @ normal(k, m)
    else:                                    # half of the singular values at 1e-3 of the others
        u, v = torch.linalg.qr(normal(n, n))[0], torch.linalg.qr(normal(m, n))[0]
        s = torch.ones(n, device="cuda", dtype=torch.float64)
        s[n // 2:] = 1e-3
        x = (u * s) @ v.t().contiguous()
    return (x * 1e-4).float()


def _exact(x, steps=5, coeffs=e8q.NEWTON_SCHULZ):
    a, b, c = (float(np.float32(v)) for v in coeffs)
    y = x.double()
    y = y / y.norm()
    tall = y.shape[0] > y.shape[1]
    y = y.t().contiguous() if tall else y
    for _ in range(steps):
        s = y @ y.t().contiguous()
        y = a * y + (b * s + c * (s @ s)) @ y
    return y.t().contiguous() if tall else y


def _orthogonalize(x, steps=5, coeffs=e8q.NEWTON_SCHULZ):
    out = torch.full(x.shape, 9.0, dtype=torch.bfloat16, device=x.device)
    st = torch.zeros(1, dtype=torch.int32, device=x.device)
    ws = torch.full((e8q.e8q_orthogonalize_workspace_size(*x.shape),), 0xFF, dtype=torch.uint8, device=x.device)
    e8q.e8q_orthogonalize(x, out, ws, st, steps=steps, coeffs=coeffs)
    assert int(st.item()) == 0
    return out


def _rel(shape, steps=5):
    n = min(shape[1:])
    return REL * (1 + 2 / math.sqrt(n)) * math.sqrt(max(steps, 5) / 5) * (2 if plan(*shape)[2] else 1)


def _near(got, want, rel):
    off = got.double() - want
    rms = want.pow(2).mean().sqrt()
    assert off.norm() <= (rel + 2.0 ** -9) * want.norm(), float(off.norm() / want.norm())
    assert (off.abs() <= 6 * rel * rms + 2.0 ** -8 * want.abs()).all()


KINDS = ["flat", "fall", "rank8", "rank4", "rank2", "half"]
SHAPES = [((256, 8, 64), (128, 128, False)), ((8, 16, 4096), (128, 128, False)), ((64, 32, 1024), (128, 128, False)),
          ((256, 64, 64), (128, 128, False)), ((256, 264, 64), (128, 128, False)), ((140, 257, 1280), (128, 256, False)),
          ((1, 2048, 2048), (128, 128, False)), ((8, 1024, 1024), (128, 128, False)), ((1, 1024, 4096), (128, 128, True)),
          ((1, 2056, 1032), (64, 64, False)), ((20, 769, 1280), (256, 256, False)), ((24, 704, 1408), (128, 256, True)),
          ((24, 1411, 704), (128, 256, True)), ((128, 768, 2048), (256, 256, True)), ((1, 2048, 8192), (128, 256, True)),
          ((1, 8195, 2048), (128, 256, True)), ((1, 4096, 4096), (256, 256, False)), ((1, 5503, 4096), (256, 256, False))]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,takes", SHAPES)
def test_spectra(shape, takes, kind):
    device()
    assert plan(*shape) == takes
    x = _matrix(min(shape[1:]), max(shape[1:]), kind)
    x = x.t().contiguous() if shape[1] > shape[2] else x
    got = _orthogonalize(x.expand(shape).contiguous())
    _near(got[0], _exact(x), _rel(shape))
    assert torch.equal(got[0], got[-1])


@pytest.mark.parametrize("steps,coeffs,growth", [
    (1, e8q.NEWTON_SCHULZ, 3.4), (2, e8q.NEWTON_SCHULZ, 12.0), (3, e8q.NEWTON_SCHULZ, 41.0), (4, e8q.NEWTON_SCHULZ, 141.0),
    (6, e8q.NEWTON_SCHULZ, 1670.0), (6, (1.5, -0.5, 0.0), 11.4), (4, (1.875, -1.25, 0.375), 12.4), (3, (2.0, -1.5, 0.5), 8.0)])
@pytest.mark.parametrize("shape", [(24, 704, 1408), (2, 4096, 1536), (8, 1024, 1024)])
def test_steps_and_coefficients(shape, steps, coeffs, growth):
    """Even and odd numbers of steps, wide, tall and square; six default steps are too many for pairs."""
    device()
    assert plan(*shape, growth)[2] == (shape != (8, 1024, 1024) and steps * (coeffs == e8q.NEWTON_SCHULZ) < 6)
    for kind in ("fall", "rank4"):
        x = _matrix(min(shape[1:]), max(shape[1:]), kind)
        x = x.t().contiguous() if shape[1] > shape[2] else x
        got = _orthogonalize(x.expand(shape).contiguous(), steps, coeffs)
        _near(got[0], _exact(x, steps, coeffs), _rel(shape, steps))


@pytest.mark.parametrize("shape,takes", [((8, 1024, 1024), (128, 128, False)), ((2, 2048, 1024), (128, 128, True)),
                                         ((24, 704, 1408), (128, 256, True)), ((24, 1411, 704), (128, 256, True)),
                                         ((1, 4096, 4096), (256, 256, False)), ((1, 14337, 4096), (256, 256, True))])
@pytest.mark.parametrize("nesterov", [True, False])
def test_latents_step(shape, takes, nesterov):
    """The whole step, momentum and latents in place and not, in the larger tiles, wide and tall."""
    d = device()
    assert plan(*shape) == takes
    turn = shape[1] > shape[2]
    n, m = min(shape[1:]), max(shape[1:])

    def matrix(kind, seed):
        x = _matrix(n, m, kind, seed)
        return (x.t() if turn else x).expand(shape).contiguous()

    grad, mom = matrix("fall", 1).to(torch.bfloat16), matrix("rank8", 2)
    w = (torch.randn(shape[1:], generator=torch.Generator(device="cuda").manual_seed(3), device=d) * 0.02)
    w = w.to(torch.bfloat16).expand(shape).contiguous()
    mu, lr, decay, gamma = 0.95, 0.05, 0.1, 1.5
    w_out, m_out = torch.empty_like(w), torch.empty_like(mom)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_orthogonalize_workspace_size(*shape), dtype=torch.uint8, device=d)
    e8q.e8q_orthogonal_step(w, grad, mom, ws, st, mu=mu, nesterov=nesterov, lr=lr, decay=decay, gamma=gamma,
                            w_out=w_out, momentum_out=m_out)
    mu64 = float(np.float32(mu))
    m1 = mu64 * mom[0].double() + grad[0].double()
    assert ((m_out[0].double() - m1).abs() <= 2.0 ** -23 * (mom[0].double().abs() + grad[0].double().abs())).all()
    o = _exact(grad[0].double() + mu64 * m1 if nesterov else m1)
    want = w[0].double() * (1 - lr * decay) - lr * gamma * o
    lim = (lr * gamma * 6 * _rel(shape) * o.pow(2).mean().sqrt() + 2.0 ** -8 * want.abs()
           + 2.0 ** -21 * (w[0].double().abs() + lr * gamma * o.abs()))
    assert ((w_out[0].double() - want).abs() <= lim).all()
    # the steps themselves to the bound of the whole: what the latents moved by, less their rounding
    moved = w_out[0].double() - w[0].double() * (1 - lr * decay)
    assert (moved + lr * gamma * o).norm() <= lr * gamma * _rel(shape) * o.norm() + 2.0 ** -9 * want.norm()
    assert torch.equal(w_out[0], w_out[-1]) and torch.equal(m_out[0], m_out[-1])
    e8q.e8q_orthogonal_step(w, grad, mom, ws, st, mu=mu, nesterov=nesterov, lr=lr, decay=decay, gamma=gamma)
    assert torch.equal(w, w_out) and torch.equal(mom, m_out) and int(st.item()) == 0


def test_step_of_a_batch_with_nonfinite_and_zero_matrices():
    d, shape = device(), (24, 704, 1408)
    assert plan(*shape) == (128, 256, True)
    grad = _matrix(704, 1408, "flat").expand(shape).contiguous()
    grad[1] = 0
    grad[2, 700, 4] = float("inf")
    w = torch.full(shape, 0.5, dtype=torch.bfloat16, device=d)
    mom, st = torch.zeros(shape, device=d), torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_orthogonalize_workspace_size(*shape), dtype=torch.uint8, device=d)
    e8q.e8q_orthogonal_step(w, grad, mom, ws, st, lr=0.5, decay=0.25)
    assert int(st.item()) == e8q.STATUS_BITS["NONFINITE"]
    assert (w[1] == torch.tensor(0.5 * (1 - 0.125), dtype=torch.bfloat16)).all() and torch.isnan(w[2]).all()
    assert torch.isfinite(w[0]).all() and torch.equal(w[0], w[3]) and torch.equal(w[0], w[-1])


def test_oracle_agrees_with_the_reference_here():
    x = _matrix(72, 136, "half")
    want = oracle.orthogonalize(x[None].double().cpu().numpy())[0]
    assert np.abs(_exact(x).cpu().numpy() - want).max() <= 1e-9
