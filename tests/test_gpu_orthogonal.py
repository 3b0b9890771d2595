"""e8q_orthogonalize and e8q_orthogonal_step against float64.

Bound.  An operand rounded to float16 is off by at most 2^-12 of itself, 2^-12 /
sqrt(3) in the root mean square.  In a step the rounding of D = M - alpha I and
of X meet |D| <= 3.5 each, and that of A meets |b + 2 c s^2| <= 4.8 (s <= 1.2):
together (3.5 + 3.5 + 4.8) 2^-12 / sqrt(3) of |X|; five steps add up in
quadrature to 3.7e-3 of |O|_F.  No entry is further off than six times that
(in units of the root mean square), plus the last rounding to bf16 (2^-9 rms,
2^-8 of an entry at most)."""

import numpy as np
import pytest
import torch

import bit_e8_lattice_amd as e8q
import oracle
from gpu_util import device

pytestmark = pytest.mark.gpu
REL = 3.7e-3


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _gradient(shape, seed, kind):
    g = torch.Generator().manual_seed(seed)
    b, r, c = shape
    noise = torch.randn(shape, generator=g)
    if kind == "flat":
        return noise * 1e-4
    k = max(1, min(r, c) // 8)
    left = torch.randn((b, r, k), generator=g) * torch.linspace(1.0, 0.1, k)
    low = torch.bmm(left, torch.randn((b, k, c), generator=g))
    return low * 1e-4 if kind == "rank" else (low + 0.1 * noise) * 1e-4


def _run(x, steps=5, coeffs=e8q.NEWTON_SCHULZ, stream=None):
    d = x.device
    b, r, c = x.shape if x.dim() == 3 else (1,) + tuple(x.shape)
    out = torch.full(x.shape, 9.0, dtype=torch.bfloat16, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.full((e8q.e8q_orthogonalize_workspace_size(b, r, c),), 0xFF, dtype=torch.uint8, device=d)  # NaNs
    e8q.e8q_orthogonalize(x, out, ws, st, steps=steps, coeffs=coeffs, stream=stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def _near(got, want, extra=0.0):
    for g, w in zip(got, want):
        rms = np.sqrt((w * w).mean())
        if rms == 0.0:
            assert not g.any()
            continue
        assert np.linalg.norm(g - w) <= (REL + 2.0 ** -9 + extra) * np.linalg.norm(w)
        assert (np.abs(g - w) <= 6 * REL * rms + (2.0 ** -8 + extra) * np.abs(w)).all()


SHAPES = [(1, 1, 8), (1, 8, 8), (1, 3, 64), (2, 65, 8), (1, 64, 64), (3, 63, 72), (1, 130, 128), (1, 128, 1000),
          (1, 1001, 136), (2, 256, 256), (5, 200, 328), (1, 768, 520), (1, 520, 768), (40, 136, 264), (1, 1025, 1032)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["flat", "fall", "rank"])
def test_orthogonalize(shape, kind):
    for dtype in (torch.bfloat16, torch.float32):
        x = _gradient(shape, sum(shape), kind).to(dtype).to(device())
        got, st = _run(x)
        assert st == 0
        _near(_f64(got), oracle.orthogonalize(_f64(x)))


@pytest.mark.parametrize("shape", [(140, 257, 512), (20, 769, 1280), (3, 2049, 2056), (1, 4096, 3840)])
def test_large_tiles(shape):
    """Shapes that fill the chip: against float64 products on the GPU."""
    x = _gradient((1,) + shape[1:], 5, "fall").to(torch.bfloat16).to(device())
    x = (x * torch.linspace(0.5, 2.0, shape[0], device=x.device)[:, None, None].to(torch.bfloat16)).contiguous()
    x[-1] = x[-1].flip(0)
    got, st = _run(x)
    assert st == 0
    for i in {0, shape[0] // 2, shape[0] - 1}:
        y = x[i].double()
        y = y / y.norm()
        y = y.t().contiguous() if y.shape[0] > y.shape[1] else y
        for _ in range(5):
            s = y @ y.t().contiguous()
            y = 3.4445 * y + (-4.775 * s + 2.0315 * (s @ s)) @ y
        y = y.t() if shape[1] > shape[2] else y
        _near([got[i].double().cpu().numpy()], [y.cpu().numpy()])


def test_long_matrix_with_small_square_tiles():
    """One side much longer: the square products take smaller tiles than those with X."""
    test_large_tiles((1, 1537, 6144))


@pytest.mark.parametrize("shape", [(20, 769, 1280), (40, 257, 1280)])
def test_rounding_spares_no_rows(shape):
    """Errors of products taken for symmetric would gather in some tiles' rows."""
    x = _gradient((1,) + shape[1:], 5, "fall").to(torch.bfloat16).expand(shape).contiguous().to(device())
    got, _ = _run(x)
    want = oracle.orthogonalize(_f64(x[:1]))[0]
    err = np.linalg.norm(_f64(got[:1])[0] - want, axis=1) / np.linalg.norm(want, axis=1)
    blocks = [err[i:i + 64].mean() for i in range(0, shape[1] - shape[1] % 64, 64)]
    assert max(blocks) <= 1.25 * min(blocks)


@pytest.mark.parametrize("shape", [(20, 769, 1280), (2, 1025, 1032), (5, 200, 328)])
def test_runs_agree_bit_for_bit(shape):
    x = _gradient(shape, 5, "fall").to(torch.bfloat16).to(device())
    first, _ = _run(x)
    for _ in range(10):
        assert torch.equal(_run(x)[0], first)


def test_nonfinite_and_zero_matrices_in_large_batches():
    for shape in ((40, 136, 264), (20, 769, 1280)):
        x = _gradient((1,) + shape[1:], 6, "flat").expand(shape).contiguous().to(device())
        x[1] = 0
        x[2, 100, 4] = float("-inf")
        got, st = _run(x)
        assert st == e8q.STATUS_BITS["NONFINITE"]
        assert not got[1].any() and torch.isnan(got[2]).all()
        assert torch.equal(got[3], got[0]) and torch.equal(got[-1], got[0]) and torch.isfinite(got[0]).all()


@pytest.mark.parametrize("steps,coeffs", [(1, e8q.NEWTON_SCHULZ), (2, e8q.NEWTON_SCHULZ), (9, (1.5, -0.5, 0.0)),
                                          (4, (1.875, -1.25, 0.375))])
def test_steps_and_coefficients(steps, coeffs):
    x = _gradient((2, 96, 200), 9, "fall").to(device())
    got, _ = _run(x, steps, coeffs)
    _near(_f64(got), oracle.orthogonalize(_f64(x), steps, coeffs))


@pytest.mark.parametrize("steps,coeffs", [(2, e8q.NEWTON_SCHULZ), (4, e8q.NEWTON_SCHULZ), (1, e8q.NEWTON_SCHULZ),
                                          (9, (1.5, -0.5, 0.0))])
def test_steps_in_pairs(steps, coeffs):
    """Batches that fill the chip take two steps at a time where one side is longer."""
    x = _gradient((1, 136, 264), 9, "fall").expand(40, 136, 264).contiguous().to(device())
    got, _ = _run(x, steps, coeffs)
    _near(_f64(got[:1]), oracle.orthogonalize(_f64(x[:1]), steps, coeffs))
    assert torch.equal(got[0], got[39])


@pytest.mark.parametrize("size", [1e-30, 1e30, 1.0])
def test_magnitude_does_not_matter(size):
    x = (_gradient((1, 64, 160), 2, "flat") * 1e4 * size).to(device())
    got, st = _run(x)
    assert st == 0
    _near(_f64(got), oracle.orthogonalize(_f64(x)))


def test_outlier_entry():
    """One entry holds nearly all of the norm."""
    x = _gradient((1, 128, 256), 2, "flat")
    x[0, 5, 7] = 3.0
    x = x.to(device())
    got, _ = _run(x)
    _near(_f64(got), oracle.orthogonalize(_f64(x)))


def test_zero_and_nonfinite_matrices_of_a_batch():
    x = _gradient((4, 72, 144), 3, "flat").to(device())
    x[1] = 0
    x[2, 3, 4] = float("inf")
    x[3, 71, 0] = float("nan")
    got, st = _run(x)
    assert st == e8q.STATUS_BITS["NONFINITE"]
    _near(_f64(got)[:1], oracle.orthogonalize(_f64(x)[:1]))
    assert not got[1].any() and torch.isnan(got[2]).all() and torch.isnan(got[3]).all()


def test_two_dimensional_and_other_stream_and_repeat():
    x = _gradient((1, 200, 264), 4, "fall").to(device())[0]
    a, _ = _run(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = _run(x, stream=s)
    assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(1, 40, 64), (2, 264, 136), (1, 136, 1000)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step(shape, nesterov, dtype):
    d = device()
    grad = _gradient(shape, 1, "fall").to(dtype).to(d)
    mom = _gradient(shape, 2, "fall").to(d)
    w = (torch.randn(shape, generator=torch.Generator().manual_seed(3)) * 0.02).to(torch.bfloat16).to(d)
    mu, lr, decay, gamma = 0.95, 0.05, 0.1, 1.5
    w_out, m_out = torch.empty_like(w), torch.empty_like(mom)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_orthogonalize_workspace_size(*shape), dtype=torch.uint8, device=d)
    e8q.e8q_orthogonal_step(w, grad, mom, ws, st, mu=mu, nesterov=nesterov, lr=lr, decay=decay, gamma=gamma,
                            w_out=w_out, momentum_out=m_out)
    ref_w, ref_m, o = oracle.orthogonal_step(_f64(w), _f64(grad), _f64(mom), np.float64(np.float32(mu)), nesterov,
                                             lr, decay, gamma)
    # momentum: one product and sum in float32
    assert (np.abs(_f64(m_out) - ref_m) <= 2.0 ** -23 * (np.abs(_f64(mom)) + np.abs(_f64(grad)))).all()
    rms = np.sqrt((o * o).mean())
    lim = lr * gamma * 6 * REL * rms + 2.0 ** -8 * np.abs(ref_w) + 2.0 ** -21 * (np.abs(_f64(w)) + lr * gamma * np.abs(o))
    assert (np.abs(_f64(w_out) - ref_w) <= lim).all()
    # in place
    w2, m2 = w.clone(), mom.clone()
    e8q.e8q_orthogonal_step(w2, grad, m2, ws, st, mu=mu, nesterov=nesterov, lr=lr, decay=decay, gamma=gamma)
    assert torch.equal(w2, w_out) and torch.equal(m2, m_out) and int(st.item()) == 0


def test_refusals():
    d = device()
    x = torch.zeros((64, 64), device=d)
    out = torch.empty((64, 64), dtype=torch.bfloat16, device=d)
    st = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(e8q.e8q_orthogonalize_workspace_size(1, 64, 64), dtype=torch.uint8, device=d)
    for kw in ({"steps": 0}, {"steps": 17}, {"coeffs": (9.0, 0.0, 0.0)}, {"coeffs": (3.4445, 0.0, 0.0)},
               {"coeffs": (float("nan"), 0.0, 0.0)}):
        with pytest.raises(e8q.E8QError):
            e8q.e8q_orthogonalize(x, out, ws, st, **kw)
    with pytest.raises(e8q.E8QError):
        e8q.e8q_orthogonalize(x, out, ws[:-256], st)
    with pytest.raises(e8q.E8QError):
        e8q.e8q_orthogonalize(x[:, :60].contiguous(), out[:, :60].contiguous(), ws, st)      # cols % 8
    with pytest.raises(TypeError):
        e8q.e8q_orthogonalize(x, x, ws, st)
    with pytest.raises(ValueError):
        e8q.e8q_orthogonalize(x, out[:32], ws, st)
    with pytest.raises(ValueError):
        e8q.e8q_orthogonal_step(out, x, x[:32], ws, st)
    assert int(st.item()) == 0
