"""CPU checks of the operators' C entry points: bad arguments are refused on
the host, before anything is launched (the pointers are never followed)."""

import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    import bit_e8_lattice_amd as e8q
    if not os.path.exists(e8q.library_path):
        from bit_e8_lattice_amd.build import build
        build()
    return e8q.lib()


def _with(base, **changes):
    out = list(base)
    for k, v in changes.items():
        out[int(k[1:])] = v
    return out


def test_token_logprobs_rejects(L):
    # logits, dtype, rows, vocab, stride, scale, tokens, index, n, logprob, lse, entropy, k, idx, lp, ws, bytes, status, stream
    base = [FAKE, 1, 4, 100, 100, 1.0, FAKE, 1, 1, FAKE, FAKE, FAKE, 5, FAKE, FAKE, FAKE, 1 << 30, FAKE, None]
    f = L.e8q_token_logprobs
    bad = [_with(base, a0=None), _with(base, a1=2), _with(base, a2=0), _with(base, a3=0), _with(base, a4=99),
           _with(base, a5=0.0), _with(base, a5=float("inf")), _with(base, a5=float("nan")), _with(base, a6=None),
           _with(base, a7=2), _with(base, a8=0), _with(base, a8=-1), _with(base, a12=-1), _with(base, a12=101),
           _with(base, a12=0), _with(base, a13=None, a14=None), _with(base, a17=None), _with(base, a0=ODD),
           _with(base, a9=None, a10=None, a11=None, a12=0, a13=None, a14=None)]
    for args in bad:
        assert f(*args) == INVALID, args
    for args in (_with(base, a8=1025), _with(base, a12=65), _with(base, a2=1 << 24),
                 _with(base, a3=(1 << 31) - 16, a4=1 << 31)):
        assert f(*args) == UNSUPPORTED, args
    # few long rows are split and need the workspace
    long = _with(base, a2=1, a3=131072, a4=131072)
    need = L.e8q_token_logprobs_workspace_size(1, 131072, 5)
    assert need > 0 and L.e8q_token_logprobs_workspace_size(8192, 131072, 0) == 0
    for args in (_with(long, a15=None), _with(long, a16=0), _with(long, a15=ctypes.c_void_p(0x10010))):
        assert f(*args) == INVALID, args
    assert L.e8q_token_logprobs_workspace_size(0, 10, 0) == 0
    assert L.e8q_token_logprobs_workspace_size(1, 131072, 65) == 0


def test_token_logprobs_gradients_reject(L):
    # logits, dtype, rows, vocab, stride, scale, tokens, index, n, lse, g, entropy, g_entropy, dx, dx_stride, status, stream
    base = [FAKE, 0, 4, 100, 100, 1.0, FAKE, 0, 1, FAKE, FAKE, None, None, FAKE, 100, FAKE, None]
    f = L.e8q_token_logprobs_backward
    for args in (_with(base, a9=None), _with(base, a10=None), _with(base, a11=FAKE), _with(base, a12=FAKE),
                 _with(base, a13=None), _with(base, a14=99), _with(base, a14=101), _with(base, a13=ODD),
                 _with(base, a15=None)):
        assert f(*args) == INVALID, args                # (dx is logits: the strides have to agree)
    # logits, dtype, rows, vocab, stride, scale, tokens, index, n, g, g_entropy, logprob, lse, entropy, dx, dx_stride, ws, bytes,
    # status, stream
    base = [FAKE, 0, 4, 100, 100, 1.0, FAKE, 0, 1, FAKE, None, FAKE, None, None, FAKE, 100, None, 0, FAKE, None]
    f = L.e8q_token_logprobs_grad
    for args in (_with(base, a9=None), _with(base, a14=None), _with(base, a15=99), _with(base, a18=None),
                 _with(base, a6=None, a8=0), _with(base, a2=1, a3=131072, a4=131072, a15=131072)):
        assert f(*args) == INVALID, args


def test_embed_rejects(L):
    # table, dtype, vocab, dim, tokens, index, n, scale, out, dtype, status, stream
    base = [FAKE, 1, 100, 16, FAKE, 1, 5, 1.0, FAKE, 0, FAKE, None]
    f = L.e8q_embed
    for args in (_with(base, a0=None), _with(base, a1=7), _with(base, a2=0), _with(base, a3=0), _with(base, a4=None),
                 _with(base, a5=3), _with(base, a6=0), _with(base, a8=None), _with(base, a9=5), _with(base, a10=None),
                 _with(base, a0=ODD), _with(base, a4=ctypes.c_void_p(0x10004))):
        assert f(*args) == INVALID, args
    assert f(*_with(base, a2=1 << 31)) == UNSUPPORTED
    # grad_out, dtype, n, dim, tokens, index, vocab, scale, grad_table, dtype, latents, lr, ws, bytes, status, stream
    size = L.e8q_embed_backward_workspace_size(5, 100, 16)
    base = [FAKE, 1, 5, 16, ctypes.c_void_p(0x20000), 1, 100, 1.0, ctypes.c_void_p(0x30000), 0,
            ctypes.c_void_p(0x40000), 0.1, ctypes.c_void_p(0x50000), size, FAKE, None]
    f = L.e8q_embed_backward
    for args in (_with(base, a0=None), _with(base, a8=None, a10=None), _with(base, a8=FAKE), _with(base, a10=FAKE),
                 _with(base, a10=ctypes.c_void_p(0x30000)), _with(base, a12=None), _with(base, a13=size - 1),
                 _with(base, a12=ctypes.c_void_p(0x50010)), _with(base, a2=0), _with(base, a9=2), _with(base, a14=None)):
        assert f(*args) == INVALID, args
    assert L.e8q_embed_backward_workspace_size(0, 1, 1) == 0 and L.e8q_embed_backward_workspace_size(1, 1 << 31, 1) == 0


def test_orthogonalize_rejects(L):
    c = (3.4445, -4.775, 2.0315)
    size = L.e8q_orthogonalize_workspace_size(1, 64, 64)
    assert size > 0 and L.e8q_orthogonalize_workspace_size(1, 64, 60) == 0
    assert L.e8q_orthogonalize_workspace_size(0, 64, 64) == 0 and L.e8q_orthogonalize_workspace_size(1, 65537, 64) == 0
    # g, dtype, batch, rows, cols, steps, a, b, c, out, ws, bytes, status, stream
    base = [FAKE, 1, 1, 64, 64, 5, *c, FAKE, FAKE, size, FAKE, None]
    f = L.e8q_orthogonalize
    for args in (_with(base, a0=None), _with(base, a0=ctypes.c_void_p(0x10008)), _with(base, a1=2), _with(base, a2=0),
                 _with(base, a3=0), _with(base, a4=60), _with(base, a6=float("nan")), _with(base, a9=None),
                 _with(base, a10=None), _with(base, a11=size - 1), _with(base, a12=None)):
        assert f(*args) == INVALID, args
    for args in (_with(base, a5=0), _with(base, a5=17), _with(base, a3=65537), _with(base, a2=65536),
                 _with(base, a6=8.0), _with(base, a6=3.4445, a7=0.0, a8=0.0)):
        assert f(*args) == UNSUPPORTED, args
    # w, w_out, grad, dtype, m, m_out, mu, nesterov, lr, decay, gamma, batch, rows, cols, steps, a, b, c, ws, bytes, status, stream
    p = [ctypes.c_void_p(0x10000 * i) for i in range(1, 6)]
    base = [p[0], p[0], p[1], 1, p[2], p[2], 0.9, 1, 0.1, 0.0, 1.0, 1, 64, 64, 5, *c, p[3], size, p[4], None]
    f = L.e8q_orthogonal_step
    for args in (_with(base, a0=None), _with(base, a1=None), _with(base, a4=None), _with(base, a5=None),
                 _with(base, a1=p[1]), _with(base, a5=p[1]), _with(base, a5=p[0]), _with(base, a6=float("inf")),
                 _with(base, a8=float("nan")), _with(base, a18=None), _with(base, a3=9)):
        assert f(*args) == INVALID, args
