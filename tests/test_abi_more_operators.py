"""CPU checks of further C entry points: bad arguments are refused on the host,
before anything is launched (the pointers are never followed)."""

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


def test_distill_rejects(L):
    # logits, dtype, rows, vocab, stride, scale, idx, index, logprob, k, tail, loss, logprob_out, stats, ws, bytes, status, stream
    base = [FAKE, 1, 4, 100, 100, 1.0, FAKE, 1, FAKE, 5, 2, FAKE, FAKE, FAKE, None, 0, FAKE, None]
    f = L.e8q_distill
    for args in (_with(base, a0=None), _with(base, a1=2), _with(base, a2=0), _with(base, a3=0), _with(base, a4=99),
                 _with(base, a5=0.0), _with(base, a5=-1.0), _with(base, a5=float("inf")), _with(base, a5=float("nan")),
                 _with(base, a6=None), _with(base, a7=2), _with(base, a8=None), _with(base, a9=0), _with(base, a9=-1),
                 _with(base, a10=3), _with(base, a10=-1), _with(base, a11=None, a12=None, a13=None),
                 _with(base, a13=ctypes.c_void_p(0x10008)), _with(base, a16=None), _with(base, a0=ODD),
                 _with(base, a6=ctypes.c_void_p(0x10004)), _with(base, a8=ODD)):
        assert f(*args) == INVALID, args
    for args in (_with(base, a9=1025), _with(base, a2=1 << 24), _with(base, a3=(1 << 31) - 16, a4=1 << 31),
                 _with(base, a4=1 << 40)):
        assert f(*args) == UNSUPPORTED, args
    # few long rows are split and need the workspace
    need = L.e8q_distill_workspace_size(1, 131072, 5)
    assert need > 0 and L.e8q_distill_workspace_size(8192, 131072, 64) == 0
    long = _with(base, a2=1, a3=131072, a4=131072, a14=FAKE, a15=need)
    for args in (_with(long, a14=None), _with(long, a15=0), _with(long, a14=ctypes.c_void_p(0x10010))):
        assert f(*args) == INVALID, args
    for bad in ((0, 10, 1), (1, 0, 1), (1, 10, 0), (1, 10, 1025), (1 << 24, 10, 1), (1, 1 << 31, 1)):
        assert L.e8q_distill_workspace_size(*bad) == 0


def test_distill_gradients_reject(L):
    # logits, dtype, rows, vocab, stride, scale, idx, index, logprob, k, tail, stats, g, dx, dx_stride, status, stream
    base = [FAKE, 0, 4, 100, 100, 1.0, FAKE, 0, FAKE, 5, 0, FAKE, FAKE, FAKE, 100, FAKE, None]
    f = L.e8q_distill_backward
    for args in (_with(base, a11=None), _with(base, a11=ctypes.c_void_p(0x10004)), _with(base, a12=None),
                 _with(base, a13=None), _with(base, a13=ODD), _with(base, a14=99), _with(base, a14=101),
                 _with(base, a15=None), _with(base, a10=9)):
        assert f(*args) == INVALID, args               # (dx is logits: the strides have to agree)
    assert f(*_with(base, a13=ctypes.c_void_p(0x20000), a14=1 << 40)) == UNSUPPORTED
    # logits, dtype, rows, vocab, stride, scale, idx, index, logprob, k, tail, g, loss, logprob_out, dx, dx_stride, ws, bytes,
    # status, stream
    base = [FAKE, 0, 4, 100, 100, 1.0, FAKE, 0, FAKE, 5, 0, FAKE, None, None, FAKE, 100, None, 0, FAKE, None]
    f = L.e8q_distill_grad
    for args in (_with(base, a11=None), _with(base, a14=None), _with(base, a15=99), _with(base, a15=101),
                 _with(base, a18=None), _with(base, a2=1, a3=131072, a4=131072, a15=131072)):
        assert f(*args) == INVALID, args
    # 2^32 threads
    assert f(*_with(base, a2=1 << 22, a3=40000, a4=40000, a15=40000)) == UNSUPPORTED


def test_adjust_rejects(L):
    # logits, dtype, rows, vocab, stride, index, history, cols, hstride, hlen, plen, rep, freq, pres, bias_idx, bias, n, bstride,
    # mask, mstride, out, ostride, status, stream
    base = [FAKE, 1, 4, 100, 100, 0, FAKE, 9, 9, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 3, 3, FAKE, 4, FAKE, 100, FAKE, None]
    f = L.e8q_adjust_logits
    for args in (_with(base, a0=None), _with(base, a1=2), _with(base, a2=0), _with(base, a3=0), _with(base, a4=99),
                 _with(base, a5=2), _with(base, a6=None), _with(base, a7=0), _with(base, a8=8),
                 _with(base, a11=None, a12=None, a13=None), _with(base, a6=None, a11=None, a12=None, a13=None),
                 _with(base, a14=None), _with(base, a15=None), _with(base, a16=0), _with(base, a16=-1),
                 _with(base, a17=2), _with(base, a19=3), _with(base, a20=None), _with(base, a21=99),
                 _with(base, a21=101), _with(base, a22=None), _with(base, a0=ODD), _with(base, a20=ODD),
                 _with(base, a5=1, a6=ctypes.c_void_p(0x10004)), _with(base, a11=ODD), _with(base, a18=ODD)):
        assert f(*args) == INVALID, args
    big = _with(base, a6=None, a9=None, a10=None, a11=None, a12=None, a13=None)
    for args in (_with(base, a16=1025, a17=1025), _with(base, a2=1 << 24), _with(base, a7=1 << 30, a8=1 << 30),
                 _with(base, a4=1 << 40, a21=1 << 40), _with(big, a2=1 << 22, a3=16384, a4=16384, a19=0, a21=16384),
                 _with(base, a3=(1 << 31) - 16, a4=1 << 31, a19=0, a21=1 << 31)):
        assert f(*args) == UNSUPPORTED, args


def test_moe_rejects(L):
    import bit_e8_lattice_amd as e8q
    ok = e8q._ExpertsStruct(0x10000, 0x10000, 5, 0x10000, 0x10000)
    ref = ctypes.addressof
    P = lambda v: ctypes.c_void_p(v)  # noqa: E731
    need = L.e8q_moe_workspace_size(8, 256, 64, 4, 2)
    assert need > 0
    # gate, up, down, experts, hidden, inter, bound, signs_in, had, signs_down, had, act, x, dtype, tokens, router, dtype, k,
    # normalize, idx, weight, y, dtype, ws, bytes, status, stream
    base = [ref(ok), ref(ok), ref(ok), 8, 256, 64, 16, FAKE, 128, FAKE, 64, 0, FAKE, 1, 4, FAKE, 1, 2, 1, FAKE, FAKE, FAKE,
            1, FAKE, need, FAKE, None]
    f = L.e8q_moe_core_escape
    structs = [e8q._ExpertsStruct(*v) for v in ((0, 0x10000, 5, 0x10000, 0x10000), (0x10001, 0x10000, 5, 0x10000, 0x10000),
                                                (0x10000, 0, 5, 0x10000, 0x10000), (0x10000, 0x10000, -1, 0x10000, 0x10000),
                                                (0x10000, 0x10002, 5, 0x10000, 0x10000), (0x10000, 0x10000, 5, 0, 0x10000),
                                                (0x10000, 0x10000, 5, 0x10004, 0x10000), (0x10000, 0x10000, 5, 0x10000, 0))]
    bad = [_with(base, **{f"a{i}": ref(s)}) for s in structs for i in range(3)]
    bad += [_with(base, **{f"a{i}": None}) for i in (0, 1, 2, 12, 19, 20, 21, 23, 25)]
    bad += [_with(base, a3=0), _with(base, a4=0), _with(base, a4=252), _with(base, a5=0), _with(base, a5=60),
            _with(base, a6=-1), _with(base, a6=41), _with(base, a8=96), _with(base, a8=512), _with(base, a10=128),
            _with(base, a11=2), _with(base, a13=2), _with(base, a14=0), _with(base, a16=3), _with(base, a17=0),
            _with(base, a17=9), _with(base, a22=7), _with(base, a24=need - 1), _with(base, a23=P(0x10010)),
            _with(base, a7=P(0x10004)), _with(base, a9=P(0x10004)), _with(base, a12=ODD), _with(base, a15=ODD),
            _with(base, a21=ODD), _with(base, a19=P(0x10002)), _with(base, a20=P(0x10002))]
    for args in bad:
        assert f(*args) == INVALID, args
    for args in (_with(base, a3=1025), _with(base, a4=32896), _with(base, a5=32832), _with(base, a14=2049),
                 _with(base, a3=1024, a17=65)):
        assert f(*args) == UNSUPPORTED, args
    for args in ((0, 256, 64, 4, 2), (8, 252, 64, 4, 2), (8, 256, 64, 0, 2), (8, 256, 64, 4, 9), (8, 256, 64, 2049, 2),
                 (1025, 256, 64, 4, 2), (8, 32776, 64, 4, 2)):
        assert L.e8q_moe_workspace_size(*args) == 0
    # host memory is read for the structs only; enough for fewer tokens too
    assert all(L.e8q_moe_workspace_size(8, 256, 64, t, 2) <= need for t in (1, 2, 3))
