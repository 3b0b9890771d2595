"""CPU checks of sizes at the operators' limits: what a launch could not hold is
refused on the host (the pointers are never followed)."""

import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(0x10000)
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def L():
    import bit_e8_lattice_amd as e8q
    if not os.path.exists(e8q.library_path):
        from bit_e8_lattice_amd.build import build
        build()
    return e8q.lib()


@pytest.mark.parametrize("dtype,rows,vocab", [(1, 1 << 22, 32769), (1, 1 << 23, 131072), (0, 1 << 22, 32769),
                                              (0, 1 << 23, 16385), (0, (1 << 24) - 1, 20000)])
def test_rows_past_the_threads_of_a_launch(L, dtype, rows, vocab):
    # logits, dtype, rows, vocab, stride, scale, tokens, index, n, g, g_entropy, logprob, lse, entropy, dx, dx_stride, ws, bytes,
    # status, stream
    args = [FAKE, dtype, rows, vocab, vocab, 1.0, FAKE, 0, 1, FAKE, None, FAKE, None, None, FAKE, vocab, None, 0, FAKE, None]
    assert L.e8q_token_logprobs_grad(*args) == UNSUPPORTED


@pytest.mark.parametrize("vocab,dim", [(100, 16), (1024, 300), (131072, 4096)])
def test_embedding_workspace_serves_smaller_batches(L, vocab, dim):
    sizes = [L.e8q_embed_backward_workspace_size(n, vocab, dim)
             for n in list(range(1, 9000, 7)) + list(range(9000, 400000, 997))]
    assert sizes[0] > 0 and sizes == sorted(sizes)
