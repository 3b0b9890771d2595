"""bit_e8_lattice_amd -- MI355X (gfx950) E8 lattice projection for E8-QAT.

A thin ctypes binding over ``libe8q.so`` (C ABI in ``include/e8q.h``).  The
Python functions carry the same names as the C entry points and only marshal
arguments: torch tensors supply device memory and the current HIP stream; every
step of the computation runs in the library's HIP kernels.  Nothing here falls
back to the CPU: if the library is missing, calls raise.
"""

import ctypes
import os

import torch

__all__ = [
    "E8QError", "lib", "library_path",
    "e8q_project", "e8q_project_hadamard", "e8q_project_hadamard_restore", "e8q_sgd_project_hadamard",
    "e8q_sgd_project_hadamard_restore", "e8q_sgd_rotated_project_hadamard",
    "e8q_encode_core_escape", "e8q_encode_workspace_size", "e8q_encode_core_escape_noalloc",
    "ENCODE_NOALLOC_SCRATCH_BYTES", "e8q_ste_backward",
    "e8q_ste_backward_hadamard", "e8q_decode_core_escape", "e8q_decode_workspace_size",
    "e8q_gemv_core_escape", "e8q_gemv_workspace_size", "Experts", "e8q_moe_core_escape", "e8q_moe_workspace_size",
    "ACT_SILU", "ACT_GELU_TANH", "e8q_pack_escapes", "e8q_unpack_escapes",
    "e8q_pack_workspace_size", "PACKED_RECORD_BYTES", "e8q_ptq_init", "e8q_ptq_workspace_size",
    "e8q_token_logprobs", "e8q_token_logprobs_workspace_size", "e8q_token_logprobs_backward",
    "e8q_token_logprobs_grad", "e8q_adjust_logits", "e8q_distill", "e8q_distill_workspace_size", "e8q_distill_backward",
    "e8q_distill_grad", "TAIL_NONE", "TAIL_RENORM", "TAIL_REST", "e8q_embed", "e8q_embed_backward",
    "e8q_embed_backward_workspace_size",
    "e8q_orthogonalize", "e8q_orthogonal_step", "e8q_orthogonalize_workspace_size", "NEWTON_SCHULZ",
    "e8q_core_size",
    "e8q_status_string", "e8q_version",
    "ESCAPE_RECORD_BYTES", "STATUS_BITS", "F32", "BF16", "I32", "I64",
]

F32, BF16 = 0, 1
I32, I64 = 0, 1
TAIL_NONE, TAIL_RENORM, TAIL_REST = 0, 1, 2
ACT_SILU, ACT_GELU_TANH = 0, 1
# sigma -> a sigma + b sigma^3 + c sigma^5: five steps bring singular values in [0.01, 1] into [0.68, 1.14]
# (coefficients published by K. Jordan and others, 2024)
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)
ESCAPE_RECORD_BYTES = 20
ENCODE_NOALLOC_SCRATCH_BYTES = 64 << 20      # E8Q_ENCODE_NOALLOC_SCRATCH_BYTES
PACKED_RECORD_BYTES = 8
STATUS_BITS = {
    "NONFINITE": 1, "BAD_SCALE": 2, "INT8_RANGE": 4, "ESC_OVERFLOW": 8,
    "X_RANGE": 16, "LOOKBACK_TIMEOUT": 32, "BAD_INDEX": 64, "ESC_MISSING": 128,
}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libe8q.so")
_lib = None


class E8QError(RuntimeError):
    def __init__(self, fn, code):
        msg = lib().e8q_status_string(code).decode() if _lib is not None else str(code)
        super().__init__(f"{fn} failed: {msg} (code {code})")
        self.code = code


def lib():
    """Load ``libe8q.so`` (built in-tree by ``bit_e8_lattice_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: run `python -m bit_e8_lattice_amd.build`")
    L = ctypes.CDLL(library_path)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    e = ctypes.c_int
    L.e8q_project.argtypes = [vp, e, i64, i64, i64, vp, vp, e, vp, i32, vp, vp, vp]
    L.e8q_project.restype = e
    L.e8q_project_hadamard.argtypes = [vp, e, i64, i64, i64, vp, vp, i32, vp, e, vp, vp, i32, vp, vp, vp]
    L.e8q_project_hadamard.restype = e
    L.e8q_project_hadamard_restore.argtypes = [vp, e, i64, i64, i64, vp, vp, i32, vp, e, vp, i32, vp, vp, vp]
    L.e8q_project_hadamard_restore.restype = e
    L.e8q_ste_backward_hadamard.argtypes = [vp, e, i64, i64, vp, i32, vp, vp, f32, vp]
    L.e8q_ste_backward_hadamard.restype = e
    L.e8q_decode_core_escape.argtypes = [vp, vp, i64, vp, i64, i64, i64, i32, vp, vp, i32, vp, vp, e, vp, e,
                                         vp, sz, vp, vp]
    L.e8q_decode_core_escape.restype = e
    L.e8q_decode_workspace_size.argtypes = [i64]
    L.e8q_decode_workspace_size.restype = sz
    L.e8q_gemv_core_escape.argtypes = [vp, vp, i64, vp, i64, i64, i64, i32, vp, vp, i32, vp, e, i64, vp,
                                       vp, sz, vp, vp]
    L.e8q_gemv_core_escape.restype = e
    L.e8q_gemv_workspace_size.argtypes = [i64, i64, i64, i64]
    L.e8q_gemv_workspace_size.restype = sz
    L.e8q_moe_core_escape.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, i32, vp, i32, i32, vp, e, i64, vp, e, i64, i32,
                                      vp, vp, vp, e, vp, sz, vp, vp]
    L.e8q_moe_core_escape.restype = e
    L.e8q_moe_workspace_size.argtypes = [i64, i64, i64, i64, i64]
    L.e8q_moe_workspace_size.restype = sz
    L.e8q_pack_escapes.argtypes = [vp, i64, i32, vp, vp, i64, vp, vp, sz, vp, vp]
    L.e8q_pack_escapes.restype = e
    L.e8q_unpack_escapes.argtypes = [vp, i64, vp, i64, i32, vp, vp, sz, vp, vp]
    L.e8q_unpack_escapes.restype = e
    L.e8q_pack_workspace_size.argtypes = [i64]
    L.e8q_pack_workspace_size.restype = sz
    L.e8q_ptq_init.argtypes = [vp, e, i64, i64, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.e8q_ptq_init.restype = e
    L.e8q_ptq_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_ptq_workspace_size.restype = sz
    L.e8q_encode_core_escape.argtypes = [vp, e, i64, i64, i64, vp, vp, i32, i32, vp, vp, i64, vp, vp,
                                         vp, sz, vp, vp]
    L.e8q_encode_core_escape.restype = e
    L.e8q_encode_core_escape_noalloc.argtypes = [vp, e, i64, i64, i64, vp, vp, i32, i32, vp, vp, i64, vp, vp,
                                                 vp, vp]
    L.e8q_encode_core_escape_noalloc.restype = e
    L.e8q_encode_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_encode_workspace_size.restype = sz
    L.e8q_sgd_project_hadamard.argtypes = [vp, vp, f32, i64, i64, i64, vp, vp, i32, vp, e, vp, i32, vp, vp, vp]
    L.e8q_sgd_project_hadamard.restype = e
    L.e8q_sgd_project_hadamard_restore.argtypes = [vp, vp, f32, i64, i64, i64, vp, vp, i32, vp, e, vp, i32, vp, vp,
                                                   vp]
    L.e8q_sgd_project_hadamard_restore.restype = e
    L.e8q_sgd_rotated_project_hadamard.argtypes = [vp, vp, f32, i64, i64, i64, vp, vp, i32, vp, e, vp, i32, vp, vp,
                                                   vp]
    L.e8q_sgd_rotated_project_hadamard.restype = e
    L.e8q_ste_backward.argtypes = [vp, vp, vp, f32, e, i64, vp]
    L.e8q_ste_backward.restype = e
    L.e8q_token_logprobs.argtypes = [vp, e, i64, i64, i64, f32, vp, e, i64, vp, vp, vp, i64, vp, vp, vp, sz, vp, vp]
    L.e8q_token_logprobs.restype = e
    L.e8q_token_logprobs_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_token_logprobs_workspace_size.restype = sz
    L.e8q_token_logprobs_backward.argtypes = [vp, e, i64, i64, i64, f32, vp, e, i64, vp, vp, vp, vp, vp, i64, vp, vp]
    L.e8q_token_logprobs_backward.restype = e
    L.e8q_token_logprobs_grad.argtypes = [vp, e, i64, i64, i64, f32, vp, e, i64, vp, vp, vp, vp, vp, vp, i64,
                                          vp, sz, vp, vp]
    L.e8q_token_logprobs_grad.restype = e
    L.e8q_adjust_logits.argtypes = [vp, e, i64, i64, i64, e, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, i64, i64, vp, i64,
                                    vp, i64, vp, vp]
    L.e8q_adjust_logits.restype = e
    L.e8q_distill.argtypes = [vp, e, i64, i64, i64, f32, vp, e, vp, i64, i32, vp, vp, vp, vp, sz, vp, vp]
    L.e8q_distill.restype = e
    L.e8q_distill_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_distill_workspace_size.restype = sz
    L.e8q_distill_backward.argtypes = [vp, e, i64, i64, i64, f32, vp, e, vp, i64, i32, vp, vp, vp, i64, vp, vp]
    L.e8q_distill_backward.restype = e
    L.e8q_distill_grad.argtypes = [vp, e, i64, i64, i64, f32, vp, e, vp, i64, i32, vp, vp, vp, vp, i64, vp, sz, vp, vp]
    L.e8q_distill_grad.restype = e
    L.e8q_embed.argtypes = [vp, e, i64, i64, vp, e, i64, f32, vp, e, vp, vp]
    L.e8q_embed.restype = e
    L.e8q_embed_backward.argtypes = [vp, e, i64, i64, vp, e, i64, f32, vp, e, vp, f32, vp, sz, vp, vp]
    L.e8q_embed_backward.restype = e
    L.e8q_embed_backward_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_embed_backward_workspace_size.restype = sz
    L.e8q_orthogonalize.argtypes = [vp, e, i64, i64, i64, i32, f32, f32, f32, vp, vp, sz, vp, vp]
    L.e8q_orthogonalize.restype = e
    L.e8q_orthogonal_step.argtypes = [vp, vp, vp, e, vp, vp, f32, i32, f32, f32, f32, i64, i64, i64,
                                      i32, f32, f32, f32, vp, sz, vp, vp]
    L.e8q_orthogonal_step.restype = e
    L.e8q_orthogonalize_workspace_size.argtypes = [i64, i64, i64]
    L.e8q_orthogonalize_workspace_size.restype = sz
    L.e8q_core_size.argtypes = [i32]
    L.e8q_core_size.restype = i64
    L.e8q_status_string.argtypes = [e]
    L.e8q_status_string.restype = ctypes.c_char_p
    L.e8q_version.argtypes = []
    L.e8q_version.restype = ctypes.c_char_p
    _lib = L
    return L


# ------------------------------------------------------------------ marshalling

def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev(t, name, dtypes=None):
    if t is None or (type(t) is torch.Tensor and t.is_cuda and t.dtype in (dtypes or (t.dtype,)) and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")


def _dtype_code(t):
    return BF16 if t.dtype == torch.bfloat16 else F32


def _shape3(w):
    if w.dim() == 2:
        return 1, w.shape[0], w.shape[1]
    if w.dim() == 3:
        return tuple(w.shape)
    raise ValueError("weights must be [rows, cols] or [batch, rows, cols]")


def _stream(t, stream):
    if stream is None:
        # the handle that torch.cuda.current_stream(t.device).cuda_stream gives, without the 1.8 us that
        # making its Stream object takes (a call of a small operator takes 5.6 us in all)
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream


def _check(fn, code):
    if code != 0:
        raise E8QError(fn, code)


_WDT = (torch.float32, torch.bfloat16)


def e8q_project(w, row_scale, status, q_out=None, two_z_out=None, core_bound=-1,
                esc_count_out=None, stream=None):
    """``e8q_project``: q = s * nearest_E8(w / s) per 8-column group (no rotation)."""
    _dev(w, "w", _WDT); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(q_out, "q_out", _WDT); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    b, r, c = _shape3(w)
    code = lib().e8q_project(_ptr(w), _dtype_code(w), b, r, c, _ptr(row_scale), _ptr(q_out),
                             _dtype_code(q_out) if q_out is not None else F32, _ptr(two_z_out),
                             int(core_bound), _ptr(esc_count_out), _ptr(status), _stream(w, stream))
    _check("e8q_project", code)


def e8q_project_hadamard(w, row_scale, signs, had_block, status, q_out=None, two_z_out=None,
                         rotated_out=None, core_bound=-1, esc_count_out=None, stream=None):
    """``e8q_project_hadamard``: sign flip + blockwise Walsh-Hadamard, then project."""
    _dev(w, "w", _WDT); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(signs, "signs", (torch.int8,)); _dev(q_out, "q_out", _WDT)
    _dev(two_z_out, "two_z_out", (torch.int8,)); _dev(rotated_out, "rotated_out", (torch.float32,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    b, r, c = _shape3(w)
    code = lib().e8q_project_hadamard(_ptr(w), _dtype_code(w), b, r, c, _ptr(row_scale), _ptr(signs),
                                      int(had_block), _ptr(q_out),
                                      _dtype_code(q_out) if q_out is not None else F32,
                                      _ptr(two_z_out), _ptr(rotated_out), int(core_bound),
                                      _ptr(esc_count_out), _ptr(status), _stream(w, stream))
    _check("e8q_project_hadamard", code)


def e8q_sgd_project_hadamard(w_latent, grad, lr, row_scale, status, signs=None, had_block=0, q_out=None,
                             two_z_out=None, core_bound=-1, esc_count_out=None, stream=None):
    """``e8q_sgd_project_hadamard``: the identity STE with SGD on the bf16
    latents (in place), then the projection of the updated latents."""
    _dev(w_latent, "w_latent", (torch.bfloat16,)); _dev(grad, "grad", (torch.bfloat16,))
    _dev(row_scale, "row_scale", (torch.float32,)); _dev(signs, "signs", (torch.int8,))
    _dev(q_out, "q_out", _WDT); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    if grad.shape != w_latent.shape:
        raise ValueError("grad must have the shape of w_latent")
    b, r, c = _shape3(w_latent)
    code = lib().e8q_sgd_project_hadamard(_ptr(w_latent), _ptr(grad), float(lr), b, r, c, _ptr(row_scale),
                                          _ptr(signs), int(had_block), _ptr(q_out),
                                          _dtype_code(q_out) if q_out is not None else F32,
                                          _ptr(two_z_out), int(core_bound), _ptr(esc_count_out), _ptr(status),
                                          _stream(w_latent, stream))
    _check("e8q_sgd_project_hadamard", code)


def e8q_sgd_rotated_project_hadamard(w_latent, grad_q, lr, row_scale, signs, had_block, status, q_out=None,
                                     two_z_out=None, core_bound=-1, esc_count_out=None, stream=None):
    """``e8q_sgd_rotated_project_hadamard``: the rotated-basis gradient taken
    back through the rotation, SGD on the bf16 latents (in place), then the
    rotated projection of the updated latents."""
    _dev(w_latent, "w_latent", (torch.bfloat16,)); _dev(grad_q, "grad_q", (torch.bfloat16,))
    _dev(row_scale, "row_scale", (torch.float32,)); _dev(signs, "signs", (torch.int8,))
    _dev(q_out, "q_out", _WDT); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    if grad_q.shape != w_latent.shape:
        raise ValueError("grad_q must have the shape of w_latent")
    b, r, c = _shape3(w_latent)
    code = lib().e8q_sgd_rotated_project_hadamard(_ptr(w_latent), _ptr(grad_q), float(lr), b, r, c, _ptr(row_scale),
                                                  _ptr(signs), int(had_block), _ptr(q_out),
                                                  _dtype_code(q_out) if q_out is not None else F32,
                                                  _ptr(two_z_out), int(core_bound), _ptr(esc_count_out), _ptr(status),
                                                  _stream(w_latent, stream))
    _check("e8q_sgd_rotated_project_hadamard", code)


def e8q_sgd_project_hadamard_restore(w_latent, grad, lr, row_scale, signs, had_block, w_hat_out, status,
                                     two_z_out=None, core_bound=-1, esc_count_out=None, stream=None):
    """``e8q_sgd_project_hadamard_restore``: the identity STE with SGD on the
    bf16 latents (in place), then the projection of the updated latents
    restored to the original basis (``w_hat_out`` float32 or bf16)."""
    _dev(w_latent, "w_latent", (torch.bfloat16,)); _dev(grad, "grad", (torch.bfloat16,))
    _dev(row_scale, "row_scale", (torch.float32,)); _dev(signs, "signs", (torch.int8,))
    _dev(w_hat_out, "w_hat_out", _WDT); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    if w_hat_out is None:
        raise ValueError("w_hat_out is required")
    if grad.shape != w_latent.shape:
        raise ValueError("grad must have the shape of w_latent")
    b, r, c = _shape3(w_latent)
    code = lib().e8q_sgd_project_hadamard_restore(_ptr(w_latent), _ptr(grad), float(lr), b, r, c, _ptr(row_scale),
                                                  _ptr(signs), int(had_block), _ptr(w_hat_out),
                                                  _dtype_code(w_hat_out), _ptr(two_z_out), int(core_bound),
                                                  _ptr(esc_count_out), _ptr(status), _stream(w_latent, stream))
    _check("e8q_sgd_project_hadamard_restore", code)


def e8q_project_hadamard_restore(w, row_scale, signs, had_block, w_hat_out, status, two_z_out=None,
                                 core_bound=-1, esc_count_out=None, stream=None):
    """``e8q_project_hadamard_restore``: the projection rotated back to the
    original basis (``w_hat_out`` float32 or bf16, shaped like ``w``)."""
    _dev(w, "w", _WDT); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(signs, "signs", (torch.int8,)); _dev(w_hat_out, "w_hat_out", _WDT)
    _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(esc_count_out, "esc_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    if w_hat_out is None:
        raise ValueError("w_hat_out is required")
    b, r, c = _shape3(w)
    code = lib().e8q_project_hadamard_restore(_ptr(w), _dtype_code(w), b, r, c, _ptr(row_scale),
                                              _ptr(signs), int(had_block), _ptr(w_hat_out),
                                              _dtype_code(w_hat_out), _ptr(two_z_out), int(core_bound),
                                              _ptr(esc_count_out), _ptr(status), _stream(w, stream))
    _check("e8q_project_hadamard_restore", code)


def e8q_encode_workspace_size(batch, rows, cols):
    return int(lib().e8q_encode_workspace_size(batch, rows, cols))


def e8q_encode_core_escape(w, row_scale, core_bound, core_idx_out, esc_out, esc_count_out,
                           workspace, status, signs=None, had_block=0, two_z_out=None, stream=None):
    """``e8q_encode_core_escape``: core indices (uint16 stored in an int16 tensor)
    plus escape records (``esc_out``: uint8 tensor of 20-byte records)."""
    _dev(w, "w", _WDT); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(signs, "signs", (torch.int8,)); _dev(core_idx_out, "core_idx_out", (torch.int16,))
    _dev(esc_out, "esc_out", (torch.uint8,)); _dev(esc_count_out, "esc_count_out", (torch.int64,))
    _dev(workspace, "workspace", (torch.uint8,)); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(status, "status", (torch.int32,))
    b, r, c = _shape3(w)
    cap = 0 if esc_out is None else esc_out.numel() // ESCAPE_RECORD_BYTES
    code = lib().e8q_encode_core_escape(_ptr(w), _dtype_code(w), b, r, c, _ptr(row_scale), _ptr(signs),
                                        int(had_block), int(core_bound), _ptr(core_idx_out),
                                        _ptr(esc_out), cap, _ptr(esc_count_out), _ptr(two_z_out),
                                        _ptr(workspace), workspace.numel(), _ptr(status),
                                        _stream(w, stream))
    _check("e8q_encode_core_escape", code)


def e8q_encode_core_escape_noalloc(w, row_scale, core_bound, core_idx_out, esc_out, esc_count_out,
                                   status, signs=None, had_block=0, two_z_out=None, stream=None):
    """``e8q_encode_core_escape_noalloc``: ``e8q_encode_core_escape`` without a
    workspace (the library's fixed per-GPU scratch; calls that overlap on one
    GPU race)."""
    _dev(w, "w", _WDT); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(signs, "signs", (torch.int8,)); _dev(core_idx_out, "core_idx_out", (torch.int16,))
    _dev(esc_out, "esc_out", (torch.uint8,)); _dev(esc_count_out, "esc_count_out", (torch.int64,))
    _dev(two_z_out, "two_z_out", (torch.int8,)); _dev(status, "status", (torch.int32,))
    b, r, c = _shape3(w)
    cap = 0 if esc_out is None else esc_out.numel() // ESCAPE_RECORD_BYTES
    code = lib().e8q_encode_core_escape_noalloc(_ptr(w), _dtype_code(w), b, r, c, _ptr(row_scale), _ptr(signs),
                                                int(had_block), int(core_bound), _ptr(core_idx_out),
                                                _ptr(esc_out), cap, _ptr(esc_count_out), _ptr(two_z_out),
                                                _ptr(status), _stream(w, stream))
    _check("e8q_encode_core_escape_noalloc", code)


def e8q_ste_backward(grad_q, grad_w=None, w_latent=None, lr=1.0, stream=None):
    """``e8q_ste_backward``: identity STE copy and/or fused SGD on the latents."""
    _dev(grad_q, "grad_q", _WDT); _dev(grad_w, "grad_w", (grad_q.dtype,))
    _dev(w_latent, "w_latent", (grad_q.dtype,))
    code = lib().e8q_ste_backward(_ptr(grad_q), _ptr(grad_w), _ptr(w_latent), float(lr),
                                  _dtype_code(grad_q), grad_q.numel(), _stream(grad_q, stream))
    _check("e8q_ste_backward", code)


def e8q_ste_backward_hadamard(grad_q, signs, had_block, grad_w=None, w_latent=None, lr=1.0, stream=None):
    """``e8q_ste_backward_hadamard``: gradient of the latents for a rotated-basis
    projection (R^T applied to ``grad_q``), and/or the fused SGD step."""
    _dev(grad_q, "grad_q", _WDT); _dev(signs, "signs", (torch.int8,))
    _dev(grad_w, "grad_w", (grad_q.dtype,)); _dev(w_latent, "w_latent", (grad_q.dtype,))
    cols = grad_q.shape[-1]
    rows = grad_q.numel() // cols
    code = lib().e8q_ste_backward_hadamard(_ptr(grad_q), _dtype_code(grad_q), rows, cols, _ptr(signs),
                                           int(had_block), _ptr(grad_w), _ptr(w_latent), float(lr),
                                           _stream(grad_q, stream))
    _check("e8q_ste_backward_hadamard", code)


def e8q_decode_workspace_size(batch):
    return int(lib().e8q_decode_workspace_size(batch))


def e8q_decode_core_escape(core_idx, esc, esc_count, shape, core_bound, workspace, status, row_scale=None,
                           signs=None, had_block=0, two_z_out=None, q_out=None, w_hat_out=None,
                           esc_records=None, stream=None):
    """``e8q_decode_core_escape``: core indices (int16 tensor of uint16 values)
    and escape records (uint8 tensor of 20-byte records) back to 2z, q
    (rotated basis) and/or w_hat (original basis), for ``shape = (batch, rows,
    cols)``.  ``esc_records`` overrides the record count taken from ``esc``."""
    _dev(core_idx, "core_idx", (torch.int16,)); _dev(esc, "esc", (torch.uint8,))
    _dev(esc_count, "esc_count", (torch.int64,)); _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,)); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(signs, "signs", (torch.int8,)); _dev(two_z_out, "two_z_out", (torch.int8,))
    _dev(q_out, "q_out", _WDT); _dev(w_hat_out, "w_hat_out", _WDT)
    b, r, c = shape
    cap = 0 if esc is None else esc.numel() // ESCAPE_RECORD_BYTES
    if esc_records is not None:
        cap = min(cap, int(esc_records))
    code = lib().e8q_decode_core_escape(
        _ptr(core_idx), _ptr(esc), cap, _ptr(esc_count), b, r, c, int(core_bound), _ptr(row_scale),
        _ptr(signs), int(had_block), _ptr(two_z_out), _ptr(q_out),
        _dtype_code(q_out) if q_out is not None else F32, _ptr(w_hat_out),
        _dtype_code(w_hat_out) if w_hat_out is not None else F32, _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(core_idx, stream))
    _check("e8q_decode_core_escape", code)


def e8q_gemv_workspace_size(batch, m, rows, cols):
    return int(lib().e8q_gemv_workspace_size(batch, m, rows, cols))


def e8q_gemv_core_escape(core_idx, esc, esc_count, shape, core_bound, row_scale, x, y_out, workspace, status,
                         signs=None, had_block=0, esc_records=None, stream=None):
    """``e8q_gemv_core_escape``: ``y_out[b, t, r] = sum_c W_hat[b, r, c] x[b, t, c]``
    from the exported form, for ``shape = (batch, rows, cols)`` and ``x``
    [batch, m, cols]."""
    _dev(core_idx, "core_idx", (torch.int16,)); _dev(esc, "esc", (torch.uint8,))
    _dev(esc_count, "esc_count", (torch.int64,)); _dev(row_scale, "row_scale", (torch.float32,))
    _dev(x, "x", _WDT); _dev(y_out, "y_out", (torch.float32,)); _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,)); _dev(signs, "signs", (torch.int8,))
    b, r, c = shape
    if x.dim() != 3 or x.shape[0] != b or x.shape[2] != c:
        raise ValueError("x must be [batch, m, cols]")
    cap = 0 if esc is None else esc.numel() // ESCAPE_RECORD_BYTES
    if esc_records is not None:
        cap = min(cap, int(esc_records))
    code = lib().e8q_gemv_core_escape(
        _ptr(core_idx), _ptr(esc), cap, _ptr(esc_count), b, r, c, int(core_bound), _ptr(row_scale), _ptr(signs),
        int(had_block), _ptr(x), _dtype_code(x), x.shape[1], _ptr(y_out), _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(core_idx, stream))
    _check("e8q_gemv_core_escape", code)


class _ExpertsStruct(ctypes.Structure):
    _fields_ = [("core_idx", ctypes.c_void_p), ("esc", ctypes.c_void_p), ("esc_capacity", ctypes.c_int64),
                ("esc_count", ctypes.c_void_p), ("row_scale", ctypes.c_void_p)]


class Experts:
    """``e8q_experts_t``: the exported form of ``shape = (experts, rows, cols)``
    matrices, as ``e8q_encode_core_escape`` writes it for that batch (the
    tensors are kept and must stay as they are)."""

    def __init__(self, core_idx, esc, esc_count, row_scale, shape, esc_records=None):
        experts, rows, cols = shape
        _sized(core_idx, "core_idx", experts * rows * cols // 8, (torch.int16,)); _dev(esc, "esc", (torch.uint8,))
        _sized(esc_count, "esc_count", experts, (torch.int64,)); _sized(row_scale, "row_scale", experts * rows)
        cap = 0 if esc is None else esc.numel() // ESCAPE_RECORD_BYTES
        if esc_records is not None:
            cap = min(cap, int(esc_records))
        self.shape, self.tensors = tuple(shape), (core_idx, esc, esc_count, row_scale)
        self.struct = _ExpertsStruct(_ptr(core_idx), _ptr(esc), cap, _ptr(esc_count), _ptr(row_scale))
        self.ref = ctypes.addressof(self.struct)


def e8q_moe_workspace_size(experts, hidden, inter, tokens, top_k):
    return int(lib().e8q_moe_workspace_size(int(experts), int(hidden), int(inter), int(tokens), int(top_k)))


def e8q_moe_core_escape(gate, up, down, core_bound, x, expert_idx, expert_weight, y_out, workspace, status, router=None,
                        signs_in=None, had_block_in=0, signs_down=None, had_block_down=0, activation=ACT_SILU,
                        normalize=True, stream=None):
    """``e8q_moe_core_escape``: a mixture-of-experts layer of ``x`` [tokens,
    hidden] from the exported form.  ``gate`` and ``up`` are ``Experts`` of
    shape (experts, inter, hidden), ``down`` of (experts, hidden, inter).  With
    ``router`` [experts, hidden] the ``expert_idx`` (int32) and
    ``expert_weight`` [tokens, k] are written; without it they are read."""
    experts, inter, hidden = gate.shape
    if up.shape != gate.shape or down.shape != (experts, hidden, inter):
        raise ValueError("gate and up must be (experts, inter, hidden), down (experts, hidden, inter)")
    _dev(x, "x", _WDT); _dev(router, "router", _WDT); _dev(y_out, "y_out", _WDT)
    if x.dim() != 2 or x.shape[1] != hidden or y_out.shape != x.shape:
        raise ValueError("x and y_out must be [tokens, hidden]")
    if router is not None and tuple(router.shape) != (experts, hidden):
        raise ValueError("router must be [experts, hidden]")
    tokens = x.shape[0]
    _dev(expert_idx, "expert_idx", (torch.int32,))
    if expert_idx.dim() != 2 or expert_idx.shape[0] != tokens:
        raise ValueError("expert_idx must be [tokens, k]")
    k = expert_idx.shape[1]
    _sized(expert_weight, "expert_weight", tokens * k)
    _sized(signs_in, "signs_in", hidden, (torch.int8,)); _sized(signs_down, "signs_down", inter, (torch.int8,))
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    code = lib().e8q_moe_core_escape(gate.ref, up.ref, down.ref, experts, hidden, inter, int(core_bound),
                                     _ptr(signs_in), int(had_block_in), _ptr(signs_down), int(had_block_down),
                                     int(activation), _ptr(x), _dtype_code(x), tokens, _ptr(router),
                                     _dtype_code(router) if router is not None else F32, k, int(bool(normalize)),
                                     _ptr(expert_idx), _ptr(expert_weight), _ptr(y_out), _dtype_code(y_out),
                                     _ptr(workspace), _size(workspace), _ptr(status), _stream(x, stream))
    _check("e8q_moe_core_escape", code)


def e8q_pack_workspace_size(n):
    return int(lib().e8q_pack_workspace_size(n))


def e8q_pack_escapes(esc, n, core_bound, packed_out, wide_out, wide_count_out, workspace, status, stream=None):
    """``e8q_pack_escapes``: ``n`` 20-byte records in ``esc`` (uint8 tensor) to
    8-byte packed records in ``packed_out`` (uint8) plus the wide list."""
    for t, nm in ((esc, "esc"), (packed_out, "packed_out"), (wide_out, "wide_out"), (workspace, "workspace")):
        _dev(t, nm, (torch.uint8,))
    _dev(wide_count_out, "wide_count_out", (torch.int64,)); _dev(status, "status", (torch.int32,))
    cap = 0 if wide_out is None else wide_out.numel() // ESCAPE_RECORD_BYTES
    code = lib().e8q_pack_escapes(_ptr(esc), int(n), int(core_bound), _ptr(packed_out), _ptr(wide_out), cap,
                                  _ptr(wide_count_out), _ptr(workspace), workspace.numel(), _ptr(status),
                                  _stream(workspace, stream))
    _check("e8q_pack_escapes", code)


def e8q_unpack_escapes(packed, n, wide, wide_count, core_bound, esc_out, workspace, status, stream=None):
    """``e8q_unpack_escapes``: packed records (+ ``wide_count`` wide records) back to
    20-byte records in ``esc_out`` (uint8)."""
    for t, nm in ((packed, "packed"), (wide, "wide"), (esc_out, "esc_out"), (workspace, "workspace")):
        _dev(t, nm, (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    code = lib().e8q_unpack_escapes(_ptr(packed), int(n), _ptr(wide), int(wide_count), int(core_bound),
                                    _ptr(esc_out), _ptr(workspace), workspace.numel(), _ptr(status),
                                    _stream(workspace, stream))
    _check("e8q_unpack_escapes", code)


def e8q_ptq_workspace_size(batch, rows, cols):
    return int(lib().e8q_ptq_workspace_size(batch, rows, cols))


def e8q_ptq_init(w, base_scale, alphas, core_bound, scale_out, core_idx_out, two_z_out, workspace, status,
                 signs=None, had_block=0, choice_out=None, err_out=None, stream=None):
    """``e8q_ptq_init``: per-row scale search over ``alphas * base_scale`` and the
    finite-core projection at the chosen scale."""
    _dev(w, "w", _WDT); _dev(base_scale, "base_scale", (torch.float32,)); _dev(alphas, "alphas", (torch.float32,))
    _dev(scale_out, "scale_out", (torch.float32,)); _dev(core_idx_out, "core_idx_out", (torch.int16,))
    _dev(two_z_out, "two_z_out", (torch.int8,)); _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,)); _dev(signs, "signs", (torch.int8,))
    _dev(choice_out, "choice_out", (torch.int32,)); _dev(err_out, "err_out", (torch.float64,))
    b, r, c = _shape3(w)
    code = lib().e8q_ptq_init(_ptr(w), _dtype_code(w), b, r, c, _ptr(base_scale), _ptr(alphas), alphas.numel(),
                              _ptr(signs), int(had_block), int(core_bound), _ptr(scale_out), _ptr(choice_out),
                              _ptr(err_out), _ptr(core_idx_out), _ptr(two_z_out), _ptr(workspace),
                              workspace.numel(), _ptr(status), _stream(w, stream))
    _check("e8q_ptq_init", code)


# ------------------------------------------------------------------ around the projection

_IDX = (torch.int32, torch.int64)


def _index_code(t):
    return I64 if t is not None and t.dtype == torch.int64 else I32


def _size(t):
    return 0 if t is None else t.numel()


def _rows(t, name, dtypes):
    """Row stride of a [rows, vocab] device tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, vocab] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _token_count(tokens, rows):
    """Tokens per row of ``tokens`` [rows] or [rows, n]."""
    _dev(tokens, "tokens", _IDX)
    if tokens is None:
        return 0
    if tokens.dim() not in (1, 2) or tokens.shape[0] != rows:
        raise ValueError("tokens must be [rows] or [rows, n]")
    return tokens.shape[1] if tokens.dim() == 2 else 1


def _sized(t, name, n, dtypes=(torch.float32,)):
    _dev(t, name, dtypes)
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, has {t.numel()}")


def e8q_token_logprobs_workspace_size(rows, vocab, top_k=0):
    return int(lib().e8q_token_logprobs_workspace_size(int(rows), int(vocab), int(top_k)))


def e8q_token_logprobs(logits, workspace, status, tokens=None, scale=1.0, logprob_out=None, lse_out=None,
                       entropy_out=None, top_idx_out=None, top_logprob_out=None, stream=None):
    """``e8q_token_logprobs``: log probabilities of ``tokens`` ([rows] or
    [rows, n], negative: ignored) under ``softmax(scale * logits)``, the rows'
    log-sum-exp and entropy, and the most likely alternatives (``top_idx_out``
    int32 and/or ``top_logprob_out`` float32, [rows, k])."""
    stride = _rows(logits, "logits", _WDT)
    rows, vocab = logits.shape
    n = _token_count(tokens, rows)
    k = 0
    for t, nm, dt in ((top_idx_out, "top_idx_out", torch.int32), (top_logprob_out, "top_logprob_out", torch.float32)):
        if t is not None:
            k = k or t.numel() // max(rows, 1)
            _sized(t, nm, rows * k, (dt,))
    _sized(logprob_out, "logprob_out", rows * n); _sized(lse_out, "lse_out", rows)
    _sized(entropy_out, "entropy_out", rows)
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    code = lib().e8q_token_logprobs(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale),
                                    _ptr(tokens) if n else None, _index_code(tokens), n, _ptr(logprob_out),
                                    _ptr(lse_out), _ptr(entropy_out), k, _ptr(top_idx_out), _ptr(top_logprob_out),
                                    _ptr(workspace), _size(workspace), _ptr(status), _stream(logits, stream))
    _check("e8q_token_logprobs", code)


def e8q_token_logprobs_backward(logits, lse, grad_logits, status, tokens=None, grad_logprob=None, scale=1.0,
                                entropy=None, grad_entropy=None, stream=None):
    """``e8q_token_logprobs_backward``: the gradient of ``sum(grad_logprob *
    logprob) + sum(grad_entropy * entropy)`` with respect to ``logits``
    (``grad_logits`` may be ``logits``)."""
    stride, gstride = _rows(logits, "logits", _WDT), _rows(grad_logits, "grad_logits", (logits.dtype,))
    rows, vocab = logits.shape
    if grad_logits.shape != logits.shape:
        raise ValueError("grad_logits must have the shape of logits")
    n = _token_count(tokens, rows)
    _sized(lse, "lse", rows); _sized(grad_logprob, "grad_logprob", rows * n); _sized(entropy, "entropy", rows)
    _sized(grad_entropy, "grad_entropy", rows); _dev(status, "status", (torch.int32,))
    if grad_entropy is None:
        entropy = None
    code = lib().e8q_token_logprobs_backward(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale),
                                             _ptr(tokens) if n else None, _index_code(tokens), n, _ptr(lse),
                                             _ptr(grad_logprob), _ptr(entropy), _ptr(grad_entropy),
                                             _ptr(grad_logits), gstride, _ptr(status), _stream(logits, stream))
    _check("e8q_token_logprobs_backward", code)


def e8q_token_logprobs_grad(logits, tokens, grad_logprob, grad_logits, workspace, status, grad_entropy=None,
                            scale=1.0, logprob_out=None, lse_out=None, entropy_out=None, stream=None):
    """``e8q_token_logprobs_grad``: log probabilities (and entropy) and, for
    upstream gradients known beforehand, the gradient of the logits in one
    call (``grad_logits`` may be ``logits``)."""
    stride, gstride = _rows(logits, "logits", _WDT), _rows(grad_logits, "grad_logits", (logits.dtype,))
    rows, vocab = logits.shape
    if grad_logits.shape != logits.shape:
        raise ValueError("grad_logits must have the shape of logits")
    n = _token_count(tokens, rows)
    _sized(grad_logprob, "grad_logprob", rows * n); _sized(grad_entropy, "grad_entropy", rows)
    _sized(logprob_out, "logprob_out", rows * n); _sized(lse_out, "lse_out", rows)
    _sized(entropy_out, "entropy_out", rows)
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    code = lib().e8q_token_logprobs_grad(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale),
                                         _ptr(tokens) if n else None, _index_code(tokens), n, _ptr(grad_logprob),
                                         _ptr(grad_entropy), _ptr(logprob_out), _ptr(lse_out), _ptr(entropy_out),
                                         _ptr(grad_logits), gstride, _ptr(workspace), _size(workspace), _ptr(status),
                                         _stream(logits, stream))
    _check("e8q_token_logprobs_grad", code)


def _row_list(t, name, rows, dtypes):
    """Columns and row stride (0: one list for all rows) of ``t`` [rows, n] or [n] with contiguous rows."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    if t.dim() not in (1, 2) or (t.dim() == 2 and t.shape[0] != rows) or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be [n] or [rows, n] with contiguous rows")
    n = t.shape[-1]
    if t.dim() == 1 or t.shape[0] == 1:
        return n, 0
    return n, t.stride(0)


def e8q_adjust_logits(logits, out, status, history=None, history_len=None, prompt_len=None, repetition=None,
                      frequency=None, presence=None, bias_idx=None, bias=None, mask=None, stream=None):
    """``e8q_adjust_logits``: ``out`` (may be ``logits``) = the logits after
    repetition, frequency and presence penalties ([rows] float32 each) for the
    tokens of ``history`` [rows, n] (``history_len`` and ``prompt_len`` [rows]
    int32), biases (``bias_idx`` and ``bias`` [rows, n], or [n] for all rows) and a
    mask of allowed tokens (int32 words [rows, words], or [words])."""
    stride, ostride = _rows(logits, "logits", _WDT), _rows(out, "out", (logits.dtype,))
    rows, vocab = logits.shape
    if out.shape != logits.shape:
        raise ValueError("out must have the shape of logits")
    if history is not None and history.dim() != 2:
        raise ValueError("history must be [rows, n]")
    hcols, hstride = _row_list(history, "history", rows, _IDX)
    if history is not None and rows > 1 and hstride < hcols:
        raise ValueError("history must have a row of its own for each row of logits")
    nb, bstride = _row_list(bias_idx, "bias_idx", rows, _IDX)
    nv, vstride = _row_list(bias, "bias", rows, (torch.float32,))
    if (nb, bstride) != (nv, vstride) or (bias_idx is None) != (bias is None):
        raise ValueError("bias_idx and bias must have the same shape and strides")
    words, mstride = _row_list(mask, "mask", rows, (torch.int32,))
    if mask is not None and words < (vocab + 31) // 32:
        raise ValueError(f"mask must have {(vocab + 31) // 32} words a row, has {words}")
    if history is not None and bias_idx is not None and history.dtype != bias_idx.dtype:
        raise TypeError("history and bias_idx must have one dtype")
    _sized(history_len, "history_len", rows, (torch.int32,)); _sized(prompt_len, "prompt_len", rows, (torch.int32,))
    _sized(repetition, "repetition", rows); _sized(frequency, "frequency", rows); _sized(presence, "presence", rows)
    _dev(status, "status", (torch.int32,))
    if repetition is None and frequency is None and presence is None:
        history = history_len = prompt_len = None
    if history is not None and hcols == 0:
        history = history_len = prompt_len = repetition = frequency = presence = None
    code = lib().e8q_adjust_logits(_ptr(logits), _dtype_code(logits), rows, vocab, stride,
                                   _index_code(history if history is not None else bias_idx), _ptr(history), hcols,
                                   max(hstride, hcols), _ptr(history_len), _ptr(prompt_len), _ptr(repetition),
                                   _ptr(frequency), _ptr(presence), _ptr(bias_idx) if nb else None,
                                   _ptr(bias) if nb else None, nb, bstride, _ptr(mask), mstride, _ptr(out), ostride,
                                   _ptr(status), _stream(logits, stream))
    _check("e8q_adjust_logits", code)


def e8q_distill_workspace_size(rows, vocab, k):
    return int(lib().e8q_distill_workspace_size(int(rows), int(vocab), int(k)))


def _places(logits, teacher_idx, teacher_logprob):
    """Rows, vocabulary and places of a distillation call."""
    rows, vocab = logits.shape
    _dev(teacher_idx, "teacher_idx", _IDX)
    if teacher_idx.dim() != 2 or teacher_idx.shape[0] != rows:
        raise ValueError("teacher_idx must be [rows, k]")
    _sized(teacher_logprob, "teacher_logprob", teacher_idx.numel())
    return rows, vocab, teacher_idx.shape[1]


def e8q_distill(logits, teacher_idx, teacher_logprob, workspace, status, scale=1.0, tail=TAIL_NONE, loss_out=None,
                logprob_out=None, stats_out=None, stream=None):
    """``e8q_distill``: the divergence of ``softmax(scale * logits)`` from a
    teacher's top logits (``teacher_idx`` [rows, k], negative: not used;
    ``teacher_logprob`` [rows, k]) per row, the student's log probabilities at
    the places, and the statistics for the backward call (``stats_out``
    [rows, 4]).  ``tail``: ``TAIL_NONE``, ``TAIL_RENORM`` or ``TAIL_REST``."""
    stride = _rows(logits, "logits", _WDT)
    rows, vocab, k = _places(logits, teacher_idx, teacher_logprob)
    _sized(loss_out, "loss_out", rows); _sized(logprob_out, "logprob_out", rows * k)
    _sized(stats_out, "stats_out", rows * 4)
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    code = lib().e8q_distill(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale), _ptr(teacher_idx),
                             _index_code(teacher_idx), _ptr(teacher_logprob), k, int(tail), _ptr(loss_out),
                             _ptr(logprob_out), _ptr(stats_out), _ptr(workspace), _size(workspace), _ptr(status),
                             _stream(logits, stream))
    _check("e8q_distill", code)


def e8q_distill_backward(logits, teacher_idx, teacher_logprob, stats, grad_loss, grad_logits, status, scale=1.0,
                         tail=TAIL_NONE, stream=None):
    """``e8q_distill_backward``: the gradient of ``sum(grad_loss * loss)`` with
    respect to ``logits`` (``grad_logits`` may be ``logits``)."""
    stride, gstride = _rows(logits, "logits", _WDT), _rows(grad_logits, "grad_logits", (logits.dtype,))
    rows, vocab, k = _places(logits, teacher_idx, teacher_logprob)
    if grad_logits.shape != logits.shape:
        raise ValueError("grad_logits must have the shape of logits")
    _sized(stats, "stats", rows * 4); _sized(grad_loss, "grad_loss", rows); _dev(status, "status", (torch.int32,))
    code = lib().e8q_distill_backward(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale),
                                      _ptr(teacher_idx), _index_code(teacher_idx), _ptr(teacher_logprob), k, int(tail),
                                      _ptr(stats), _ptr(grad_loss), _ptr(grad_logits), gstride, _ptr(status),
                                      _stream(logits, stream))
    _check("e8q_distill_backward", code)


def e8q_distill_grad(logits, teacher_idx, teacher_logprob, grad_loss, grad_logits, workspace, status, scale=1.0,
                     tail=TAIL_NONE, loss_out=None, logprob_out=None, stream=None):
    """``e8q_distill_grad``: loss and, for row weights known beforehand, the
    gradient of the logits in one call (``grad_logits`` may be ``logits``)."""
    stride, gstride = _rows(logits, "logits", _WDT), _rows(grad_logits, "grad_logits", (logits.dtype,))
    rows, vocab, k = _places(logits, teacher_idx, teacher_logprob)
    if grad_logits.shape != logits.shape:
        raise ValueError("grad_logits must have the shape of logits")
    _sized(grad_loss, "grad_loss", rows); _sized(loss_out, "loss_out", rows)
    _sized(logprob_out, "logprob_out", rows * k)
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    code = lib().e8q_distill_grad(_ptr(logits), _dtype_code(logits), rows, vocab, stride, float(scale),
                                  _ptr(teacher_idx), _index_code(teacher_idx), _ptr(teacher_logprob), k, int(tail),
                                  _ptr(grad_loss), _ptr(loss_out), _ptr(logprob_out), _ptr(grad_logits), gstride,
                                  _ptr(workspace), _size(workspace), _ptr(status), _stream(logits, stream))
    _check("e8q_distill_grad", code)


def e8q_embed(table, tokens, out, status, scale=1.0, stream=None):
    """``e8q_embed``: ``out[t] = scale * table[tokens[t]]`` (negative ids: zeros)."""
    _dev(table, "table", _WDT); _dev(tokens, "tokens", _IDX); _dev(out, "out", _WDT)
    _dev(status, "status", (torch.int32,))
    if table.dim() != 2:
        raise ValueError("table must be [vocab, dim]")
    vocab, dim = table.shape
    _sized(out, "out", tokens.numel() * dim, _WDT)
    code = lib().e8q_embed(_ptr(table), _dtype_code(table), vocab, dim, _ptr(tokens), _index_code(tokens),
                           tokens.numel(), float(scale), _ptr(out), _dtype_code(out), _ptr(status),
                           _stream(table, stream))
    _check("e8q_embed", code)


def e8q_embed_backward_workspace_size(n, vocab, dim):
    return int(lib().e8q_embed_backward_workspace_size(int(n), int(vocab), int(dim)))


def e8q_embed_backward(grad_out, tokens, vocab, workspace, status, scale=1.0, grad_table=None, w_latent=None, lr=1.0,
                       stream=None):
    """``e8q_embed_backward``: the table's gradient by sorted tokens
    (``grad_table`` [vocab, dim], written whole) and/or SGD on the bf16
    latents of the rows that occur (``w_latent`` [vocab, dim], in place)."""
    _dev(grad_out, "grad_out", _WDT); _dev(tokens, "tokens", _IDX); _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    n = tokens.numel()
    if n == 0 or grad_out.numel() % n:
        raise ValueError("grad_out must be [n, dim] for n tokens")
    dim = grad_out.numel() // n
    _sized(grad_table, "grad_table", int(vocab) * dim, _WDT)
    _sized(w_latent, "w_latent", int(vocab) * dim, (torch.bfloat16,))
    code = lib().e8q_embed_backward(_ptr(grad_out), _dtype_code(grad_out), n, dim, _ptr(tokens), _index_code(tokens),
                                    int(vocab), float(scale), _ptr(grad_table),
                                    _dtype_code(grad_table) if grad_table is not None else F32, _ptr(w_latent),
                                    float(lr), _ptr(workspace), workspace.numel(), _ptr(status),
                                    _stream(grad_out, stream))
    _check("e8q_embed_backward", code)


def e8q_orthogonalize_workspace_size(batch, rows, cols):
    return int(lib().e8q_orthogonalize_workspace_size(int(batch), int(rows), int(cols)))


def e8q_orthogonalize(g, update_out, workspace, status, steps=5, coeffs=NEWTON_SCHULZ, stream=None):
    """``e8q_orthogonalize``: every matrix of ``g`` towards its orthogonal factor
    by ``steps`` Newton-Schulz products (``update_out`` bf16)."""
    _dev(g, "g", _WDT); _dev(update_out, "update_out", (torch.bfloat16,))
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    if update_out.shape != g.shape:
        raise ValueError("update_out must have the shape of g")
    b, r, c = _shape3(g)
    ca, cb, cc = (float(v) for v in coeffs)
    code = lib().e8q_orthogonalize(_ptr(g), _dtype_code(g), b, r, c, int(steps), ca, cb, cc, _ptr(update_out),
                                   _ptr(workspace), workspace.numel(), _ptr(status), _stream(g, stream))
    _check("e8q_orthogonalize", code)


def e8q_orthogonal_step(w, grad, momentum, workspace, status, mu=0.95, nesterov=True, lr=0.02, decay=0.0, gamma=1.0,
                        steps=5, coeffs=NEWTON_SCHULZ, w_out=None, momentum_out=None, stream=None):
    """``e8q_orthogonal_step``: momentum, its orthogonalization and the step of
    the bf16 latents ``w`` (in place unless ``w_out`` / ``momentum_out`` are
    given)."""
    w_out = w if w_out is None else w_out
    momentum_out = momentum if momentum_out is None else momentum_out
    _dev(w, "w", (torch.bfloat16,)); _dev(grad, "grad", _WDT); _dev(momentum, "momentum", (torch.float32,))
    _dev(w_out, "w_out", (torch.bfloat16,)); _dev(momentum_out, "momentum_out", (torch.float32,))
    _dev(workspace, "workspace", (torch.uint8,)); _dev(status, "status", (torch.int32,))
    if any(t.shape != w.shape for t in (grad, momentum, w_out, momentum_out)):
        raise ValueError("grad, momentum and outputs must have the shape of w")
    b, r, c = _shape3(w)
    ca, cb, cc = (float(v) for v in coeffs)
    code = lib().e8q_orthogonal_step(_ptr(w), _ptr(w_out), _ptr(grad), _dtype_code(grad), _ptr(momentum),
                                     _ptr(momentum_out), float(mu), int(bool(nesterov)), float(lr), float(decay),
                                     float(gamma), b, r, c, int(steps), ca, cb, cc, _ptr(workspace),
                                     workspace.numel(), _ptr(status), _stream(w, stream))
    _check("e8q_orthogonal_step", code)


def e8q_core_size(core_bound):
    return int(lib().e8q_core_size(int(core_bound)))


def e8q_status_string(code):
    return lib().e8q_status_string(int(code)).decode()


def e8q_version():
    return lib().e8q_version().decode()
