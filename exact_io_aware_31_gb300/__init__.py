"""Exact fused attention for NVIDIA GB300 (sm_103a): Python binding of ``libfa.so``.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/fa.h``.  PyTorch supplies
device memory and streams.  There is no fallback: if the library is missing
or the device is not sm_103, calls raise.

Raw entry points (same names and argument order as the C ABI, pointers as
ints):  ``fa_fwd``, ``fa_fwd_fp8``, ``fa_bwd``, ``fa_bwd_workspace_size``, the three phases
of ``fa_bwd`` (``fa_bwd_preprocess``, ``fa_bwd_dkdv``, ``fa_bwd_dq_convert``),
the split-KV decode forward (``fa_fwd_splitkv``,
``fa_fwd_splitkv_workspace_size``), the norm and rotation of queries and keys
(``fa_qk_norm_rope``, ``fa_qk_norm_rope_bwd``,
``fa_qk_norm_rope_bwd_workspace_size``), the paged cache (``fa_paged_append``, ``fa_paged_extend``, ``fa_paged_release``,
``fa_fwd_paged``, ``fa_fwd_paged_workspace_size``, ``fa_fwd_paged_shared``,
``fa_fwd_paged_shared_workspace_size``),
``fa_get_device_status``, ``fa_status_string``.
Tensor helpers: :func:`forward`, :func:`forward_fp8`, :func:`backward`, :func:`decode_forward`,
:func:`rope_table`, :func:`qk_norm_rope`, :func:`qk_norm_rope_backward`, :func:`paged_append`,
:func:`paged_pool`, :func:`paged_extend`, :func:`paged_release`, :func:`paged_forward`, :func:`paged_forward_shared`.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "LIB_PATH", "FaError", "load_library", "fa_fwd", "fa_fwd_fp8", "forward_fp8", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_deterministic",
    "fa_fwd_dropout", "fa_bwd_dropout",
    "fa_bwd_preprocess", "fa_bwd_dkdv", "fa_bwd_dq_convert", "fa_bwd_noalloc", "NOALLOC_SCRATCH_BYTES",
    "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size", "decode_forward",
    "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size", "fa_paged_append",
    "fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_fwd_paged_shared", "fa_fwd_paged_shared_workspace_size",
    "rope_table", "qk_norm_rope", "qk_norm_rope_backward", "paged_append", "paged_forward",
    "paged_forward_shared", "fa_paged_extend", "fa_paged_release", "paged_pool", "paged_extend", "paged_release",
    "fa_get_device_status", "fa_status_string", "forward", "backward", "EXPORTED_SYMBOLS",
    "FA_OK", "FA_ERR_INVALID_ARG", "FA_ERR_UNSUPPORTED", "FA_ERR_WORKSPACE", "FA_ERR_CUDA",
    "FA_ERR_DEVICE_TIMEOUT", "FA_ERR_INTERNAL", "FA_ERR_DEVICE_INDEX",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_DEVICE_TIMEOUT = 5
FA_ERR_INTERNAL = 6
FA_ERR_DEVICE_INDEX = 7

EXPORTED_SYMBOLS = ("fa_fwd", "fa_fwd_fp8", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_deterministic", "fa_fwd_dropout",
                    "fa_bwd_dropout", "fa_bwd_preprocess",
                    "fa_bwd_dkdv",
                    "fa_bwd_dq_convert", "fa_bwd_noalloc", "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size",
                    "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size", "fa_paged_append",
                    "fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_fwd_paged_shared",
                    "fa_fwd_paged_shared_workspace_size", "fa_paged_extend", "fa_paged_release",
                    "fa_get_device_status", "fa_status_string")

# Size of the library-owned scratch behind fa_bwd_noalloc (FA_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None


class FaError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so (once) and declare its signatures.  Raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m exact_io_aware_31_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.restype = i
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, f, f, i, vp]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    u64, u32 = ctypes.c_ulonglong, ctypes.c_uint
    lib.fa_fwd_dropout.restype = i
    lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u32, vp]
    lib.fa_bwd_dropout.restype = i
    lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u32, vp, sz, vp]
    lib.fa_bwd_deterministic.restype = i
    lib.fa_bwd_deterministic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd_preprocess.restype = i
    lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, vp, sz, vp]
    lib.fa_bwd_dkdv.restype = i
    lib.fa_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd_dq_convert.restype = i
    lib.fa_bwd_dq_convert.argtypes = [vp, i, i, i, i, f, vp, sz, vp]
    lib.fa_bwd_noalloc.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_fwd_splitkv_workspace_size.restype = sz
    lib.fa_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i, i]
    ll = ctypes.c_longlong
    lib.fa_qk_norm_rope.restype = i
    lib.fa_qk_norm_rope.argtypes = [vp] * 4 + [i] * 5 + [ll] * 6 + [i, vp, vp, i, f, vp, i, i, i, vp, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 8 + [i] * 5 + [ll] * 12 + [i, vp, vp, i, f, vp, i, i, i, vp, vp, sz, vp]
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.fa_paged_append.restype = i
    lib.fa_paged_append.argtypes = [vp] * 9 + [i] * 8 + [ll] * 12 + [i, vp, vp, i, f, vp, i, i, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_paged.argtypes = [vp] * 8 + [i] * 8 + [ll] * 8 + [f, i, i, vp, sz, vp]
    lib.fa_paged_extend.restype = i
    lib.fa_paged_extend.argtypes = [vp] * 10 + [i] * 6 + [vp]
    lib.fa_paged_release.restype = i
    lib.fa_paged_release.argtypes = [vp] * 6 + [i] * 5 + [vp]
    lib.fa_fwd_paged_shared.restype = i
    lib.fa_fwd_paged_shared.argtypes = [vp] * 10 + [i] * 9 + [ll] * 8 + [f, i, i, vp, sz, vp]
    lib.fa_fwd_paged_shared_workspace_size.restype = sz
    lib.fa_fwd_paged_shared_workspace_size.argtypes = [i] * 5
    lib.fa_fwd_paged_workspace_size.restype = sz
    lib.fa_fwd_paged_workspace_size.argtypes = [i]
    lib.fa_get_device_status.restype = i
    lib.fa_get_device_status.argtypes = [vp]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_status_string.argtypes = [i]
    _lib = lib
    return lib


# ------------------------------------------------------------- raw C ABI ----
def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream) -> int:
    return load_library().fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream)


def fa_fwd_fp8(q8, k8, v, o, lse, B, H, N, d, scale, q_descale, k_descale, causal, stream) -> int:
    return load_library().fa_fwd_fp8(q8, k8, v, o, lse, B, H, N, d, scale, q_descale, k_descale, causal, stream)


def fa_bwd_workspace_size(B, H, N, d) -> int:
    return load_library().fa_bwd_workspace_size(B, H, N, d)


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, workspace, workspace_bytes,
           stream) -> int:
    return load_library().fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                                 workspace_bytes, stream)


def fa_fwd_dropout(q, k, v, o, lse, B, H, N, d, scale, causal, p_drop, seed, offset, stream) -> int:
    return load_library().fa_fwd_dropout(q, k, v, o, lse, B, H, N, d, scale, causal, p_drop, seed, offset, stream)


def fa_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, p_drop, seed, offset, workspace,
                   workspace_bytes, stream) -> int:
    return load_library().fa_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, p_drop, seed,
                                         offset, workspace, workspace_bytes, stream)


def fa_bwd_deterministic(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, workspace, workspace_bytes,
                         stream) -> int:
    return load_library().fa_bwd_deterministic(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal,
                                               workspace, workspace_bytes, stream)


def fa_bwd_preprocess(o, dout, lse, B, H, N, d, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_preprocess(o, dout, lse, B, H, N, d, workspace, workspace_bytes, stream)


def fa_bwd_dkdv(q, k, v, dout, dk, dv, B, H, N, d, scale, causal, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_dkdv(q, k, v, dout, dk, dv, B, H, N, d, scale, causal, workspace,
                                      workspace_bytes, stream)


def fa_bwd_dq_convert(dq, B, H, N, d, scale, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_dq_convert(dq, B, H, N, d, scale, workspace, workspace_bytes, stream)


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, stream) -> int:
    """fa_bwd with the library's own scratch instead of a workspace (for callers that cannot allocate)."""
    return load_library().fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, stream)


def fa_fwd_splitkv(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, num_splits, workspace, workspace_bytes,
                   stream) -> int:
    return load_library().fa_fwd_splitkv(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, num_splits, workspace,
                                         workspace_bytes, stream)


def fa_fwd_splitkv_workspace_size(B, H, Nq, Nk, d, num_splits) -> int:
    return load_library().fa_fwd_splitkv_workspace_size(B, H, Nq, Nk, d, num_splits)


def fa_qk_norm_rope(q, k, q_out, k_out, B, Hq, Hk, N, d, q_stride_b, q_stride_h, q_stride_n, k_stride_b, k_stride_h,
                    k_stride_n, norm, q_weight, k_weight, weights_f32, eps, rope, rope_len, rope_dim, interleaved,
                    positions, stream) -> int:
    return load_library().fa_qk_norm_rope(q, k, q_out, k_out, B, Hq, Hk, N, d, q_stride_b, q_stride_h, q_stride_n,
                                          k_stride_b, k_stride_h, k_stride_n, norm, q_weight, k_weight, weights_f32,
                                          eps, rope, rope_len, rope_dim, interleaved, positions, stream)


def fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, B, Hq, Hk, N, d, q_stride_b, q_stride_h,
                        q_stride_n, k_stride_b, k_stride_h, k_stride_n, dq_stride_b, dq_stride_h, dq_stride_n,
                        dk_stride_b, dk_stride_h, dk_stride_n, norm, q_weight, k_weight, weights_f32, eps, rope,
                        rope_len, rope_dim, interleaved, positions, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, B, Hq, Hk, N, d,
                                              q_stride_b, q_stride_h, q_stride_n, k_stride_b, k_stride_h, k_stride_n,
                                              dq_stride_b, dq_stride_h, dq_stride_n, dk_stride_b, dk_stride_h,
                                              dk_stride_n, norm, q_weight, k_weight, weights_f32, eps, rope, rope_len,
                                              rope_dim, interleaved, positions, workspace, workspace_bytes, stream)


def fa_qk_norm_rope_bwd_workspace_size(d) -> int:
    return load_library().fa_qk_norm_rope_bwd_workspace_size(d)


def fa_paged_append(q, k, v, q_out, k_pages, v_pages, page_table, cu_seqlens, kv_lens, T, S, Hq, Hk, d, num_pages,
                    page_size, max_pages, q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                    kp_stride_p, kp_stride_h, kp_stride_r, vp_stride_p, vp_stride_h, vp_stride_r, norm, q_weight,
                    k_weight, weights_f32, eps, rope, rope_len, rope_dim, interleaved, stream) -> int:
    return load_library().fa_paged_append(q, k, v, q_out, k_pages, v_pages, page_table, cu_seqlens, kv_lens, T, S, Hq,
                                          Hk, d, num_pages, page_size, max_pages, q_stride_t, q_stride_h, k_stride_t,
                                          k_stride_h, v_stride_t, v_stride_h, kp_stride_p, kp_stride_h, kp_stride_r,
                                          vp_stride_p, vp_stride_h, vp_stride_r, norm, q_weight, k_weight,
                                          weights_f32, eps, rope, rope_len, rope_dim, interleaved, stream)


def fa_paged_extend(requests, new_lens, request_lens, request_table, pool, cu_seqlens, kv_lens, page_table, positions,
                    slots, T, S, R, num_pages, page_size, max_pages, stream) -> int:
    return load_library().fa_paged_extend(requests, new_lens, request_lens, request_table, pool, cu_seqlens, kv_lens,
                                          page_table, positions, slots, T, S, R, num_pages, page_size, max_pages,
                                          stream)


def fa_paged_release(requests, keep_lens, kept_pages, request_lens, request_table, pool, S, R, num_pages, page_size,
                     max_pages, stream) -> int:
    return load_library().fa_paged_release(requests, keep_lens, kept_pages, request_lens, request_table, pool, S, R,
                                           num_pages, page_size, max_pages, stream)


def fa_fwd_paged(q, k_pages, v_pages, o, lse, page_table, cu_seqlens, kv_lens, T, S, Hq, Hk, d, num_pages, page_size,
                 max_pages, q_stride_t, q_stride_h, kp_stride_p, kp_stride_h, kp_stride_r, vp_stride_p, vp_stride_h,
                 vp_stride_r, scale, causal, max_q, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_fwd_paged(q, k_pages, v_pages, o, lse, page_table, cu_seqlens, kv_lens, T, S, Hq, Hk, d,
                                       num_pages, page_size, max_pages, q_stride_t, q_stride_h, kp_stride_p,
                                       kp_stride_h, kp_stride_r, vp_stride_p, vp_stride_h, vp_stride_r, scale, causal,
                                       max_q, workspace, workspace_bytes, stream)


def fa_fwd_paged_workspace_size(d) -> int:
    return load_library().fa_fwd_paged_workspace_size(d)


def fa_fwd_paged_shared(q, k_pages, v_pages, o, lse, page_table, cu_seqlens, kv_lens, groups, prefix_lens, T, S,
                        num_groups, Hq, Hk, d, num_pages, page_size, max_pages, q_stride_t, q_stride_h, kp_stride_p,
                        kp_stride_h, kp_stride_r, vp_stride_p, vp_stride_h, vp_stride_r, scale, causal, max_q,
                        workspace, workspace_bytes, stream) -> int:
    return load_library().fa_fwd_paged_shared(q, k_pages, v_pages, o, lse, page_table, cu_seqlens, kv_lens, groups,
                                              prefix_lens, T, S, num_groups, Hq, Hk, d, num_pages, page_size,
                                              max_pages, q_stride_t, q_stride_h, kp_stride_p, kp_stride_h,
                                              kp_stride_r, vp_stride_p, vp_stride_h, vp_stride_r, scale, causal,
                                              max_q, workspace, workspace_bytes, stream)


def fa_fwd_paged_shared_workspace_size(T, S, num_groups, Hq, d) -> int:
    return load_library().fa_fwd_paged_shared_workspace_size(T, S, num_groups, Hq, d)


def fa_get_device_status(stream) -> int:
    return load_library().fa_get_device_status(stream)


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(status).decode()


# --------------------------------------------------------- tensor helpers ----
def _check(t, name, shape, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def forward(q, k, v, scale=None, causal=False, out=None, lse=None, stream=None):
    """Exact attention forward on [B, H, N, d] bf16 CUDA tensors; returns ``(o, lse)``."""
    import torch
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, (B, H, N, d), torch.bfloat16)
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "out", (B, H, N, d), torch.bfloat16)
    _check(l, "lse", (B, H, N), torch.float32)
    st = fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), B, H, N, d,
                float(scale), int(bool(causal)), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd")
    return o, l


def forward_fp8(q8, k8, v, q_descale=1.0, k_descale=1.0, scale=None, causal=False, out=None, lse=None,
                stream=None):
    """Forward with E4M3 queries and keys (``torch.float8_e4m3fn`` or their ``uint8`` codes,
    [B, H, N, 128]) and bf16 values; returns ``(o, lse)``."""
    import torch
    B, H, N, d = q8.shape
    for name, t in (("q8", q8), ("k8", k8)):
        want = t.dtype if t.dtype in (torch.uint8, torch.float8_e4m3fn) else torch.float8_e4m3fn
        _check(t, name, (B, H, N, d), want)
    _check(v, "v", (B, H, N, d), torch.bfloat16)
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(v) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=v.device) if lse is None else lse
    _check(o, "out", (B, H, N, d), torch.bfloat16)
    _check(l, "lse", (B, H, N), torch.float32)
    st = fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), B, H, N, d,
                    float(scale), float(q_descale), float(k_descale), int(bool(causal)), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_fp8")
    return o, l


def backward(q, k, v, o, lse, dout, scale=None, causal=False, workspace=None, grads=None, stream=None,
             deterministic=False):
    """Gradients ``(dq, dk, dv)`` of ``sum(O * dout)``; ``o`` and ``lse`` from :func:`forward`.

    ``deterministic=True`` uses ``fa_bwd_deterministic`` (bitwise reproducible, slower)."""
    import torch
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check(t, name, (B, H, N, d), torch.bfloat16)
    _check(lse, "lse", (B, H, N), torch.float32)
    if scale is None:
        scale = d ** -0.5
    need = fa_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if grads is None:
        grads = tuple(torch.empty_like(q) for _ in range(3))
    dq, dk, dv = grads
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check(t, name, (B, H, N, d), torch.bfloat16)
    fn = fa_bwd_deterministic if deterministic else fa_bwd
    st = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_deterministic" if deterministic else "fa_bwd")
    return dq, dk, dv


def decode_forward(q, k, v, scale=None, causal=True, num_splits=0, out=None, lse=None, workspace=None,
                   stream=None):
    """Split-KV attention of ``q [B, H, Nq, d]`` (Nq <= 8, the last Nq positions) against the cache
    ``k, v [B, H, Nk, d]`` (bf16 CUDA tensors); returns ``(o, lse)``."""
    import torch
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    _check(q, "q", (B, H, Nq, d), torch.bfloat16)
    for name, t in (("k", k), ("v", v)):
        _check(t, name, (B, H, Nk, d), torch.bfloat16)
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "out", (B, H, Nq, d), torch.bfloat16)
    _check(l, "lse", (B, H, Nq), torch.float32)
    need = fa_fwd_splitkv_workspace_size(B, H, Nq, Nk, d, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), B, H, Nq, Nk, d,
                        float(scale), int(bool(causal)), int(num_splits), wptr, wbytes, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_splitkv")
    return o, l


# ------------------------------------------------ norm, rotation and paged cache ----
# A decode step makes several of these calls a layer, each of a few microseconds
# on the GPU: the helpers below look at each tensor once and call the library
# directly.
def _refuse(t, name, shape, dtype, device):
    """The error of a tensor that is not a CUDA tensor of this type and shape on device ``device``."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the first tensor on cuda:{device}")
    raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} with a contiguous last dimension, got {t.dtype} "
                     f"{tuple(t.shape)}, strides {t.stride()}")


def _elsewhere(first, stream):
    """Where a helper must not run as it is called: None, or the context that makes the first tensor's device and the
    given stream current (what is allocated there belongs to the stream that uses it)."""
    import torch
    device = first.get_device() if isinstance(first, torch.Tensor) else -1
    if device < 0:
        raise ValueError("the first argument must be a CUDA tensor")
    if stream is not None:
        if stream.device != first.device:
            raise ValueError(f"the stream is on {stream.device}, the first tensor on {first.device}")
        return torch.cuda.stream(stream)
    return None if device == torch._C._cuda_getDevice() else torch.cuda.device(device)


# The checks below run before every call, so they are short: a serving step of a few tokens takes the device no longer
# than its call takes the host.


def _rows(t, name, shape, dtype, device):
    """Check rows of any layout; their strides without the last (where a size is 1 a stride may be anything)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and (steps := t.stride())[-1] == 1:
            return steps[:-1]
    except AttributeError:  # not a tensor
        pass
    _refuse(t, name, shape, dtype, device)


def _flat(t, name, shape, dtype, device):
    """Check a contiguous tensor (None passes); its address."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _refuse(t, name, shape, dtype, device)


_rooms = {}


def _room_for(size, device, d):
    """Workspace bytes that ``size(d)`` gives on the current device, asked for once."""
    need = _rooms.get((size, device, d))
    if need is None:
        need = size(d)
        if need:  # (0: refused by the call itself)
            _rooms[size, device, d] = need
    return need


_shared_rooms = {}


def _shared_room(T, S, groups, Hq, d, device):
    """Workspace bytes of :func:`paged_forward_shared` on the current device, asked for once for each batch shape (at
    most 4096 of them are kept)."""
    key = T, S, groups, Hq, d, device
    need = _shared_rooms.get(key)
    if need is None:
        need = load_library().fa_fwd_paged_shared_workspace_size(T, S, groups, Hq, d)
        if need:  # (0: refused by the call itself, or nothing to do)
            if len(_shared_rooms) >= 4096:
                _shared_rooms.clear()
            _shared_rooms[key] = need
    return need


def _room(workspace, device):
    """Address and bytes of a workspace (None: no room)."""
    if workspace is None:
        return None, 0
    try:
        if workspace.get_device() == device and workspace.is_contiguous():
            return workspace.data_ptr(), workspace.nbytes
    except AttributeError:  # not a tensor
        pass
    _refuse(workspace, "workspace", getattr(workspace, "shape", ()), getattr(workspace, "dtype", None), device)


def _shape(t, name, n):
    """Shape of a tensor of n dimensions."""
    shape = getattr(t, "shape", ())
    if len(shape) != n:
        raise ValueError(f"{name} must be a CUDA tensor of {n} dimensions")
    return shape


def _norm_rope_args(d, norm, q_weight, k_weight, eps, rope, interleaved, device):
    """The shared trailing arguments of the norm-and-rotation calls, checked."""
    import torch
    first = q_weight if q_weight is not None else k_weight
    wt = torch.float32 if getattr(first, "dtype", None) == torch.float32 else torch.bfloat16
    qw, kw = _flat(q_weight, "q_weight", (d,), wt, device), _flat(k_weight, "k_weight", (d,), wt, device)
    rope_len, rope_dim = (0, 0) if rope is None else _shape(rope, "rope", 2)
    return (1 if norm else 0, qw, kw, 1 if wt == torch.float32 else 0, eps,
            _flat(rope, "rope", (rope_len, rope_dim), torch.float32, device), rope_len, rope_dim,
            1 if interleaved else 0)


def rope_table(length, rope_dim, base=10000.0, device="cuda"):
    """Rotation table ``[length, rope_dim]`` fp32 of the angles ``p * base ** (-2 i / rope_dim)``: row p holds the
    ``rope_dim / 2`` cosines, then the sines.  Angles are formed in fp64 (in fp32 they lose bits at far positions).
    A program makes it once; any table of that layout (scaled frequencies, say) serves as well."""
    import torch
    if length < 1 or rope_dim < 2 or rope_dim % 2:
        raise ValueError("length must be >= 1 and rope_dim a positive even number")
    i = torch.arange(rope_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * float(base) ** (-2.0 * i / rope_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6, interleaved=False,
                 norm=True, out=None, stream=None):
    """Norm of queries and keys for each head, then rotation: ``q [B, Hq, N, d]``, ``k [B, Hk, N, d]`` bf16 of any
    strides that are multiples of 8 (``x.transpose(1, 2)`` of a token-major projection, a slice of a wider row, an
    ``expand``) -> contiguous ``(q_out, k_out)``, what :func:`forward` takes (where Hk < Hq with keys and values
    repeated for the query heads of their group).  ``rope`` is a :func:`rope_table` (None: no rotation),
    ``positions`` int32 ``[B, N]`` (None: 0 .. N-1), ``norm=False`` rotates only."""
    where = _elsewhere(q, stream)
    if where is not None:
        with where:
            return qk_norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved, norm, out)
    import torch
    bf16 = torch.bfloat16
    B, Hq, N, d = _shape(q, "q", 4)
    dev, Hk = q.get_device(), _shape(k, "k", 4)[1]
    sq, sk = _rows(q, "q", (B, Hq, N, d), bf16, dev), _rows(k, "k", (B, Hk, N, d), bf16, dev)
    args = _norm_rope_args(d, norm, q_weight, k_weight, eps, rope, interleaved, dev)
    pos = _flat(positions, "positions", (B, N), torch.int32, dev)
    if out is None:
        q_out = torch.empty(B, Hq, N, d, dtype=bf16, device=q.device)
        k_out = torch.empty(B, Hk, N, d, dtype=bf16, device=q.device)
    else:
        q_out, k_out = out
        _flat(q_out, "q_out", (B, Hq, N, d), bf16, dev)
        _flat(k_out, "k_out", (B, Hk, N, d), bf16, dev)
    st = load_library().fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), B, Hq, Hk, N,
                                        d, *sq, *sk, *args, pos, torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6,
                          interleaved=False, norm=True, grads=None, weight_grads=True, workspace=None, stream=None):
    """Gradients ``(dq, dk, dq_weight, dk_weight)`` of :func:`qk_norm_rope` from those of its outputs
    (:func:`backward`'s ``dq, dk``).  ``dq, dk`` have q's and k's shapes, token-major in memory
    (``[B, N, H, d]``) unless ``grads=(dq, dk)`` gives tensors of any strides.  The weights' gradients are
    fp32 ``[d]`` (None with ``norm=False`` or ``weight_grads=False``)."""
    where = _elsewhere(dq_out, stream)
    if where is not None:
        with where:
            return qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, rope, positions, eps, interleaved,
                                         norm, grads, weight_grads, workspace)
    import torch
    B, Hq, N, d = _shape(q, "q", 4)
    dev, Hk = q.get_device(), _shape(k, "k", 4)[1]
    bf16 = torch.bfloat16
    sq, sk = _rows(q, "q", (B, Hq, N, d), bf16, dev), _rows(k, "k", (B, Hk, N, d), bf16, dev)
    dqo = _flat(dq_out, "dq_out", (B, Hq, N, d), bf16, dev)
    dko = _flat(dk_out, "dk_out", (B, Hk, N, d), bf16, dev)
    args = _norm_rope_args(d, norm, q_weight, k_weight, eps, rope, interleaved, dev)
    pos = _flat(positions, "positions", (B, N), torch.int32, dev)
    if grads is None:
        sdq, sdk = (N * Hq * d, d, Hq * d), (N * Hk * d, d, Hk * d)
        dq = torch.empty_strided((B, Hq, N, d), (*sdq, 1), dtype=bf16, device=q.device)
        dk = torch.empty_strided((B, Hk, N, d), (*sdk, 1), dtype=bf16, device=q.device)
    else:
        dq, dk = grads
        sdq, sdk = _rows(dq, "dq", (B, Hq, N, d), bf16, dev), _rows(dk, "dk", (B, Hk, N, d), bf16, dev)
    dqw = dkw = None
    if norm and weight_grads:
        dqw = torch.empty(d, dtype=torch.float32, device=q.device)
        dkw = torch.empty(d, dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(_room_for(fa_qk_norm_rope_bwd_workspace_size, dev, d), dtype=torch.uint8,
                                    device=q.device)
    ws, wbytes = _room(workspace, dev)
    st = load_library().fa_qk_norm_rope_bwd(dqo, dko, q.data_ptr(), k.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                            None if dqw is None else dqw.data_ptr(),
                                            None if dkw is None else dkw.data_ptr(), B, Hq, Hk, N, d, *sq, *sk, *sdq,
                                            *sdk, *args, pos, ws, wbytes, torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_qk_norm_rope_bwd")
    return dq, dk, dqw, dkw


def _cache_args(k_pages, v_pages, page_table, cu_seqlens, kv_lens, d, device):
    """Checks of the paged cache's tensors: their addresses, ``(S, Hk, num_pages, page_size, max_pages)``, strides."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    num_pages, Hk, page_size, _ = _shape(k_pages, "k_pages", 4)
    shape = (num_pages, Hk, page_size, d)
    steps = (*_rows(k_pages, "k_pages", shape, bf16, device), *_rows(v_pages, "v_pages", shape, bf16, device))
    S, max_pages = _shape(page_table, "page_table", 2)
    addresses = (_flat(page_table, "page_table", (S, max_pages), i32, device),
                 _flat(cu_seqlens, "cu_seqlens", (S + 1,), i32, device), _flat(kv_lens, "kv_lens", (S,), i32, device))
    return addresses, S, Hk, num_pages, page_size, max_pages, steps


def paged_append(q, k, v, k_pages, v_pages, page_table, cu_seqlens, kv_lens, q_weight=None, k_weight=None, rope=None,
                 eps=1e-6, interleaved=False, norm=True, out=None, stream=None):
    """Norm and rotate the new tokens' ``q [T, Hq, d]`` and ``k [T, Hk, d]`` at their positions, write keys and values
    into the cache ``k_pages, v_pages [num_pages, Hk, page_size, d]`` (strides of whole rows, multiples of 8: a
    token-major pool is a ``transpose(1, 2)`` view), and return the queries ``[T, Hq, d]`` for :func:`paged_forward`
    (rows of no sequence are not written).
    ``page_table [S, max_pages]``, ``cu_seqlens [S + 1]`` and ``kv_lens [S]`` (new tokens included) are int32 on
    the device.  ``rope=None, norm=False`` caches k and v as they are."""
    where = _elsewhere(q, stream)
    if where is not None:
        with where:
            return paged_append(q, k, v, k_pages, v_pages, page_table, cu_seqlens, kv_lens, q_weight, k_weight, rope,
                                eps, interleaved, norm, out)
    import torch
    bf16 = torch.bfloat16
    T, Hq, d = _shape(q, "q", 3)
    dev = q.get_device()
    meta, S, Hk, num_pages, page_size, max_pages, steps = _cache_args(k_pages, v_pages, page_table, cu_seqlens, kv_lens,
                                                                      d, dev)
    sq, sk, sv = (_rows(q, "q", (T, Hq, d), bf16, dev), _rows(k, "k", (T, Hk, d), bf16, dev),
                  _rows(v, "v", (T, Hk, d), bf16, dev))
    args = _norm_rope_args(d, norm, q_weight, k_weight, eps, rope, interleaved, dev)
    if out is None:
        out = torch.empty(T, Hq, d, dtype=bf16, device=q.device)
    else:
        _flat(out, "out", (T, Hq, d), bf16, dev)
    st = load_library().fa_paged_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), k_pages.data_ptr(),
                                        v_pages.data_ptr(), *meta, T, S, Hq, Hk, d, num_pages, page_size, max_pages,
                                        *sq, *sk, *sv, *steps, *args, torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_paged_append")
    return out


def paged_pool(num_pages, device="cuda"):
    """A pool ``[num_pages + 2]`` int32 of free pages, page 0 the first to be taken."""
    import torch
    if num_pages < 1:
        raise ValueError("num_pages must be >= 1")
    pool = torch.zeros(num_pages + 2, dtype=torch.int32, device=device)
    pool[0] = num_pages
    pool[2:] = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
    return pool


def _tables_args(requests, request_lens, request_table, pool, device):
    """Checks of the tensors that hold the requests: their addresses, ``(S, R, num_pages, max_pages)``."""
    import torch
    i32 = torch.int32
    try:
        (S,), (R, max_pages), (room,) = requests.shape, request_table.shape, pool.shape
    except (AttributeError, TypeError, ValueError):  # one of them has not these dimensions
        S, (R, max_pages), room = (_shape(requests, "requests", 1)[0], _shape(request_table, "request_table", 2),
                                   _shape(pool, "pool", 1)[0])
    if room < 3:
        raise ValueError("pool must hold at least one page")
    return (_flat(requests, "requests", (S,), i32, device), _flat(request_lens, "request_lens", (R,), i32, device),
            _flat(request_table, "request_table", (R, max_pages), i32, device),
            _flat(pool, "pool", (room,), i32, device), S, R, room - 2, max_pages)


def paged_extend(requests, new_lens, request_lens, request_table, pool, page_size, tokens, out=None, stream=None):
    """Room in a paged cache for the new tokens of a step, and the step's tables: ``requests [S]`` says which request
    each sequence is (negative: a place without one), ``new_lens [S]`` how many tokens it brings; all int32 on the
    device.  ``request_lens [R]``, ``request_table [R, max_pages]`` and ``pool`` (:func:`paged_pool`) are the
    requests' state and brought up to date.  Returns ``(cu_seqlens [S + 1], kv_lens [S], page_table [S, max_pages],
    positions [tokens], slots [tokens] int64)`` for the other calls; ``out`` gives tensors to write to (any of the
    last two may be None: not wanted), as a captured step does.  Of ``page_table`` only entries in use are written.
    A sequence that finds no room has ``kv_lens`` 0 and leaves its request as it was.  Rows behind the last sequence
    (all of them in a step without any) have position 0 and slot -1.  Pages that requests share are full ones."""
    where = _elsewhere(requests, stream)
    if where is not None:
        with where:
            return paged_extend(requests, new_lens, request_lens, request_table, pool, page_size, tokens, out)
    import torch
    i32 = torch.int32
    dev = requests.get_device()
    req, lens, table, pool_at, S, R, num_pages, max_pages = _tables_args(requests, request_lens, request_table, pool, dev)
    new = _flat(new_lens, "new_lens", (S,), i32, dev)
    if not 0 <= tokens < 1 << 31:
        raise ValueError("tokens must be in 0 .. 2^31 - 1")
    if out is None:
        out = (torch.empty(S + 1, dtype=i32, device=requests.device), torch.empty(S, dtype=i32, device=requests.device),
               torch.empty(S, max_pages, dtype=i32, device=requests.device),
               torch.empty(tokens, dtype=i32, device=requests.device),
               torch.empty(tokens, dtype=torch.int64, device=requests.device))
    cu, kv, pages, positions, slots = out
    st = load_library().fa_paged_extend(req, new, lens, table, pool_at, _flat(cu, "cu_seqlens", (S + 1,), i32, dev),
                                        _flat(kv, "kv_lens", (S,), i32, dev),
                                        _flat(pages, "page_table", (S, max_pages), i32, dev),
                                        _flat(positions, "positions", (tokens,), i32, dev),
                                        _flat(slots, "slots", (tokens,), torch.int64, dev), tokens, S, R, num_pages,
                                        page_size, max_pages, torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_paged_extend")
    if S == 0:  # (the call did nothing: all rows are behind the last sequence)
        for t, value in ((cu, 0), (positions, 0), (slots, -1)):
            if t is not None:
                t.fill_(value)
    return cu, kv, pages, positions, slots


def paged_release(requests, request_lens, request_table, pool, page_size, keep_lens=None, kept_pages=None,
                  stream=None):
    """The requests ``requests [S]`` (negative: none) give pages back to the pool and keep their first ``keep_lens
    [S]`` keys (None: none).  ``kept_pages [R]`` counts the pages at the front of each request that it shares and
    does not own (None: it owns all); a request that keeps fewer keys than those hold has its count brought down by
    the caller."""
    where = _elsewhere(requests, stream)
    if where is not None:
        with where:
            return paged_release(requests, request_lens, request_table, pool, page_size, keep_lens, kept_pages)
    import torch
    dev = requests.get_device()
    req, lens, table, pool_at, S, R, num_pages, max_pages = _tables_args(requests, request_lens, request_table, pool, dev)
    st = load_library().fa_paged_release(req, _flat(keep_lens, "keep_lens", (S,), torch.int32, dev),
                                         _flat(kept_pages, "kept_pages", (R,), torch.int32, dev), lens, table, pool_at,
                                         S, R, num_pages, page_size, max_pages,
                                         torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_paged_release")


def paged_forward(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, scale=None, causal=True, max_q=0, out=None,
                  lse=None, workspace=None, stream=None):
    """Attention of the new tokens ``q [T, Hq, d]`` (strides of whole rows: multiples of 8, at least d) over the paged
    cache that :func:`paged_append` wrote; returns ``(o [T, Hq, d], lse [T, Hq])``, in which rows of no sequence are
    not written.  ``max_q`` is the longest chunk of the step (0: not known; a hint that selects the kernel variant)."""
    where = _elsewhere(q, stream)
    if where is not None:
        with where:
            return paged_forward(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, scale, causal, max_q, out, lse,
                                 workspace)
    import torch
    bf16 = torch.bfloat16
    T, Hq, d = _shape(q, "q", 3)
    dev = q.get_device()
    meta, S, Hk, num_pages, page_size, max_pages, steps = _cache_args(k_pages, v_pages, page_table, cu_seqlens, kv_lens,
                                                                      d, dev)
    sq = _rows(q, "q", (T, Hq, d), bf16, dev)
    if out is None:
        out = torch.empty(T, Hq, d, dtype=bf16, device=q.device)
    else:
        _flat(out, "out", (T, Hq, d), bf16, dev)
    if lse is None:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device)
    else:
        _flat(lse, "lse", (T, Hq), torch.float32, dev)
    if workspace is None:
        workspace = torch.empty(_room_for(fa_fwd_paged_workspace_size, dev, d), dtype=torch.uint8, device=q.device)
    ws, wbytes = _room(workspace, dev)
    st = load_library().fa_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), *meta, T, S, Hq, Hk, d, num_pages, page_size, max_pages, *sq,
                                     *steps, d ** -0.5 if scale is None else scale, 1 if causal else 0, max_q,
                                     ws, wbytes, torch._C._cuda_getCurrentRawStream(dev))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_paged")
    return out, lse


def paged_forward_shared(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, groups, prefix_lens, scale=None,
                         causal=True, max_q=0, out=None, lse=None, workspace=None, stream=None):
    """:func:`paged_forward` for a batch whose sequences share their first keys, which are read and multiplied once for
    each group: ``groups [n + 1]`` int32 on the device holds each group's first sequence and the last one's end,
    ``prefix_lens [n]`` how many keys its sequences share (any number that is true: what is not worth computing once
    is not).  Same results up to rounding."""
    where = _elsewhere(q, stream)
    if where is not None:
        with where:
            return paged_forward_shared(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, groups, prefix_lens,
                                        scale, causal, max_q, out, lse, workspace)
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    T, Hq, d = _shape(q, "q", 3)
    dev = q.get_device()
    meta, S, Hk, num_pages, page_size, max_pages, steps = _cache_args(k_pages, v_pages, page_table, cu_seqlens, kv_lens,
                                                                      d, dev)
    n = _shape(prefix_lens, "prefix_lens", 1)[0]
    shared = _flat(groups, "groups", (n + 1,), i32, dev), _flat(prefix_lens, "prefix_lens", (n,), i32, dev)
    sq = _rows(q, "q", (T, Hq, d), bf16, dev)
    if out is None:
        out = torch.empty_like(q) if sq == (Hq * d, d) else torch.empty(T, Hq, d, dtype=bf16, device=q.device)
    else:
        _flat(out, "out", (T, Hq, d), bf16, dev)
    if lse is None:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device)
    else:
        _flat(lse, "lse", (T, Hq), torch.float32, dev)
    on = torch._C._cuda_getCurrentRawStream(dev)
    ws, wbytes = _room(workspace, dev)
    own = None  # a workspace of this call alone: the allocator's bytes, without a tensor around them (2 us)
    if workspace is None and (wbytes := _shared_room(T, S, n, Hq, d, dev)):
        ws = own = torch._C._cuda_cudaCachingAllocator_raw_alloc(wbytes, on)
    try:
        st = load_library().fa_fwd_paged_shared(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(),
                                                lse.data_ptr(), *meta, *shared, T, S, n, Hq, Hk, d, num_pages,
                                                page_size, max_pages, *sq, *steps,
                                                d ** -0.5 if scale is None else scale, 1 if causal else 0, max_q, ws,
                                                wbytes, on)
    finally:
        if own is not None:
            torch._C._cuda_cudaCachingAllocator_raw_delete(own)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_paged_shared")
    return out, lse
