"""ctypes binding of libtriattn.so: one Python function per C entry point, same names.

Argument marshalling only (pointers and sizes in, status code out); every step
of the computation runs in the library's CUDA kernels.  A non-OK status is
raised: TA_ERR_INVALID_ARG as ValueError, TA_ERR_UNSUPPORTED as
NotImplementedError, anything else as RuntimeError.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtriattn.so")

TA_OK, TA_ERR_INVALID_ARG, TA_ERR_UNSUPPORTED, TA_ERR_CUDA, TA_ERR_TIMEOUT, TA_ERR_DEVICE = range(6)
TA_F32, TA_F16, TA_BF16, TA_E4M3 = 0, 1, 2, 3
TA_MASK_NONE, TA_MASK_CAUSAL, TA_MASK_SLIDING_WINDOW, TA_MASK_PREFIX_LM, TA_MASK_SINK_WINDOW = 0, 1, 2, 3, 6

# Every symbol include/triattn.h declares.
EXPORTS = ("tri_attn_fwd", "tri_attn_fwd_strided", "tri_attn_varlen_fwd", "tri_attn_varlen_fwd_strided", "tri_attn_varlen_fwd_masked",
           "tri_attn_bwd", "tri_attn_bwd_workspace_size", "tri_attn_bwd_noalloc", "tri_attn_varlen_bwd",
           "tri_attn_varlen_bwd_workspace_size", "tri_attn_varlen_bwd_sink_workspace_size",
           "tri_attn_rotary", "tri_attn_kv_append", "tri_attn_paged_fwd", "tri_attn_paged_workspace_size",
           "tri_attn_mask_to_kv_lengths", "tri_attn_get_status", "tri_attn_error_string", "tri_attn_version")

_lock = threading.Lock()
_lib = None


class TriAttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load() -> ctypes.CDLL:
    """Load the built library; raise loudly if it is missing (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run masked_attention_tri_gb300.build.build() "
                              "(nvcc, sm_103a) first")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.tri_attn_fwd.argtypes = [P, P, P, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P, P]
        lib.tri_attn_fwd.restype = I
        lib.tri_attn_fwd_strided.argtypes = [P, P, P, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P, P, P, P, P]
        lib.tri_attn_fwd_strided.restype = I
        lib.tri_attn_varlen_fwd.argtypes = [P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P, P, P, I, I, I, I, I, I,
                                            P, P, P, P]
        lib.tri_attn_varlen_fwd.restype = I
        L = ctypes.c_longlong
        lib.tri_attn_varlen_fwd_strided.argtypes = [P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P, P, P, I, I, I, I,
                                                    I, I, L, L, L, P, P, P, P]
        lib.tri_attn_varlen_fwd_strided.restype = I
        lib.tri_attn_varlen_fwd_masked.argtypes = [P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P, P, P, I, I, I, I,
                                                   I, I, I, P, I, P, I, L, L, L, P, P, P, P]
        lib.tri_attn_varlen_fwd_masked.restype = I
        Z = ctypes.c_size_t
        lib.tri_attn_bwd.argtypes = [P, P, P, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P, P, P, P, P, P, Z, P]
        lib.tri_attn_bwd.restype = I
        lib.tri_attn_bwd_noalloc.argtypes = [P, P, P, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P, P, P, P, P, P]
        lib.tri_attn_bwd_noalloc.restype = I
        lib.tri_attn_varlen_bwd.argtypes = [P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P, P, P, I, I, I, I, I, I,
                                            I, P, I, P, I, P, P, P, P, P, P, P, P, Z, P]
        lib.tri_attn_varlen_bwd.restype = I
        lib.tri_attn_varlen_bwd_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.tri_attn_varlen_bwd_workspace_size.restype = Z
        lib.tri_attn_varlen_bwd_sink_workspace_size.argtypes = [I] * 9
        lib.tri_attn_varlen_bwd_sink_workspace_size.restype = Z
        lib.tri_attn_bwd_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.tri_attn_bwd_workspace_size.restype = Z
        lib.tri_attn_rotary.argtypes = [P, P, I, P, P, I, I, F, I, I, I, I, I, L, L, L, L, P, P, P]
        lib.tri_attn_rotary.restype = I
        lib.tri_attn_kv_append.argtypes = [P, P, P, I, P, P, P, I, I, I, I, I, I, L, L, L, L, P, P, I, I, F, P, P, I, P,
                                           P, I, I, I, P, P, P, P]
        lib.tri_attn_kv_append.restype = I
        lib.tri_attn_paged_fwd.argtypes = [P, I, P, P, P, I, I, I, I, I, I, L, F, I, I, P, P, I, P, P, I, I, I, P, P, P,
                                           P, P, Z, P]
        lib.tri_attn_paged_fwd.restype = I
        lib.tri_attn_paged_workspace_size.argtypes = [I, I, I, I, I]
        lib.tri_attn_paged_workspace_size.restype = Z
        lib.tri_attn_mask_to_kv_lengths.argtypes = [P, I, I, I, P, P, P]
        lib.tri_attn_mask_to_kv_lengths.restype = I
        lib.tri_attn_get_status.argtypes = [P]
        lib.tri_attn_get_status.restype = I
        lib.tri_attn_error_string.argtypes = [I]
        lib.tri_attn_error_string.restype = ctypes.c_char_p
        lib.tri_attn_version.argtypes = []
        lib.tri_attn_version.restype = I
        _lib = lib
        return lib


def tri_attn_error_string(status: int) -> str:
    return load().tri_attn_error_string(int(status)).decode()


def _check(status: int, fn: str) -> None:
    if status == TA_OK:
        return
    msg = f"{fn}: {tri_attn_error_string(status)} (status {status})"
    if status == TA_ERR_INVALID_ARG:
        raise ValueError(msg)
    if status == TA_ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise TriAttnError(status, msg)


def tri_attn_fwd(q, k, v, qkv_dtype, bias, bias_dtype, mask, kv_lengths, B, N, H, Q, K, D, scale, out, lse, max_,
                 stream) -> None:
    """Pointers are ints (0 = NULL); stream is a cudaStream_t handle as int."""
    st = load().tri_attn_fwd(q, k, v, qkv_dtype, bias, bias_dtype, mask or None, kv_lengths or None, B, N, H, Q, K,
                             D, float(scale), out, lse or None, max_ or None, stream or None)
    _check(st, "tri_attn_fwd")


def tri_attn_bwd(q, k, v, qkv_dtype, bias, bias_dtype, mask, kv_lengths, B, N, H, Q, K, D, scale, lse, out, d_out,
                 dq, dk, dv, dbias, workspace, workspace_bytes, stream) -> None:
    """Gradients of tri_attn_fwd; pointers are ints (0 = NULL), workspace_bytes an int."""
    st = load().tri_attn_bwd(q, k, v, qkv_dtype, bias, bias_dtype, mask or None, kv_lengths or None, B, N, H, Q, K, D,
                             float(scale), lse, out or None, d_out, dq, dk, dv, dbias or None, workspace,
                             int(workspace_bytes), stream or None)
    _check(st, "tri_attn_bwd")


def tri_attn_bwd_noalloc(q, k, v, qkv_dtype, bias, bias_dtype, mask, kv_lengths, B, N, H, Q, K, D, scale, lse, out,
                         d_out, dq, dk, dv, dbias, stream) -> None:
    """tri_attn_bwd in the library's own static scratch (no workspace, no allocation)."""
    st = load().tri_attn_bwd_noalloc(q, k, v, qkv_dtype, bias, bias_dtype, mask or None, kv_lengths or None, B, N, H,
                                     Q, K, D, float(scale), lse, out or None, d_out, dq, dk, dv, dbias or None,
                                     stream or None)
    _check(st, "tri_attn_bwd_noalloc")


# Bytes of the static scratch tri_attn_bwd_noalloc works in (TRI_ATTN_BWD_NOALLOC_SCRATCH_BYTES).
BWD_NOALLOC_SCRATCH_BYTES = 16 << 20


def tri_attn_varlen_bwd(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                        max_seqlen_k, H, D, scale, kv_num_blocks, kv_indices, full_kv_num_blocks, full_kv_indices,
                        mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod, window,
                        prefix_lengths, prefix_length, bias, bias_dtype, lse, out, d_out, dq, dk, dv, dbias,
                        workspace, workspace_bytes, stream) -> None:
    st = load().tri_attn_varlen_bwd(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                    max_seqlen_q, max_seqlen_k, H, D, float(scale), kv_num_blocks or None,
                                    kv_indices or None, full_kv_num_blocks or None, full_kv_indices or None,
                                    mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod, window,
                                    prefix_lengths or None, prefix_length, bias or None, bias_dtype, lse, out,
                                    d_out, dq, dk, dv, dbias or None, workspace, int(workspace_bytes),
                                    stream or None)
    _check(st, "tri_attn_varlen_bwd")


def tri_attn_varlen_bwd_workspace_size(total_q, H, D, max_seqlen_q, max_seqlen_k, with_bias) -> int:
    return int(load().tri_attn_varlen_bwd_workspace_size(total_q, H, D, max_seqlen_q, max_seqlen_k,
                                                         1 if with_bias else 0))


def tri_attn_varlen_bwd_sink_workspace_size(num_seqs, total_q, H, D, max_seqlen_q, max_seqlen_k, with_bias, window,
                                            sinks) -> int:
    """sinks: -1 where each sequence has its own number."""
    return int(load().tri_attn_varlen_bwd_sink_workspace_size(num_seqs, total_q, H, D, max_seqlen_q, max_seqlen_k,
                                                              1 if with_bias else 0, window, sinks))


def tri_attn_bwd_workspace_size(B, N, H, Q, K, D) -> int:
    return int(load().tri_attn_bwd_workspace_size(B, N, H, Q, K, D))


def _strides4(st):
    """A host array of 4 element strides (b, n, h, row) for the C call, or None (contiguous)."""
    return None if st is None else (ctypes.c_longlong * 4)(*[int(x) for x in st])


def tri_attn_fwd_strided(q, k, v, qkv_dtype, bias, bias_dtype, mask, kv_lengths, B, N, H, Q, K, D, scale, q_strides,
                         k_strides, v_strides, out, lse, max_, stream) -> None:
    """q_strides / k_strides / v_strides: 4 element strides (b, n, h, row) each, or None."""
    qs, ks, vs = _strides4(q_strides), _strides4(k_strides), _strides4(v_strides)
    st = load().tri_attn_fwd_strided(q, k, v, qkv_dtype, bias, bias_dtype, mask or None, kv_lengths or None, B, N, H,
                                     Q, K, D, float(scale), qs, ks, vs, out, lse or None, max_ or None,
                                     stream or None)
    _check(st, "tri_attn_fwd_strided")


def tri_attn_varlen_fwd(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                        max_seqlen_k, H, D, scale, kv_num_blocks, kv_indices, full_kv_num_blocks, full_kv_indices, mask_heads,
                        max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod, out, lse, max_, stream) -> None:
    st = load().tri_attn_varlen_fwd(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                    max_seqlen_q, max_seqlen_k, H, D, float(scale), kv_num_blocks or None, kv_indices or None,
                                    full_kv_num_blocks or None, full_kv_indices or None, mask_heads, max_q_blocks,
                                    max_kv_blocks, block_q, block_k, mask_mod, out, lse or None, max_ or None,
                                    stream or None)
    _check(st, "tri_attn_varlen_fwd")


def tri_attn_varlen_fwd_strided(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                max_seqlen_q, max_seqlen_k, H, D, scale, kv_num_blocks, kv_indices, full_kv_num_blocks,
                                full_kv_indices, mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod,
                                q_row_stride, k_row_stride, v_row_stride, out, lse, max_, stream) -> None:
    st = load().tri_attn_varlen_fwd_strided(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                            max_seqlen_q, max_seqlen_k, H, D, float(scale), kv_num_blocks or None,
                                            kv_indices or None, full_kv_num_blocks or None, full_kv_indices or None,
                                            mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod,
                                            int(q_row_stride), int(k_row_stride), int(v_row_stride), out,
                                            lse or None, max_ or None, stream or None)
    _check(st, "tri_attn_varlen_fwd_strided")


def tri_attn_varlen_fwd_masked(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                               max_seqlen_q, max_seqlen_k, H, D, scale, kv_num_blocks, kv_indices, full_kv_num_blocks,
                               full_kv_indices, mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod,
                               window, prefix_lengths, prefix_length, bias, bias_dtype, q_row_stride, k_row_stride,
                               v_row_stride, out, lse, max_, stream) -> None:
    st = load().tri_attn_varlen_fwd_masked(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                           max_seqlen_q, max_seqlen_k, H, D, float(scale), kv_num_blocks or None,
                                           kv_indices or None, full_kv_num_blocks or None, full_kv_indices or None,
                                           mask_heads, max_q_blocks, max_kv_blocks, block_q, block_k, mask_mod,
                                           int(window), prefix_lengths or None, int(prefix_length), bias or None,
                                           int(bias_dtype), int(q_row_stride), int(k_row_stride), int(v_row_stride), out,
                                           lse or None, max_ or None, stream or None)
    _check(st, "tri_attn_varlen_fwd_masked")


def tri_attn_rotary(q, k, dtype, positions, turns, rotary_dim, interleaved, mscale, inverse, total, Hq, Hk, D,
                    q_row_stride, k_row_stride, q_out_row_stride, k_out_row_stride, q_out, k_out, stream) -> None:
    """Rotary positions (inverse: their gradient); k / k_out 0 with Hk = 0."""
    st = load().tri_attn_rotary(q, k or None, dtype, positions, turns, rotary_dim, 1 if interleaved else 0, mscale,
                                1 if inverse else 0, total, Hq, Hk, D, q_row_stride, k_row_stride, q_out_row_stride,
                                k_out_row_stride, q_out, k_out or None, stream or None)
    _check(st, "tri_attn_rotary")


def strides3(st):
    """A host array of 3 element strides (page, head, slot) for the C calls on a paged cache."""
    return (ctypes.c_longlong * 3)(*[int(x) for x in st])


def tri_attn_kv_append(q, k, v, dtype, cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hq, Hk, D,
                       q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, positions, turns, rotary_dim,
                       interleaved, mscale, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages, page_size,
                       max_pages, k_strides, v_strides, q_out, stream) -> None:
    """k_strides / v_strides: None (contiguous) or a host array of ``strides3``."""
    st = load().tri_attn_kv_append(q or None, k, v, dtype, cu_seqlens or None, kv_lengths, page_table, num_seqs, total,
                                   max_seqlen, Hq, Hk, D, q_row_stride, k_row_stride, v_row_stride, q_out_row_stride,
                                   positions or None, turns or None, rotary_dim, 1 if interleaved else 0, mscale,
                                   k_cache, v_cache, cache_dtype, k_scale or None, v_scale or None, num_pages,
                                   page_size, max_pages, k_strides, v_strides, q_out or None, stream or None)
    _check(st, "tri_attn_kv_append")


@functools.lru_cache(maxsize=256)
def tri_attn_paged_workspace_size(dtype, max_seqlen_q, Hq, Hk, D) -> int:
    return int(load().tri_attn_paged_workspace_size(dtype, max_seqlen_q, Hq, Hk, D))


def tri_attn_paged_fwd(q, dtype, cu_seqlens_q, kv_lengths, page_table, num_seqs, total_q, max_seqlen_q, Hq, Hk, D,
                       q_row_stride, scale, window, sinks, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                       page_size, max_pages, k_strides, v_strides, out, lse, workspace, workspace_bytes,
                       stream) -> None:
    """k_strides / v_strides: None (contiguous) or a host array of ``strides3``."""
    st = load().tri_attn_paged_fwd(q, dtype, cu_seqlens_q or None, kv_lengths, page_table, num_seqs, total_q,
                                   max_seqlen_q, Hq, Hk, D, q_row_stride, scale, window, sinks, k_cache, v_cache,
                                   cache_dtype, k_scale or None, v_scale or None, num_pages, page_size, max_pages,
                                   k_strides, v_strides, out, lse or None, workspace, workspace_bytes, stream or None)
    _check(st, "tri_attn_paged_fwd")


def tri_attn_mask_to_kv_lengths(mask, B, N, K, kv_lengths, nonprefix_count, stream) -> None:
    st = load().tri_attn_mask_to_kv_lengths(mask, B, N, K, kv_lengths, nonprefix_count or None, stream or None)
    _check(st, "tri_attn_mask_to_kv_lengths")


def tri_attn_get_status(stream) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(load().tri_attn_get_status(stream or None))


def tri_attn_version() -> int:
    return int(load().tri_attn_version())
