"""Python binding of libfattn: exact attention forward, backward and paged decode on GB300.

The C ABI (``include/fattn.h``) is reached through ctypes.  The functions
``fa_forward``, ``fa_forward_fp32``, ``fa_backward`` and ``fa_paged_decode`` take the same
arguments as their C counterparts (device pointers as ints, sizes, a stream
handle) and only marshal them; every step of the computation runs in the CUDA
kernels of ``libfattn.so``.  ``forward``, ``backward`` and ``paged_decode`` are torch
conveniences that allocate the outputs and pass the tensors' device pointers; so
are ``qk_norm_rope``, ``qk_norm_rope_cache``, ``qk_norm_rope_backward`` (norm and
rotation of queries and keys), ``forward_packed``, ``backward_packed`` (prompts of
different lengths), ``paged_prefill`` (chunks of new tokens over a paged cache), their
forms with a sliding window (``forward_packed_window``, ``backward_packed_window``,
``paged_prefill_window``) and ``paged_prefill_shared`` (sequences that share a prefix).

There is no fallback: if ``libfattn.so`` is missing, cannot be loaded, or the
device is not an sm_103 GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading

__all__ = ["fa_forward", "fa_forward_f16", "fa_forward_masked", "forward_masked", "fa_forward_fp32", "fa_paged_decode", "fa_paged_decode_noalloc",
           "fa_backward", "fa_backward_workspace_bytes", "backward", "fa_paged_decode_gqa",
           "fa_decode_gqa_select",
           "fa_status_string", "fa_quantize_fp8", "fa_quantize_fp8_workspace_bytes",
           "fa_fp8_vt_stride", "fa_forward_fp8", "quantize_fp8", "forward_fp8", "Fp8Inputs",
           "fa_qk_norm_rope", "fa_qk_norm_rope_f16", "fa_qk_norm_rope_fp32",
           "fa_qk_norm_rope_cache", "fa_qk_norm_rope_backward_workspace_bytes",
           "fa_qk_norm_rope_backward", "fa_qk_norm_rope_backward_f16",
           "fa_qk_norm_rope_backward_fp32", "rope_frequencies", "qk_norm_rope",
           "qk_norm_rope_cache", "qk_norm_rope_backward", "fa_forward_packed",
           "fa_forward_packed_f16", "forward_packed", "fa_backward_packed",
           "fa_backward_packed_workspace_bytes", "backward_packed", "fa_paged_prefill",
           "fa_paged_prefill_workspace_bytes", "paged_prefill", "fa_forward_packed_window",
           "fa_forward_packed_window_f16", "forward_packed_window", "fa_backward_packed_window",
           "fa_backward_packed_window_workspace_bytes", "backward_packed_window",
           "fa_paged_prefill_window",
           "fa_paged_prefill_window_workspace_bytes", "paged_prefill_window",
           "fa_paged_prefill_shared", "fa_paged_prefill_shared_workspace_bytes",
           "paged_prefill_shared",
           "fa_device_status", "fa_release", "forward", "paged_decode", "FattnError",
           "library_path", "load"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libfattn.so")
_lock = threading.Lock()
_lib = None

FA_OK = 0
STATUS_NAMES = {0: "FA_OK", -1: "FA_ERR_INVALID_ARG", -2: "FA_ERR_UNSUPPORTED",
                -3: "FA_ERR_ALIGNMENT", -4: "FA_ERR_CUDA", -5: "FA_ERR_TIMEOUT",
                -6: "FA_ERR_NO_MEMORY", -7: "FA_ERR_NO_DEVICE"}


class FattnError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed: {STATUS_NAMES.get(status, status)} "
                         f"({fa_status_string(status)})")


def library_path() -> str:
    return _LIB_PATH


_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_ll = ctypes.c_longlong
_PREP = [_vp] * 8 + [_i] * 6 + [_ll, _ll, _f, _f, _vp]
_PREP_BWD = [_vp] * 12 + [_i] * 6 + [_ll, _ll, _f, _f, _vp, ctypes.c_ulonglong, _vp]
EXPORTS = {
    "fa_forward": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_forward_fp32": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_forward_f16": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_forward_masked": ([_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_longlong, _i, _i, _i, _i, _f,
                           _vp], _i),
    "fa_paged_decode": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_paged_decode_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_paged_decode_gqa": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_backward_workspace_bytes": ([_i, _i, _i, _i], ctypes.c_ulonglong),
    "fa_backward": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                     ctypes.c_ulonglong, _vp], _i),
    "fa_quantize_fp8_workspace_bytes": ([_i, _i, _i, _i], ctypes.c_ulonglong),
    "fa_fp8_vt_stride": ([_i], ctypes.c_longlong),
    "fa_quantize_fp8": ([_vp] * 10 + [_i, _i, _i, _i, _vp, ctypes.c_ulonglong, _vp], _i),
    "fa_forward_fp8": ([_vp] * 8 + [_i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_qk_norm_rope": (_PREP, _i),
    "fa_qk_norm_rope_f16": (_PREP, _i),
    "fa_qk_norm_rope_fp32": (_PREP, _i),
    "fa_qk_norm_rope_cache": ([_vp] * 11 + [_i] * 8 + [_ll] * 3 + [_f, _f, _vp], _i),
    "fa_qk_norm_rope_backward_workspace_bytes": ([_i, _i], ctypes.c_ulonglong),
    "fa_qk_norm_rope_backward": (_PREP_BWD, _i),
    "fa_qk_norm_rope_backward_f16": (_PREP_BWD, _i),
    "fa_qk_norm_rope_backward_fp32": (_PREP_BWD, _i),
    "fa_forward_packed": ([_vp] * 6 + [_i] * 5 + [_ll] * 3 + [_f, _i, _vp], _i),
    "fa_forward_packed_f16": ([_vp] * 6 + [_i] * 5 + [_ll] * 3 + [_f, _i, _vp], _i),
    "fa_backward_packed_workspace_bytes": ([_i] * 5, ctypes.c_ulonglong),
    "fa_backward_packed": ([_vp] * 10 + [_i] * 5 + [_ll] * 3 + [_f, _i, _vp, ctypes.c_ulonglong,
                                                               _vp], _i),
    "fa_paged_prefill_workspace_bytes": ([_i] * 5, ctypes.c_ulonglong),
    "fa_paged_prefill": ([_vp] * 7 + [_i] * 8 + [_ll, _f, _vp, ctypes.c_ulonglong, _vp], _i),
    "fa_forward_packed_window": ([_vp] * 6 + [_i] * 5 + [_ll] * 3 + [_f, _i, _i, _vp], _i),
    "fa_forward_packed_window_f16": ([_vp] * 6 + [_i] * 5 + [_ll] * 3 + [_f, _i, _i, _vp], _i),
    "fa_backward_packed_window_workspace_bytes": ([_i] * 7, ctypes.c_ulonglong),
    "fa_backward_packed_window": ([_vp] * 10 + [_i] * 5 + [_ll] * 3
                                  + [_f, _i, _i, _vp, ctypes.c_ulonglong, _vp], _i),
    "fa_paged_prefill_window_workspace_bytes": ([_i] * 7, ctypes.c_ulonglong),
    "fa_paged_prefill_window": ([_vp] * 7 + [_i] * 8 + [_ll, _f, _i, _i, _vp, ctypes.c_ulonglong,
                                                        _vp], _i),
    "fa_paged_prefill_shared_workspace_bytes": ([_i] * 6, ctypes.c_ulonglong),
    "fa_paged_prefill_shared": ([_vp] * 9 + [_i] * 9 + [_ll, _f, _vp, ctypes.c_ulonglong, _vp],
                                _i),
    "fa_status_string": ([_i], ctypes.c_char_p),
    "fa_device_status": ([], _i),
    "fa_release": ([], None),
    "fa_debug_inject_fault": ([_i], _i),
    "fa_decode_gqa_select": ([_i], _i),
    "fa_version": ([], _i),
}


def load():
    """Loads libfattn.so (raising if it is absent) and declares its exports."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"libfattn.so not found at {_LIB_PATH}; build it with "
                "`python -m exact_attention_11_gb300._build` (needs nvcc)")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (args, res) in EXPORTS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(name: str, rc: int) -> int:
    if rc != FA_OK:
        raise FattnError(name, rc)
    return rc


# ---------------------------------------------------------------- raw C ABI
def fa_forward(q, k, v, o, lse, B, H, N, d, scale, causal, stream) -> int:
    return _check("fa_forward", load().fa_forward(q, k, v, o, lse, B, H, N, d, scale,
                                                  int(causal), stream))


def fa_forward_f16(q, k, v, o, lse, B, H, N, d, scale, causal, stream) -> int:
    return _check("fa_forward_f16", load().fa_forward_f16(q, k, v, o, lse, B, H, N, d, scale,
                                                          int(causal), stream))


def fa_forward_masked(q, k, v, o, lse, mask, mask_bh_stride, B, H, N, d, scale, stream) -> int:
    return _check("fa_forward_masked", load().fa_forward_masked(
        q, k, v, o, lse, mask, mask_bh_stride, B, H, N, d, scale, stream))


def fa_forward_fp32(q, k, v, o, lse, B, H, N, d, scale, causal, stream) -> int:
    return _check("fa_forward_fp32", load().fa_forward_fp32(q, k, v, o, lse, B, H, N, d, scale,
                                                            int(causal), stream))


def fa_paged_decode(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_heads,
                    head_size, block_size, max_num_blocks_per_seq, scale, stream) -> int:
    return _check("fa_paged_decode", load().fa_paged_decode(
        q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_heads, head_size,
        block_size, max_num_blocks_per_seq, scale, stream))


def fa_paged_decode_gqa(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs,
                        num_heads, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                        scale, stream) -> int:
    return _check("fa_paged_decode_gqa", load().fa_paged_decode_gqa(
        q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_heads, num_kv_heads,
        head_size, block_size, max_num_blocks_per_seq, scale, stream))


def fa_paged_decode_noalloc(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs,
                            num_heads, head_size, block_size, max_num_blocks_per_seq, scale,
                            stream) -> int:
    """fa_paged_decode for callers that cannot allocate device memory during
    the call (a process whose memory pool owns all of HBM, a loop that cannot
    afford cudaMalloc's synchronisation).  The split-K scratch is a fixed
    12 MiB device array inside the library; larger problems raise
    FattnError(FA_ERR_UNSUPPORTED).  All calls on a device share that array,
    so calls that overlap on the GPU must not be issued; the first call on a
    device should come before any stream capture."""
    return _check("fa_paged_decode_noalloc", load().fa_paged_decode_noalloc(
        q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_heads, head_size,
        block_size, max_num_blocks_per_seq, scale, stream))


def fa_backward_workspace_bytes(B, H, N, d) -> int:
    return int(load().fa_backward_workspace_bytes(B, H, N, d))


def fa_backward(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                workspace_bytes, stream) -> int:
    return _check("fa_backward", load().fa_backward(
        q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, int(causal), workspace,
        workspace_bytes, stream))


def fa_quantize_fp8_workspace_bytes(B, H, N, d) -> int:
    return int(load().fa_quantize_fp8_workspace_bytes(B, H, N, d))


def fa_fp8_vt_stride(N) -> int:
    return int(load().fa_fp8_vt_stride(N))


def fa_quantize_fp8(q, k, v, signs, q8, k8, vt8, q_scale, k_scale, v_scale, B, H, N, d,
                    workspace, workspace_bytes, stream) -> int:
    return _check("fa_quantize_fp8", load().fa_quantize_fp8(
        q, k, v, signs, q8, k8, vt8, q_scale, k_scale, v_scale, B, H, N, d, workspace,
        workspace_bytes, stream))


def fa_forward_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, o, lse, B, H, N, d, scale, causal,
                   stream) -> int:
    return _check("fa_forward_fp8", load().fa_forward_fp8(
        q8, k8, vt8, q_scale, k_scale, v_scale, o, lse, B, H, N, d, scale, int(causal), stream))


def _prep_call(name):
    def call(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, num_tokens, num_heads,
             num_kv_heads, d, rot_dim, interleaved, q_stride, k_stride, eps, mscale,
             stream) -> int:
        return _check(name, getattr(load(), name)(
            q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, num_tokens, num_heads,
            num_kv_heads, d, rot_dim, int(interleaved), q_stride, k_stride, eps, mscale, stream))
    call.__name__ = call.__qualname__ = name
    return call


def _prep_backward_call(name):
    def call(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, dq_weight,
             dk_weight, num_tokens, num_heads, num_kv_heads, d, rot_dim, interleaved, q_stride,
             k_stride, eps, mscale, workspace, workspace_bytes, stream) -> int:
        return _check(name, getattr(load(), name)(
            dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, dq_weight,
            dk_weight, num_tokens, num_heads, num_kv_heads, d, rot_dim, int(interleaved),
            q_stride, k_stride, eps, mscale, workspace, workspace_bytes, stream))
    call.__name__ = call.__qualname__ = name
    return call


fa_qk_norm_rope = _prep_call("fa_qk_norm_rope")
fa_qk_norm_rope_f16 = _prep_call("fa_qk_norm_rope_f16")
fa_qk_norm_rope_fp32 = _prep_call("fa_qk_norm_rope_fp32")
fa_qk_norm_rope_backward = _prep_backward_call("fa_qk_norm_rope_backward")
fa_qk_norm_rope_backward_f16 = _prep_backward_call("fa_qk_norm_rope_backward_f16")
fa_qk_norm_rope_backward_fp32 = _prep_backward_call("fa_qk_norm_rope_backward_fp32")


def fa_qk_norm_rope_cache(q, k, v, q_weight, k_weight, positions, inv_freq, slots, q_out, k_cache,
                          v_cache, num_tokens, num_heads, num_kv_heads, head_size, block_size,
                          num_blocks, rot_dim, interleaved, q_stride, k_stride, v_stride, eps,
                          mscale, stream) -> int:
    return _check("fa_qk_norm_rope_cache", load().fa_qk_norm_rope_cache(
        q, k, v, q_weight, k_weight, positions, inv_freq, slots, q_out, k_cache, v_cache,
        num_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks, rot_dim,
        int(interleaved), q_stride, k_stride, v_stride, eps, mscale, stream))


def fa_qk_norm_rope_backward_workspace_bytes(num_tokens, d) -> int:
    return int(load().fa_qk_norm_rope_backward_workspace_bytes(num_tokens, d))


def fa_forward_packed(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                      num_kv_heads, d, q_stride, k_stride, v_stride, scale, causal,
                      stream) -> int:
    return _check("fa_forward_packed", load().fa_forward_packed(
        q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads, num_kv_heads, d, q_stride,
        k_stride, v_stride, scale, int(causal), stream))


def fa_forward_packed_f16(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                          num_kv_heads, d, q_stride, k_stride, v_stride, scale, causal,
                          stream) -> int:
    return _check("fa_forward_packed_f16", load().fa_forward_packed_f16(
        q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads, num_kv_heads, d, q_stride,
        k_stride, v_stride, scale, int(causal), stream))


def fa_backward_packed_workspace_bytes(num_seqs, total_tokens, num_heads, num_kv_heads, d) -> int:
    return int(load().fa_backward_packed_workspace_bytes(num_seqs, total_tokens, num_heads,
                                                         num_kv_heads, d))


def fa_backward_packed(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs, total_tokens,
                       num_heads, num_kv_heads, d, q_stride, k_stride, v_stride, scale, causal,
                       workspace, workspace_bytes, stream) -> int:
    return _check("fa_backward_packed", load().fa_backward_packed(
        q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs, total_tokens, num_heads,
        num_kv_heads, d, q_stride, k_stride, v_stride, scale, int(causal), workspace,
        workspace_bytes, stream))


def fa_paged_prefill_workspace_bytes(num_seqs, total_tokens, num_heads, num_kv_heads,
                                     max_num_blocks_per_seq) -> int:
    return int(load().fa_paged_prefill_workspace_bytes(
        num_seqs, total_tokens, num_heads, num_kv_heads, max_num_blocks_per_seq))


def fa_paged_prefill(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs,
                     total_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                     max_num_blocks_per_seq, q_stride, scale, workspace, workspace_bytes,
                     stream) -> int:
    return _check("fa_paged_prefill", load().fa_paged_prefill(
        q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs, total_tokens,
        num_heads, num_kv_heads, head_size, block_size, num_blocks, max_num_blocks_per_seq,
        q_stride, scale, workspace, workspace_bytes, stream))


def _mask_lengths(window, sinks):
    """A window and a number of first tokens (whole numbers) as C ints that see the same:
    past 2^30, which no sequence has, 2^30 (ctypes would cut them to their low 32 bits)."""
    window, sinks = operator.index(window), operator.index(sinks)
    return max(min(window, 1 << 30), -1), max(min(sinks, 1 << 30), -1)


def fa_forward_packed_window(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                             num_kv_heads, d, q_stride, k_stride, v_stride, scale, window, sinks,
                             stream) -> int:
    return _check("fa_forward_packed_window", load().fa_forward_packed_window(
        q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads, num_kv_heads, d, q_stride,
        k_stride, v_stride, scale, *_mask_lengths(window, sinks), stream))


def fa_forward_packed_window_f16(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                                 num_kv_heads, d, q_stride, k_stride, v_stride, scale, window,
                                 sinks, stream) -> int:
    return _check("fa_forward_packed_window_f16", load().fa_forward_packed_window_f16(
        q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads, num_kv_heads, d, q_stride,
        k_stride, v_stride, scale, *_mask_lengths(window, sinks), stream))


def fa_backward_packed_window_workspace_bytes(num_seqs, total_tokens, num_heads, num_kv_heads, d,
                                              window, sinks) -> int:
    return int(load().fa_backward_packed_window_workspace_bytes(
        num_seqs, total_tokens, num_heads, num_kv_heads, d, *_mask_lengths(window, sinks)))


def fa_backward_packed_window(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs,
                              total_tokens, num_heads, num_kv_heads, d, q_stride, k_stride,
                              v_stride, scale, window, sinks, workspace, workspace_bytes,
                              stream) -> int:
    return _check("fa_backward_packed_window", load().fa_backward_packed_window(
        q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs, total_tokens, num_heads,
        num_kv_heads, d, q_stride, k_stride, v_stride, scale, *_mask_lengths(window, sinks),
        workspace, workspace_bytes, stream))


def fa_paged_prefill_window_workspace_bytes(num_seqs, total_tokens, num_heads, num_kv_heads,
                                            max_num_blocks_per_seq, window, sinks) -> int:
    return int(load().fa_paged_prefill_window_workspace_bytes(
        num_seqs, total_tokens, num_heads, num_kv_heads, max_num_blocks_per_seq,
        *_mask_lengths(window, sinks)))


def fa_paged_prefill_window(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out,
                            num_seqs, total_tokens, num_heads, num_kv_heads, head_size,
                            block_size, num_blocks, max_num_blocks_per_seq, q_stride, scale,
                            window, sinks, workspace, workspace_bytes, stream) -> int:
    return _check("fa_paged_prefill_window", load().fa_paged_prefill_window(
        q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs, total_tokens,
        num_heads, num_kv_heads, head_size, block_size, num_blocks, max_num_blocks_per_seq,
        q_stride, scale, *_mask_lengths(window, sinks), workspace, workspace_bytes, stream))


def fa_paged_prefill_shared_workspace_bytes(num_seqs, total_tokens, num_groups, num_heads,
                                            num_kv_heads, max_num_blocks_per_seq) -> int:
    return int(load().fa_paged_prefill_shared_workspace_bytes(
        num_seqs, total_tokens, num_groups, num_heads, num_kv_heads, max_num_blocks_per_seq))


def fa_paged_prefill_shared(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens,
                            cu_groups, prefix_lens, out, num_seqs, total_tokens, num_groups,
                            num_heads, num_kv_heads, head_size, block_size, num_blocks,
                            max_num_blocks_per_seq, q_stride, scale, workspace, workspace_bytes,
                            stream) -> int:
    return _check("fa_paged_prefill_shared", load().fa_paged_prefill_shared(
        q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, cu_groups, prefix_lens, out,
        num_seqs, total_tokens, num_groups, num_heads, num_kv_heads, head_size, block_size,
        num_blocks, max_num_blocks_per_seq, q_stride, scale, workspace, workspace_bytes, stream))


def fa_status_string(status: int) -> str:
    try:
        return load().fa_status_string(status).decode()
    except Exception:  # library missing: still give a name
        return STATUS_NAMES.get(status, "unknown")


def fa_device_status() -> int:
    return load().fa_device_status()


def fa_release() -> None:
    load().fa_release()


def fa_debug_inject_fault(mode: int) -> int:
    """Test hook: arm a lost-copy fault in the next forward (1) or backward
    (2) launch on the current device, or disarm (0) (see fattn.h)."""
    return _check("fa_debug_inject_fault", load().fa_debug_inject_fault(mode))


def fa_decode_gqa_select(impl: int) -> int:
    """Kernel for fa_paged_decode_gqa: 0 = automatic (default), 1 = the
    CUDA-core kernel only, 2 = the tensor-core kernel only (see fattn.h)."""
    return _check("fa_decode_gqa_select", load().fa_decode_gqa_select(impl))


# ---------------------------------------------------------------- torch helpers
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def forward(q, k, v, scale=None, causal=False, out=None, lse=None, want_lse=True):
    """Exact attention on [B,H,N,d] CUDA tensors (bf16, fp16 or fp32, contiguous).

    Returns (O, LSE) with O in the input dtype and LSE fp32 [B,H,N] (None when
    ``want_lse`` is False).  Runs on the current torch stream."""
    import torch
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B,H,N,d] shape")
    if not (q.is_cuda and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous CUDA tensors")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.bfloat16, torch.float16,
                                                                torch.float32):
        raise ValueError("q, k, v must all be bf16, all fp16 or all fp32")
    B, H, N, d = q.shape
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fn = {torch.bfloat16: fa_forward, torch.float16: fa_forward_f16,
          torch.float32: fa_forward_fp32}[q.dtype]
    fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, float(scale), bool(causal),
       _stream(q))
    return out, lse


def forward_masked(q, k, v, mask, scale=None, out=None, lse=None):
    """Exact attention with a boolean mask on bf16 [B,H,N,d] CUDA tensors.
    mask: bool or uint8 CUDA tensor, [N,N] (shared) or [B,H,N,N] (nonzero =
    visible).  Returns (O, LSE); rows with no visible key give O = 0,
    LSE = -inf."""
    import torch
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B,H,N,d] shape")
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous() and t.dtype == torch.bfloat16):
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    B, H, N, d = q.shape
    m = mask.to(torch.uint8) if mask.dtype == torch.bool else mask
    if not (m.is_cuda and m.is_contiguous() and m.dtype == torch.uint8):
        raise ValueError("mask must be a contiguous bool or uint8 CUDA tensor")
    if tuple(m.shape) == (N, N):
        stride = 0
    elif tuple(m.shape) == (B, H, N, N):
        stride = N * N
    else:
        raise ValueError("mask must be [N,N] or [B,H,N,N]")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_forward_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(m), stride, B, H, N,
                      d, float(scale), _stream(q))
    return out, lse


def backward(q, k, v, o, lse, dout, scale=None, causal=False, workspace=None):
    """Gradients (dQ, dK, dV) of the bf16 forward on [B,H,N,d] CUDA tensors.

    ``o`` and ``lse`` are what ``forward`` returned for the same q, k, v,
    scale and causal.  ``workspace`` (optional) is a CUDA tensor of at least
    ``fa_backward_workspace_bytes`` bytes; one is allocated when it is None.
    Runs on the current torch stream."""
    import torch
    for t in (q, k, v, o, dout):
        if t.dim() != 4 or t.shape != q.shape:
            raise ValueError("q, k, v, o, dout must share one [B,H,N,d] shape")
        if not (t.is_cuda and t.is_contiguous() and t.dtype == torch.bfloat16):
            raise ValueError("q, k, v, o, dout must be contiguous bf16 CUDA tensors")
    B, H, N, d = q.shape
    if lse is None or tuple(lse.shape) != (B, H, N) or lse.dtype != torch.float32 \
            or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B,H,N] tensor")
    if scale is None:
        scale = d ** -0.5
    nbytes = fa_backward_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                _ptr(dv), B, H, N, d, float(scale), bool(causal), _ptr(workspace), ws_bytes,
                _stream(q))
    return dq, dk, dv


def paged_decode(q, k_cache, v_cache, block_tables, context_lens, scale=None, out=None):
    """Single-query paged decode on CUDA tensors in the layouts of fattn.h.
    The caches' second axis is the key/value head count Hk; Hk < H selects
    the grouped-head decode (fa_paged_decode_gqa)."""
    import torch
    S, H, D = q.shape
    nb, Hk, Dx, bs, x = k_cache.shape
    if Hk <= 0 or H % Hk != 0 or Dx * x != D or tuple(v_cache.shape) != (nb, Hk, D, bs):
        raise ValueError("inconsistent cache shapes")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    for t in (q, k_cache, v_cache, block_tables, context_lens):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("all decode inputs must be contiguous CUDA tensors")
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if Hk == H:
        fa_paged_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                        _ptr(context_lens), _ptr(out), S, H, D, bs, block_tables.shape[1],
                        float(scale), _stream(q))
    else:
        fa_paged_decode_gqa(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            _ptr(context_lens), _ptr(out), S, H, Hk, D, bs,
                            block_tables.shape[1], float(scale), _stream(q))
    return out


class Fp8Inputs:
    """E4M3 codes and dequantization scales of one attention problem, in the
    layouts of fa_quantize_fp8: q8, k8 uint8 [B,H,N,d]; vt8 uint8 [B,H,d,Npad]
    (V transposed); q_scale, k_scale fp32 [B,H,ceil(N/128)]; v_scale fp32
    [B,H]."""

    def __init__(self, q8, k8, vt8, q_scale, k_scale, v_scale, shape):
        self.q8, self.k8, self.vt8 = q8, k8, vt8
        self.q_scale, self.k_scale, self.v_scale = q_scale, k_scale, v_scale
        self.shape = tuple(shape)


def quantize_fp8(q, k, v, signs=None, workspace=None, out=None):
    """Block-quantizes bf16 [B,H,N,128] CUDA tensors to E4M3 (fa_quantize_fp8).
    ``signs``: optional fp32 CUDA tensor of 128 values +-1 for the random
    orthogonal transform of q and k.  ``out``: an Fp8Inputs of the same shape
    to write into.  Returns an Fp8Inputs.  Runs on the current torch stream."""
    import torch
    for t in (q, k, v):
        if t.dim() != 4 or t.shape != q.shape:
            raise ValueError("q, k, v must share one [B,H,N,d] shape")
        if not (t.is_cuda and t.is_contiguous() and t.dtype == torch.bfloat16):
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    B, H, N, d = q.shape
    if signs is not None and not (signs.is_cuda and signs.is_contiguous()
                                  and signs.dtype == torch.float32 and signs.numel() == d):
        raise ValueError("signs must be a contiguous fp32 CUDA tensor of d values")
    if out is None:
        dev = q.device
        nblk = (N + 127) // 128
        npad = fa_fp8_vt_stride(N)
        out = Fp8Inputs(torch.empty((B, H, N, d), dtype=torch.uint8, device=dev),
                        torch.empty((B, H, N, d), dtype=torch.uint8, device=dev),
                        torch.empty((B, H, d, npad), dtype=torch.uint8, device=dev),
                        torch.empty((B, H, nblk), dtype=torch.float32, device=dev),
                        torch.empty((B, H, nblk), dtype=torch.float32, device=dev),
                        torch.empty((B, H), dtype=torch.float32, device=dev), q.shape)
    elif out.shape != tuple(q.shape):
        raise ValueError("out was made for another shape")
    nbytes = fa_quantize_fp8_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q.device)
    fa_quantize_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(signs), _ptr(out.q8), _ptr(out.k8),
                    _ptr(out.vt8), _ptr(out.q_scale), _ptr(out.k_scale), _ptr(out.v_scale),
                    B, H, N, d, _ptr(workspace), workspace.numel() * workspace.element_size(),
                    _stream(q))
    return out


def forward_fp8(x, scale=None, causal=False, out=None, lse=None, want_lse=True):
    """The FP8 forward (fa_forward_fp8) on an Fp8Inputs.  Returns (O bf16
    [B,H,N,d], LSE fp32 [B,H,N] or None).  Runs on the current torch stream."""
    import torch
    B, H, N, d = x.shape
    if scale is None:
        scale = d ** -0.5
    dev = x.q8.device
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    fa_forward_fp8(_ptr(x.q8), _ptr(x.k8), _ptr(x.vt8), _ptr(x.q_scale), _ptr(x.k_scale),
                   _ptr(x.v_scale), _ptr(out), _ptr(lse), B, H, N, d, float(scale),
                   bool(causal), _stream(x.q8))
    return out, lse


# -------------------------------------------- packed tokens: [tokens, heads, d] tensors
# These calls are short (a decode step's take a few microseconds on the GPU), so
# their checks touch each tensor's attributes as few times as they can.
def _on_device(fn):
    """Runs ``fn`` with its first tensor's device current: the C calls work on
    the current device, and a caller's may be another one."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def run(*args, **kwargs):
        first = args[0] if args else kwargs.get(name)
        if first is None:
            return fn(*args, **kwargs)      # a TypeError that names what is missing
        dev = first.get_device()
        if dev >= 0 and dev != _torch()._C._cuda_getDevice():
            with _torch().cuda.device(dev):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return run


@functools.lru_cache(None)
def _torch():
    import torch
    return torch


def _raw_stream(index):
    """Handle of the current torch stream of CUDA device ``index``."""
    return _torch()._C._cuda_getCurrentRawStream(index)   # current_stream() builds an object first


def _rows(name, t, T, heads, d, dtype, dev):
    """Checks a [T, heads, d] tensor with dense heads; its token stride in elements."""
    if t.shape != (T, heads, d) or t.dtype != dtype or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a [{T},{heads},{d}] {dtype} tensor on the CUDA device "
                         f"of the rest, not {tuple(t.shape)} {t.dtype} on {t.device}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be dense")
    return s0 if T > 1 else max(heads * d, 1)


def _dense(name, t, dtype, dev, numel=None):
    """Checks a contiguous tensor and returns its address."""
    if t.dtype != dtype or t.get_device() != dev or not t.is_contiguous() \
            or (numel is not None and t.numel() != numel):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor"
                         + (f" of {numel} values" if numel is not None else "")
                         + " on the CUDA device of the rest")
    return t.data_ptr()


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_context=4096,
                     beta_slow=1.0, beta_fast=32.0, device=None, ramp="index"):
    """Rotary frequencies (fp64 [rot_dim/2], radians per position) and the
    factor ``mscale`` that goes with them, for ``qk_norm_rope``.

    ``scaling`` stretches them ``factor`` times beyond ``original_context``:
    None, "linear" (position interpolation: every frequency / factor), "ntk"
    (the base grows so that the lowest frequency is divided by factor and the
    highest stays) or "yarn" (by wavelength: frequencies that turn more than
    ``beta_fast`` times over the original context stay, those that turn less
    than ``beta_slow`` times are divided by factor, with a ramp between; mscale
    = 0.1 ln(factor) + 1).  mscale is 1 for the others.

    ``ramp`` of "yarn": "index", linear in the frequency's index between the
    indices of beta_fast and beta_slow turns, rounded down and up -- what
    models trained with YaRN use -- or "turns", linear in the number of turns,
    as the method's paper writes it."""
    import math

    import torch
    if rot_dim < 0 or rot_dim % 2 != 0:
        raise ValueError("rot_dim must be even")
    if scaling not in (None, "linear", "ntk", "yarn") or not factor >= 1.0 or not base > 1.0:
        raise ValueError("scaling is None, 'linear', 'ntk' or 'yarn', factor >= 1 and base > 1")
    if ramp not in ("index", "turns"):
        raise ValueError("ramp is 'index' or 'turns'")
    if scaling == "yarn" and not (beta_fast > beta_slow and original_context > 0):
        raise ValueError("beta_fast > beta_slow and original_context > 0")
    if scaling == "yarn" and ramp == "index" and not beta_slow > 0:
        raise ValueError("the ramp over the index needs beta_slow > 0")
    mscale = 1.0
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freq = base ** (-2.0 * i / max(rot_dim, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if ramp == "turns":
            turns = original_context * freq / (2 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        else:
            def index(turns):   # i of base^(-2 i / rot_dim) original_context = 2 pi turns
                far = original_context / (2 * math.pi * turns)
                return rot_dim * math.log(far) / (2 * math.log(base))
            first = max(math.floor(index(beta_fast)), 0)
            last = min(math.ceil(index(beta_slow)), rot_dim - 1)
            # (Bounds that meet, by the clamps, make a step.)
            keep = 1.0 - ((i - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return freq.to(device), mscale


def _workspace(t, dev):
    """Bytes of a caller's workspace tensor."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the CUDA device of the rest")
    return t.numel() * t.element_size()


def _prep_args(q, k, positions, inv_freq, q_weight, k_weight):
    """Checks the inputs that the norm-and-rotation helpers share: T, H, Hk, d,
    q's type's suffix, device, token strides, the six addresses, rot_dim."""
    T, H, d = q.shape
    Hk = k.shape[1] if k.dim() == 3 else -1
    dtype, dev = q.dtype, q.get_device()
    suffix = _prep_suffix(dtype)
    qs, ks = _rows("q", q, T, H, d, dtype, dev), _rows("k", k, T, Hk, d, dtype, dev)
    i32, f64 = _torch().int32, _torch().float64
    ptrs = (q.data_ptr(), k.data_ptr(),
            None if q_weight is None else _dense("q_weight", q_weight, dtype, dev, d),
            None if k_weight is None else _dense("k_weight", k_weight, dtype, dev, d),
            _dense("positions", positions, i32, dev, T), _dense("inv_freq", inv_freq, f64, dev))
    return T, H, Hk, d, dtype, suffix, dev, qs, ks, ptrs, 2 * inv_freq.numel()


def _prep_suffix(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return ""
    if dtype == torch.float16:
        return "_f16"
    if dtype == torch.float32:
        return "_fp32"
    raise ValueError("q and k must be bf16, fp16 or fp32")


@_on_device
def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, mscale=1.0, q_out=None, k_out=None):
    """RMS norm of each head (where its weight is given) and rotary position
    embedding of q [T,H,d] and k [T,Hk,d] (bf16, fp16 or fp32 CUDA tensors;
    heads dense, any token stride that is a multiple of 16 bytes).

    positions int32 [T]; inv_freq fp64 [rot_dim/2] (``rope_frequencies``): the
    first rot_dim values of a head are rotated.  Returns (q_out, k_out), dense.
    Runs on the current torch stream."""
    torch = _torch()
    T, H, Hk, d, dtype, suffix, dev, qs, ks, ptrs, rot = _prep_args(
        q, k, positions, inv_freq, q_weight, k_weight)
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty((T, Hk, d), dtype=dtype, device=q.device)
    outs = (_dense("q_out", q_out, dtype, dev, T * H * d),
            _dense("k_out", k_out, dtype, dev, T * Hk * d))
    if T == 0:      # empty tensors have no address to pass
        return q_out, k_out
    name = "fa_qk_norm_rope" + suffix
    _check(name, getattr(_lib or load(), name)(
        *ptrs, *outs, T, H, Hk, d, rot, int(interleaved), qs, ks, eps, mscale, _raw_stream(dev)))
    return q_out, k_out


@_on_device
def qk_norm_rope_cache(q, k, v, positions, inv_freq, slots, k_cache, v_cache, q_weight=None,
                       k_weight=None, eps=1e-6, interleaved=False, mscale=1.0, q_out=None):
    """``qk_norm_rope`` for serving (bf16, d = 128): the prepared keys, and v
    [T,Hk,d] as it is, are written into the paged caches of ``paged_decode``
    and ``paged_prefill`` at slots (int64 [T]: block * block_size + offset; a
    slot outside the cache, such as -1, stores nothing).  Returns the prepared
    queries, dense; ``q_out`` may be q itself."""
    torch = _torch()
    T, H, Hk, d, dtype, suffix, dev, qs, ks, ptrs, rot = _prep_args(
        q, k, positions, inv_freq, q_weight, k_weight)
    if suffix != "":
        raise ValueError("the cache form is bf16")
    vs = _rows("v", v, T, Hk, d, dtype, dev)
    nb, bs = _cache_shape(k_cache, v_cache, Hk, d)
    if q_out is None:
        q_out = torch.empty((T, H, d), dtype=dtype, device=q.device)
    rest = (_dense("slots", slots, torch.int64, dev, T),
            _dense("q_out", q_out, dtype, dev, T * H * d),
            _dense("k_cache", k_cache, dtype, dev), _dense("v_cache", v_cache, dtype, dev))
    if T == 0:
        return q_out
    _check("fa_qk_norm_rope_cache", (_lib or load()).fa_qk_norm_rope_cache(
        ptrs[0], ptrs[1], v.data_ptr(), *ptrs[2:], *rest, T, H, Hk, d, bs, nb, rot,
        int(interleaved), qs, ks, vs, eps, mscale, _raw_stream(dev)))
    return q_out


def _cache_shape(k_cache, v_cache, Hk, d):
    """Number and size of the blocks of a pair of paged caches of Hk heads."""
    if k_cache.dim() != 5:
        raise ValueError("inconsistent cache shapes")
    nb, hc, dx, bs, x = k_cache.shape
    if hc != Hk or x != 8 or dx * x != d or v_cache.shape != (nb, Hk, d, bs):
        raise ValueError("inconsistent cache shapes")
    return nb, bs


@_on_device
def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, q_weight=None,
                          k_weight=None, eps=1e-6, interleaved=False, mscale=1.0,
                          workspace=None):
    """Gradients of ``qk_norm_rope``: (dq, dk, dq_weight, dk_weight) from the
    dense gradients dq_out [T,H,d], dk_out [T,Hk,d] of its outputs and its
    inputs.  The weights' gradients are fp32 [d], None where there is no
    weight.  ``workspace`` (optional) is a CUDA tensor of at least
    ``fa_qk_norm_rope_backward_workspace_bytes`` bytes."""
    torch = _torch()
    T, H, Hk, d, dtype, suffix, dev, qs, ks, ptrs, rot = _prep_args(
        q, k, positions, inv_freq, q_weight, k_weight)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise ValueError("dq_out and dk_out must have the shapes of q and k")
    ins = (_dense("dq_out", dq_out, dtype, dev), _dense("dk_out", dk_out, dtype, dev))
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    dqw = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    dkw = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    if T == 0:
        return dq, dk, *(w if w is None else w.zero_() for w in (dqw, dkw))
    lib = _lib or load()
    nbytes = 0
    if workspace is not None:
        nbytes = _workspace(workspace, dev)
    elif dqw is not None or dkw is not None:
        nbytes = lib.fa_qk_norm_rope_backward_workspace_bytes(T, d)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    name = "fa_qk_norm_rope_backward" + suffix
    _check(name, getattr(lib, name)(
        *ins, *ptrs, dq.data_ptr(), dk.data_ptr(), _ptr(dqw), _ptr(dkw), T, H, Hk, d, rot,
        int(interleaved), qs, ks, eps, mscale, _ptr(workspace), nbytes, _raw_stream(dev)))
    return dq, dk, dqw, dkw


def _packed_args(q, k, v, cu_seqlens, dtypes):
    """Checks q, k, v and cu_seqlens of the packed calls."""
    torch = _torch()
    T, H, d = q.shape
    Hk = k.shape[1] if k.dim() == 3 else -1
    dtype, dev = q.dtype, q.get_device()
    if dtype not in dtypes:
        raise ValueError("q, k, v must be " + " or ".join(str(x) for x in dtypes))
    qs = _rows("q", q, T, H, d, dtype, dev)
    ks, vs = _rows("k", k, T, Hk, d, dtype, dev), _rows("v", v, T, Hk, d, dtype, dev)
    cu = _dense("cu_seqlens", cu_seqlens, torch.int32, dev)
    S = cu_seqlens.numel() - 1
    if S < 0:
        raise ValueError("cu_seqlens holds num_seqs + 1 offsets")
    return T, H, Hk, d, S, dtype, dev, qs, ks, vs, cu


@_on_device
def forward_packed(q, k, v, cu_seqlens, scale=None, causal=True, out=None, lse=None,
                   want_lse=True):
    """Exact attention over packed prompts: q [T,H,d], k and v [T,Hk,d] (bf16 or
    fp16 CUDA tensors, heads dense, any token stride that is a multiple of 8
    elements), sequence s in rows cu_seqlens[s] .. cu_seqlens[s+1] - 1
    (int32 [S+1] on the device).  d is 64 or 128; H a multiple of Hk.

    Returns (O [T,H,d], LSE fp32 [H,T] or None).  Rows of no sequence are not
    written (they are uninitialised in tensors made here).  Runs on the current
    torch stream."""
    return _forward_packed("fa_forward_packed", q, k, v, cu_seqlens, scale, out, lse, want_lse,
                           int(causal))


@_on_device
def forward_packed_window(q, k, v, cu_seqlens, window, sinks=0, scale=None, out=None, lse=None,
                          want_lse=True):
    """``forward_packed`` with a sliding window: a query at position p of its
    sequence sees keys j <= p with j > p - window, or j < sinks (the sequence's
    first tokens, which stay visible).  window >= 1, sinks >= 0."""
    return _forward_packed("fa_forward_packed_window", q, k, v, cu_seqlens, scale, out, lse,
                           want_lse, *_window_args(window, sinks))


def _window_args(window, sinks):
    """Checks a window and a number of first tokens."""
    window, sinks = _mask_lengths(window, sinks)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1 and sinks at least 0")
    return window, sinks


def _forward_packed(name, q, k, v, cu_seqlens, scale, out, lse, want_lse, *mask):
    torch = _torch()
    T, H, Hk, d, S, dtype, dev, qs, ks, vs, cu = _packed_args(
        q, k, v, cu_seqlens, (torch.bfloat16, torch.float16))
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty((T, H, d), dtype=dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    o_ptr = _dense("out", out, dtype, dev, T * H * d)
    lse_ptr = None if lse is None else _dense("lse", lse, torch.float32, dev, H * T)
    if T == 0 or S == 0:
        return out, lse
    lib = _lib or load()
    if dtype == torch.float16:
        name += "_f16"
    _check(name, getattr(lib, name)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o_ptr, lse_ptr, cu, S, T, H, Hk, d, qs, ks, vs,
        scale, *mask, _raw_stream(dev)))
    return out, lse


@_on_device
def backward_packed(q, k, v, o, lse, dout, cu_seqlens, scale=None, causal=True, workspace=None):
    """Gradients (dQ [T,H,d], dK [T,Hk,d], dV [T,Hk,d]) of the bf16
    ``forward_packed``; ``o`` and ``lse`` are what it returned for the same q, k,
    v, cu_seqlens, scale and causal, ``dout`` [T,H,d] is dense.  ``workspace``
    (optional) is a CUDA tensor of at least
    ``fa_backward_packed_workspace_bytes`` bytes.  Rows of no sequence are not
    written.  Runs on the current torch stream."""
    return _backward_packed("fa_backward_packed", q, k, v, o, lse, dout, cu_seqlens, scale,
                            workspace, (), int(causal))


@_on_device
def backward_packed_window(q, k, v, o, lse, dout, cu_seqlens, window, sinks=0, scale=None,
                           workspace=None):
    """Gradients (dQ, dK, dV) of the bf16 ``forward_packed_window``, as
    ``backward_packed``; ``o`` and ``lse`` are what it returned for the same q, k,
    v, cu_seqlens, window, sinks and scale.  ``workspace`` (optional) is a CUDA
    tensor of at least ``fa_backward_packed_window_workspace_bytes`` bytes."""
    mask = _window_args(window, sinks)
    return _backward_packed("fa_backward_packed_window", q, k, v, o, lse, dout, cu_seqlens, scale,
                            workspace, mask, *mask)


def _backward_packed(name, q, k, v, o, lse, dout, cu_seqlens, scale, workspace, sizes, *mask):
    """``sizes``: what the workspace depends on besides the tensors' sizes."""
    torch = _torch()
    T, H, Hk, d, S, dtype, dev, qs, ks, vs, cu = _packed_args(q, k, v, cu_seqlens,
                                                              (torch.bfloat16,))
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must have q's shape")
    ins = (_dense("o", o, dtype, dev), _dense("dout", dout, dtype, dev),
           _dense("lse", lse, torch.float32, dev, H * T))
    if scale is None:
        scale = d ** -0.5
    device = q.device
    dq = torch.empty((T, H, d), dtype=dtype, device=device)
    dk = torch.empty((T, Hk, d), dtype=dtype, device=device)
    dv = torch.empty((T, Hk, d), dtype=dtype, device=device)
    if T == 0 or S == 0:
        return dq, dk, dv
    lib = _lib or load()
    if workspace is None:
        nbytes = getattr(lib, name + "_workspace_bytes")(S, T, H, Hk, d, *sizes)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        nbytes = _workspace(workspace, dev)
    _check(name, getattr(lib, name)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *ins, dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), cu, S, T, H, Hk, d, qs, ks, vs, scale, *mask, workspace.data_ptr(),
        nbytes, _raw_stream(dev)))
    return dq, dk, dv


@_on_device
def paged_prefill(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, scale=None,
                  out=None, workspace=None):
    """Attention of new tokens over a paged cache (layouts of ``paged_decode``):
    q bf16 [T,H,128] holds each sequence's chunk in rows cu_seqlens[s] ..
    cu_seqlens[s+1] - 1; the chunk's own keys and values are in the cache
    already and context_lens counts them.  ``workspace`` (optional) is a CUDA
    tensor of at least ``fa_paged_prefill_workspace_bytes`` bytes.  Returns out
    [T,H,128]; rows of no sequence are not written.  Runs on the current torch
    stream."""
    return _paged_prefill("fa_paged_prefill", q, k_cache, v_cache, block_tables, context_lens,
                          cu_seqlens, scale, out, workspace)


@_on_device
def paged_prefill_window(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, window,
                         sinks=0, scale=None, out=None, workspace=None):
    """``paged_prefill`` with a sliding window: a query at position p (the last of
    a sequence at context_lens[s] - 1) sees tokens j <= p with j > p - window, or
    j < sinks.  window >= 1, sinks >= 0.  Table entries of blocks that no query of
    the chunk sees are not used and may hold anything.  ``workspace`` (optional)
    is a CUDA tensor of at least ``fa_paged_prefill_window_workspace_bytes``
    bytes."""
    return _paged_prefill("fa_paged_prefill_window", q, k_cache, v_cache, block_tables,
                          context_lens, cu_seqlens, scale, out, workspace,
                          *_window_args(window, sinks))


@_on_device
def paged_prefill_shared(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, cu_groups,
                         prefix_lens, scale=None, out=None, workspace=None):
    """``paged_prefill`` for sequences that share the cache blocks of a long prefix,
    which is read once for a whole group: sequences cu_groups[g] ..
    cu_groups[g+1] - 1 (int32 [groups + 1] on the device) have the same first
    prefix_lens[g] tokens (int32 [groups]; rounded down to whole blocks), in the
    blocks that each of their rows of ``block_tables`` begins with (not checked).
    The output is that of ``paged_prefill`` for the same tables, up to the order of
    fp32 sums; a sequence whose new tokens do not all lie behind the prefix shares
    nothing.  ``workspace`` (optional) is a CUDA tensor of at least
    ``fa_paged_prefill_shared_workspace_bytes`` bytes."""
    torch = _torch()
    T, H, Hk, S, mb, nb, bs, dev, qs, scale, out, ptrs, out_ptr = _chunk_args(
        q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, scale, out)
    P = prefix_lens.numel()
    groups = (_dense("cu_groups", cu_groups, torch.int32, dev, P + 1),
              _dense("prefix_lens", prefix_lens, torch.int32, dev))
    if T == 0 or S == 0:
        return out
    lib = _lib or load()
    if workspace is not None:
        nbytes = _workspace(workspace, dev)
    else:
        nbytes = lib.fa_paged_prefill_shared_workspace_bytes(S, T, P, H, Hk, mb)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check("fa_paged_prefill_shared", lib.fa_paged_prefill_shared(
        *ptrs, *groups, out_ptr, S, T, P, H, Hk, q.shape[2], bs, nb, mb, qs, scale,
        workspace.data_ptr(), nbytes, _raw_stream(dev)))
    return out


def _chunk_args(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, scale, out):
    """Checks what the chunk helpers share and makes the output."""
    torch = _torch()
    T, H, D = q.shape
    dtype, dev = q.dtype, q.get_device()
    if dtype != torch.bfloat16:
        raise ValueError("q must be bf16")
    qs = _rows("q", q, T, H, D, dtype, dev)
    Hk = k_cache.shape[1] if k_cache.dim() == 5 else -1
    nb, bs = _cache_shape(k_cache, v_cache, Hk, D)
    if block_tables.dim() != 2 or Hk <= 0 or H % Hk != 0:
        raise ValueError("inconsistent cache shapes")
    S, mb = block_tables.shape
    i32 = torch.int32
    ptrs = (q.data_ptr(), _dense("k_cache", k_cache, dtype, dev),
            _dense("v_cache", v_cache, dtype, dev), _dense("block_tables", block_tables, i32, dev),
            _dense("context_lens", context_lens, i32, dev, S),
            _dense("cu_seqlens", cu_seqlens, i32, dev, S + 1))
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((T, H, D), dtype=dtype, device=q.device)
    out_ptr = _dense("out", out, dtype, dev, T * H * D)
    return T, H, Hk, S, mb, nb, bs, dev, qs, scale, out, ptrs, out_ptr


def _paged_prefill(name, q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, scale, out,
                   workspace, *mask):
    T, H, Hk, S, mb, nb, bs, dev, qs, scale, out, ptrs, out_ptr = _chunk_args(
        q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, scale, out)
    if T == 0 or S == 0:
        return out
    lib = _lib or load()
    if workspace is not None:
        nbytes = _workspace(workspace, dev)
    else:
        nbytes = getattr(lib, name + "_workspace_bytes")(S, T, H, Hk, mb, *mask)
        if nbytes:
            workspace = _torch().empty(nbytes, dtype=_torch().uint8, device=q.device)
    _check(name, getattr(lib, name)(
        *ptrs, out_ptr, S, T, H, Hk, q.shape[2], bs, nb, mb, qs, scale, *mask, _ptr(workspace),
        nbytes, _raw_stream(dev)))
    return out
