"""Thin ctypes binding of libfa.so.

The functions ``fa_fwd``, ``fa_varlen_fwd``, ``fa_fwd_strided``, ``fa_varlen_fwd_strided``, ``fa_fwd_qk_rmsnorm``,
``fa_fwd_window``, ``fa_bwd_window``, ``fa_varlen_fwd_window``, ``fa_varlen_bwd_window``, ``fa_fwd_window_anchor``,
``fa_bwd_window_anchor``, ``fa_varlen_fwd_window_anchor``, ``fa_varlen_bwd_window_anchor``, ``fa_bwd_strided``,
``fa_varlen_bwd_strided``,
``fa_pack_key_mask``,
``fa_fwd_keymask``, ``fa_bwd_keymask``, ``fa_fwd_fp8``, ``fa_decode``, ``fa_decode_paged``, ``fa_decode_workspace_size``,
``fa_decode_fp8``, ``fa_decode_paged_fp8``, ``fa_decode_fp8_workspace_size``, ``fa_build_block_tables``,
``fa_cache_append_paged``, ``fa_cache_append_fp8``, ``fa_cache_append_paged_fp8``,
``fa_bwd_workspace_size``, ``fa_varlen_bwd``,
``fa_bwd``, ``fa_status_string`` and ``fa_get_last_device_error`` have the
names, argument order and meaning of the C ABI in ``include/fa.h``: pointers
are passed as integers (device addresses), streams as integers (0 = default
stream), and the return value is the ``fa_status`` code. They only marshal
arguments; every step of the computation runs in the library's kernels.

``attention_fwd``, ``attention_varlen_fwd`` and ``attention_bwd`` are the
same calls on torch CUDA tensors: torch allocates the outputs and workspace,
the library fills them. With ``stream`` they run, allocate and convert on that
stream, whichever is current: inputs and given outputs must be ready for it, and the
caller orders other streams' use of the results. There is no fallback: if ``libfa.so``
is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_MISALIGNED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_BF16, FA_FP16 = 0, 1

_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float

_SIGS = {
    "fa_fwd": ([_P, _P, _P, _P, _P] + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_varlen_fwd": ([_P, _P, _P, _P, _P, _P, _P] + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_bwd_workspace_size": ([_I] * 4, ctypes.c_size_t),
    "fa_bwd": ([_P] * 10 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_status_string": ([_I], ctypes.c_char_p),
    "fa_get_last_device_error": ([_P], _I),
    "fa_get_last_device_error_site": ([], _I),
    "fa_version": ([], ctypes.c_char_p),
    "fa_bwd_set_timing_events": ([_P, _P], None),
    "fa_bwd_noalloc": ([_P] * 9 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_varlen_bwd_workspace_size": ([_I] * 5, ctypes.c_size_t),
    "fa_fwd_strided": ([_P] * 9 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_fwd_window": ([_P] * 5 + [_I] * 6 + [_F, _I, _I, _I, _P], _I),
    "fa_bwd_window": ([_P] * 10 + [_I] * 6 + [_F, _I, _I, _I, _P], _I),
    "fa_fwd_qk_rmsnorm": ([_P] * 6 + [_I] * 6 + [_F, _I, _F, _I, _P], _I),
    "fa_fwd_qk_rmsnorm_workspace_size": ([_I] * 4, ctypes.c_size_t),
    "fa_varlen_fwd_strided": ([_P] * 11 + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_varlen_bwd": ([_P] * 12 + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_selftest_bounded_wait": ([_P], _I),
    "fa_decode_workspace_size": ([_I] * 5, ctypes.c_size_t),
    "fa_fwd_fp8": ([_P] * 8 + [_I] * 6 + [_F, _I, _P], _I),
    "fa_pack_key_mask": ([_P, _P, _I, _I, _P], _I),
    "fa_fwd_keymask": ([_P] * 6 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_bwd_keymask": ([_P] * 11 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_bwd_strided": ([_P] * 18 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_varlen_bwd_strided": ([_P] * 20 + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_fwd_window_anchor": ([_P] * 5 + [_I] * 6 + [_F, _I, _I, _I, _I, _P], _I),
    "fa_bwd_window_anchor": ([_P] * 10 + [_I] * 6 + [_F, _I, _I, _I, _I, _P], _I),
    "fa_varlen_fwd_window": ([_P] * 7 + [_I] * 8 + [_F, _I, _I, _I, _P], _I),
    "fa_varlen_bwd_window": ([_P] * 12 + [_I] * 8 + [_F, _I, _I, _I, _P], _I),
    "fa_varlen_fwd_window_anchor": ([_P] * 7 + [_I] * 8 + [_F, _I, _I, _I, _I, _P], _I),
    "fa_varlen_bwd_window_anchor": ([_P] * 12 + [_I] * 8 + [_F, _I, _I, _I, _I, _P], _I),
    "fa_decode": ([_P] * 7 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_decode_paged": ([_P] * 8 + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_decode_fp8_workspace_size": ([_I] * 5, ctypes.c_size_t),
    "fa_decode_fp8": ([_P] * 9 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "fa_decode_paged_fp8": ([_P] * 10 + [_I] * 8 + [_F, _I, _I, _P], _I),
    "fa_build_block_tables": ([_P] * 8 + [_I] * 6 + [_P], _I),
    "fa_cache_append_paged": ([_P] * 7 + [_I] * 6 + [_P], _I),
    "fa_cache_append_fp8": ([_P] * 11 + [_I] * 7 + [_P], _I),
    "fa_cache_append_paged_fp8": ([_P] * 12 + [_I] * 9 + [_P], _I),
}


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fa_status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m exact_tiled_attention_36_b200.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _lib = l
    return _lib


def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    return lib().fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream)


def fa_varlen_fwd(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                  max_seqlen_k, Hq, Hkv, d, scale, causal, dtype, stream) -> int:
    return lib().fa_varlen_fwd(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                               max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype, stream)


def fa_bwd_workspace_size(B, Hq, Nq, d) -> int:
    return int(lib().fa_bwd_workspace_size(B, Hq, Nq, d))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype,
           stream) -> int:
    return lib().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal,
                        dtype, stream)


def fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right, dtype, stream) -> int:
    return lib().fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right, dtype,
                               stream)


def fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale, window_left,
                  window_right, dtype, stream) -> int:
    return lib().fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale,
                               window_left, window_right, dtype, stream)


def fa_fwd_qk_rmsnorm_workspace_size(B, Nk, Hkv, d) -> int:
    return int(lib().fa_fwd_qk_rmsnorm_workspace_size(B, Nk, Hkv, d))


def fa_fwd_qk_rmsnorm(q, k, v, o, lse, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal, eps, dtype,
                      stream) -> int:
    return lib().fa_fwd_qk_rmsnorm(q, k, v, o, lse, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal, eps, dtype,
                                   stream)


def _strides(st):
    """A host int64 array of element strides (kept alive by the caller's reference)."""
    return (ctypes.c_longlong * len(st))(*[int(x) for x in st]) if st is not None else None


def fa_fwd_strided(q, k, v, o, lse, q_strides, k_strides, v_strides, o_strides, B, Hq, Hkv, Nq, Nk, d, scale,
                   causal, dtype, stream) -> int:
    """Strides are sequences of ints ({batch, token, head} in elements)."""
    arrs = [_strides(x) for x in (q_strides, k_strides, v_strides, o_strides)]
    return lib().fa_fwd_strided(q, k, v, o, lse, *[ctypes.cast(a, _P) if a is not None else None for a in arrs], B,
                                Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream)


def fa_varlen_fwd_strided(q, k, v, o, lse, q_strides, k_strides, v_strides, o_strides, cu_seqlens_q, cu_seqlens_k,
                          num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype,
                          stream) -> int:
    """Strides are sequences of ints ({token, head} in elements)."""
    arrs = [_strides(x) for x in (q_strides, k_strides, v_strides, o_strides)]
    return lib().fa_varlen_fwd_strided(q, k, v, o, lse, *[ctypes.cast(a, _P) if a is not None else None for a in arrs],
                                       cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                                       max_seqlen_k, Hq, Hkv, d, scale, causal, dtype, stream)


def fa_varlen_bwd_workspace_size(num_seqs, total_q, max_seqlen_q, Hq, d) -> int:
    return int(lib().fa_varlen_bwd_workspace_size(num_seqs, total_q, max_seqlen_q, Hq, d))


def fa_varlen_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q,
                  total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype, stream) -> int:
    return lib().fa_varlen_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, num_seqs,
                               total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype,
                               stream)


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    """fa_bwd with the library's own fixed-size workspace (for callers that cannot allocate)."""
    return lib().fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype,
                                stream)


def fa_pack_key_mask(keep, key_bits, B, Nk, stream) -> int:
    return lib().fa_pack_key_mask(keep, key_bits, B, Nk, stream)


def fa_fwd_keymask(q, k, v, o, lse, key_bits, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    return lib().fa_fwd_keymask(q, k, v, o, lse, key_bits, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream)


def fa_bwd_keymask(q, k, v, o, lse, dout, dq, dk, dv, workspace, key_bits, B, Hq, Hkv, Nq, Nk, d, scale, causal,
                   dtype, stream) -> int:
    return lib().fa_bwd_keymask(q, k, v, o, lse, dout, dq, dk, dv, workspace, key_bits, B, Hq, Hkv, Nq, Nk, d, scale,
                                causal, dtype, stream)


def fa_bwd_strided(q, k, v, o, lse, dout, dq, dk, dv, workspace, q_strides, k_strides, v_strides, o_strides,
                   do_strides, dq_strides, dk_strides, dv_strides, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype,
                   stream) -> int:
    """*_strides: (batch, token, head) element strides (host), as fa_fwd_strided."""
    return lib().fa_bwd_strided(q, k, v, o, lse, dout, dq, dk, dv, workspace, _strides(q_strides),
                                _strides(k_strides), _strides(v_strides), _strides(o_strides), _strides(do_strides),
                                _strides(dq_strides), _strides(dk_strides), _strides(dv_strides), B, Hq, Hkv, Nq, Nk,
                                d, scale, causal, dtype, stream)


def fa_varlen_bwd_strided(q, k, v, o, lse, dout, dq, dk, dv, workspace, q_strides, k_strides, v_strides, o_strides,
                          do_strides, dq_strides, dk_strides, dv_strides, cu_seqlens_q, cu_seqlens_k, num_seqs,
                          total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype,
                          stream) -> int:
    """*_strides: (token, head) element strides (host), as fa_varlen_fwd_strided."""
    return lib().fa_varlen_bwd_strided(q, k, v, o, lse, dout, dq, dk, dv, workspace, _strides(q_strides),
                                       _strides(k_strides), _strides(v_strides), _strides(o_strides),
                                       _strides(do_strides), _strides(dq_strides), _strides(dk_strides),
                                       _strides(dv_strides), cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                       max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, causal, dtype, stream)


def fa_fwd_window_anchor(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right, n_anchor, dtype,
                         stream) -> int:
    return lib().fa_fwd_window_anchor(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right,
                                      n_anchor, dtype, stream)


def fa_bwd_window_anchor(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale, window_left,
                         window_right, n_anchor, dtype, stream) -> int:
    return lib().fa_bwd_window_anchor(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Nq, Nk, d, scale,
                                      window_left, window_right, n_anchor, dtype, stream)


def fa_varlen_fwd_window(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                         max_seqlen_k, Hq, Hkv, d, scale, window_left, window_right, dtype, stream) -> int:
    return lib().fa_varlen_fwd_window(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                      max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, window_left, window_right, dtype,
                                      stream)


def fa_varlen_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, num_seqs,
                         total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, window_left, window_right,
                         dtype, stream) -> int:
    return lib().fa_varlen_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k,
                                      num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale,
                                      window_left, window_right, dtype, stream)


def fa_varlen_fwd_window_anchor(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q,
                                max_seqlen_k, Hq, Hkv, d, scale, window_left, window_right, n_anchor, dtype,
                                stream) -> int:
    return lib().fa_varlen_fwd_window_anchor(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                             max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, window_left, window_right,
                                             n_anchor, dtype, stream)


def fa_varlen_bwd_window_anchor(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, num_seqs,
                                total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, d, scale, window_left,
                                window_right, n_anchor, dtype, stream) -> int:
    return lib().fa_varlen_bwd_window_anchor(q, k, v, o, lse, dout, dq, dk, dv, workspace, cu_seqlens_q,
                                             cu_seqlens_k, num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq,
                                             Hkv, d, scale, window_left, window_right, n_anchor, dtype, stream)


def fa_fwd_fp8(q, k, v, q_scale, k_scale, v_scale, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream) -> int:
    return lib().fa_fwd_fp8(q, k, v, q_scale, k_scale, v_scale, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream)


def fa_decode_workspace_size(B, Hq, Hkv, Nq, d) -> int:
    return int(lib().fa_decode_workspace_size(B, Hq, Hkv, Nq, d))


def fa_decode(q, k, v, o, lse, cache_seqlens, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    return lib().fa_decode(q, k, v, o, lse, cache_seqlens, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal, dtype,
                           stream)


def fa_decode_paged(q, k_pages, v_pages, o, lse, cache_seqlens, block_table, workspace, B, Hq, Hkv, Nq, num_pages,
                    page_size, max_pages, d, scale, causal, dtype, stream) -> int:
    return lib().fa_decode_paged(q, k_pages, v_pages, o, lse, cache_seqlens, block_table, workspace, B, Hq, Hkv, Nq,
                                 num_pages, page_size, max_pages, d, scale, causal, dtype, stream)


def fa_decode_fp8_workspace_size(B, Hq, Hkv, Nq, d) -> int:
    return int(lib().fa_decode_fp8_workspace_size(B, Hq, Hkv, Nq, d))


def fa_decode_fp8(q, k, v, k_scale, v_scale, o, lse, cache_seqlens, workspace, B, Hq, Hkv, Nq, Nk, d, scale, causal,
                  dtype, stream) -> int:
    return lib().fa_decode_fp8(q, k, v, k_scale, v_scale, o, lse, cache_seqlens, workspace, B, Hq, Hkv, Nq, Nk, d,
                               scale, causal, dtype, stream)


def fa_decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, o, lse, cache_seqlens, block_table, workspace, B, Hq,
                        Hkv, Nq, num_pages, page_size, max_pages, d, scale, causal, dtype, stream) -> int:
    return lib().fa_decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, o, lse, cache_seqlens, block_table,
                                     workspace, B, Hq, Hkv, Nq, num_pages, page_size, max_pages, d, scale, causal,
                                     dtype, stream)


def fa_build_block_tables(cache_seqlens, new_lens, free_pages, block_table, slot_map, cu_new, new_seqlens, pages_used,
                          B, num_free, num_pages, page_size, max_pages, total_new, stream) -> int:
    return lib().fa_build_block_tables(cache_seqlens, new_lens, free_pages, block_table, slot_map, cu_new,
                                       new_seqlens, pages_used, B, num_free, num_pages, page_size, max_pages,
                                       total_new, stream)


def fa_cache_append_paged(k, v, k_strides, v_strides, k_pages, v_pages, slot_map, total_new, Hkv, num_pages, page_size,
                          d, dtype, stream) -> int:
    """*_strides: (token, head) element strides (host), or None for contiguous rows."""
    return lib().fa_cache_append_paged(k, v, _strides(k_strides), _strides(v_strides), k_pages, v_pages, slot_map,
                                       total_new, Hkv, num_pages, page_size, d, dtype, stream)


def fa_cache_append_fp8(k, v, k_strides, v_strides, k_cache, v_cache, k_scale, v_scale, cu_new, cache_seqlens,
                        new_seqlens, B, total_new, max_new, Hkv, Nk, d, dtype, stream) -> int:
    """*_strides: (token, head) element strides (host), or None for contiguous rows."""
    return lib().fa_cache_append_fp8(k, v, _strides(k_strides), _strides(v_strides), k_cache, v_cache, k_scale,
                                     v_scale, cu_new, cache_seqlens, new_seqlens, B, total_new, max_new, Hkv, Nk, d,
                                     dtype, stream)


def fa_cache_append_paged_fp8(k, v, k_strides, v_strides, k_pages, v_pages, k_scale, v_scale, cu_new, cache_seqlens,
                              new_seqlens, block_table, B, total_new, max_new, Hkv, num_pages, page_size, max_pages, d,
                              dtype, stream) -> int:
    """*_strides: (token, head) element strides (host), or None for contiguous rows."""
    return lib().fa_cache_append_paged_fp8(k, v, _strides(k_strides), _strides(v_strides), k_pages, v_pages, k_scale,
                                           v_scale, cu_new, cache_seqlens, new_seqlens, block_table, B, total_new,
                                           max_new, Hkv, num_pages, page_size, max_pages, d, dtype, stream)


def fa_status_string(s: int) -> str:
    return lib().fa_status_string(s).decode()


def fa_get_last_device_error(stream) -> int:
    return lib().fa_get_last_device_error(stream)


def fa_get_last_device_error_site() -> int:
    return lib().fa_get_last_device_error_site()


def fa_bwd_set_timing_events(before, after) -> None:
    lib().fa_bwd_set_timing_events(before, after)


def fa_selftest_bounded_wait(stream) -> int:
    return lib().fa_selftest_bounded_wait(stream)


def fa_version() -> str:
    return lib().fa_version().decode()


# ----------------------------------------------------------------------------- torch tensors
def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"q/k/v must be bfloat16 or float16, got {t.dtype}")


def _dev(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return t if t.is_contiguous() else t.contiguous()


def _stream(stream):
    """The raw CUDA stream handle: `stream` (a torch stream or a handle), or the current
    stream of the current device."""
    import torch
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(stream, device, fn, *args, **given):
    """fn(*args, **given) with `stream` (a torch stream or a handle) current, so that what it allocates and
    converts comes from that stream's memory and in its order: a block of another stream's memory may still
    be in use by that one's earlier work. A result that fn made may be used on the stream that was current,
    too: once dropped, its memory is kept until what that stream was given so far has run."""
    import torch
    if device.type != "cuda":
        return fn(*args, **given)  # refused there
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is one of {stream.device}, the tensors are on {device}")
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        results = fn(*args, **given)
    if here.cuda_stream != stream.cuda_stream:
        for t in results:
            if not any(t is x for x in given.values()):
                t.record_stream(here)
    return results


def _check(status: int, what: str):
    if status != FA_OK:
        raise FAError(status, what)


def attention_fwd(q, k, v, scale: float | None = None, causal: bool = False, out=None, lse=None, stream=None):
    """O, L = attention(q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d]); L is float32 [B,Hq,Nq]."""
    import torch
    if stream is not None:
        return _on_stream(stream, q.device, attention_fwd, q, k, v, scale, causal, out=out, lse=lse)
    q, k, v = _dev(q), _dev(k), _dev(v)
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q) if out is None else out
    L = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(), B, Hq, Hkv, Nq, Nk, d,
                  float(scale), int(bool(causal)), _dtype_code(q), _stream(None)), "fa_fwd")
    return o, L


def attention_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                         scale: float | None = None, causal: bool = False, out=None, lse=None, stream=None):
    """Packed varlen forward: q [total_q,Hq,d], k/v [total_k,Hkv,d]; L is float32 [Hq,total_q]."""
    import torch
    if stream is not None:
        return _on_stream(stream, q.device, attention_varlen_fwd, q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                          max_seqlen_k, scale, causal, out=out, lse=lse)
    q, k, v = _dev(q), _dev(k), _dev(v)
    cu_q = _dev(cu_seqlens_q).to(torch.int32)
    cu_k = _dev(cu_seqlens_k).to(torch.int32)
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q) if out is None else out
    L = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(fa_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(), cu_q.data_ptr(),
                         cu_k.data_ptr(), cu_q.numel() - 1, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv,
                         d, float(scale), int(bool(causal)), _dtype_code(q), _stream(None)), "fa_varlen_fwd")
    return o, L


def attention_bwd(q, k, v, o, lse, dout, scale: float | None = None, causal: bool = False, workspace=None,
                  stream=None):
    """dQ, dK, dV of the fixed-length forward (same layouts as q, k, v)."""
    import torch
    if stream is not None:
        return _on_stream(stream, q.device, attention_bwd, q, k, v, o, lse, dout, scale, causal, workspace=workspace)
    q, k, v, o, dout = _dev(q), _dev(k), _dev(v), _dev(o), _dev(dout)
    lse = _dev(lse)
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    if scale is None:
        scale = d ** -0.5
    ws_bytes = fa_bwd_workspace_size(B, Hq, Nq, d)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device) if workspace is None else workspace
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    _check(fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                  dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), B, Hq, Hkv, Nq, Nk, d, float(scale),
                  int(bool(causal)), _dtype_code(q), _stream(None)), "fa_bwd")
    return dq, dk, dv


def attention_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                         scale: float | None = None, causal: bool = False, workspace=None, stream=None):
    """dQ, dK, dV of the packed varlen forward (same layouts as q, k, v; d = 64 or 128)."""
    import torch
    if stream is not None:
        return _on_stream(stream, q.device, attention_varlen_bwd, q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k,
                          max_seqlen_q, max_seqlen_k, scale, causal, workspace=workspace)
    q, k, v, o, dout = _dev(q), _dev(k), _dev(v), _dev(o), _dev(dout)
    lse = _dev(lse)
    cu_q = _dev(cu_seqlens_q).to(torch.int32)
    cu_k = _dev(cu_seqlens_k).to(torch.int32)
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    n = cu_q.numel() - 1
    if scale is None:
        scale = d ** -0.5
    ws_bytes = fa_varlen_bwd_workspace_size(n, Tq, int(max_seqlen_q), Hq, d)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device) if workspace is None else workspace
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    _check(fa_varlen_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
                         n, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, d, float(scale),
                         int(bool(causal)), _dtype_code(q), _stream(None)), "fa_varlen_bwd")
    return dq, dk, dv


def attention_decode(q, k_cache, v_cache, cache_seqlens=None, scale: float | None = None, causal: bool = False,
                     block_table=None, workspace=None, out=None, lse=None, stream=None):
    """Split-KV decode: q [B,Nq,Hq,d] (the newest Nq tokens) against a cache.

    Contiguous cache: k/v [B,Nk,Hkv,d], sequence b using its first cache_seqlens[b]
    keys (all Nk when None). Paged cache (block_table int32 [B,max_pages]): k/v
    [num_pages,page_size,Hkv,d] and cache_seqlens required. Returns O [B,Nq,Hq,d]
    and L float32 [B,Hq,Nq]."""
    import torch
    if stream is not None:
        return _on_stream(stream, q.device, attention_decode, q, k_cache, v_cache, cache_seqlens, scale, causal,
                          block_table, workspace=workspace, out=out, lse=lse)
    q, k, v = _dev(q), _dev(k_cache), _dev(v_cache)
    B, Nq, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = d ** -0.5
    sl = None if cache_seqlens is None else _dev(cache_seqlens).to(torch.int32)
    ws_bytes = fa_decode_workspace_size(B, Hq, Hkv, Nq, d)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device) if workspace is None else workspace
    o = torch.empty_like(q) if out is None else out
    L = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    if block_table is None:
        st = fa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(),
                       0 if sl is None else sl.data_ptr(), ws.data_ptr(), B, Hq, Hkv, Nq, k.shape[1], d, float(scale),
                       int(bool(causal)), _dtype_code(q), _stream(None))
        _check(st, "fa_decode")
    else:
        if sl is None:
            raise ValueError("a paged cache needs cache_seqlens")
        bt = _dev(block_table).to(torch.int32)
        st = fa_decode_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(), sl.data_ptr(),
                             bt.data_ptr(), ws.data_ptr(), B, Hq, Hkv, Nq, k.shape[0], k.shape[1], bt.shape[1], d,
                             float(scale), int(bool(causal)), _dtype_code(q), _stream(None))
        _check(st, "fa_decode_paged")
    return o, L


def attention_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, scale: float | None = None, causal: bool = False,
                      out=None, lse=None, stream=None):
    """FP8 forward: q8 [B,Nq,Hq,d], k8/v8 [B,Nk,Hkv,d] uint8 E4M3 codes with float32 block
    factors [B,H,ceil(N/128)]; returns O bf16 [B,Nq,Hq,d] and L float32 [B,Hq,Nq]."""
    import torch
    if stream is not None:
        return _on_stream(stream, q8.device, attention_fwd_fp8, q8, k8, v8, q_scale, k_scale, v_scale, scale, causal,
                          out=out, lse=lse)
    q8, k8, v8 = _dev(q8), _dev(k8), _dev(v8)
    qs, ks, vs = (_dev(t).to(torch.float32) for t in (q_scale, k_scale, v_scale))
    B, Nq, Hq, d = q8.shape
    _, Nk, Hkv, _ = k8.shape
    if scale is None:
        scale = d ** -0.5
    o = torch.empty((B, Nq, Hq, d), dtype=torch.bfloat16, device=q8.device) if out is None else out
    L = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q8.device) if lse is None else lse
    _check(fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), qs.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                      o.data_ptr(), L.data_ptr(), B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)),
                      _stream(None)), "fa_fwd_fp8")
    return o, L


# Serving. These write caches and tables in place, so nothing is copied or converted on the way:
# every tensor must already have the type and the (contiguous) layout the entry point takes, and all
# must lie on one device, which need not be the current one. `stream`: as above, a stream of that device.
# A decode step makes these calls once per layer, next to kernels of a few microseconds, so the
# checks of a call are one expression and only a failing one looks for its message.
_T = None  # torch, imported with the first call


def _torch():
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _fits(t, dtype, index, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _own(t, name: str, dtypes, index, shape):
    """`t` as it is, or an error: its type, device, shape and layout."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(x) for x in dtypes)}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be on the CUDA device of the other tensors")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _need(t, name, dtype, index, shape):
    return t if _fits(t, dtype, index, shape) else _own(t, name, (dtype,), index, shape)


def _call(index: int, stream, what: str, fn, *args):
    """fn(*args, stream handle) with device `index` current; its status as an exception."""
    T = _torch()
    if index == T._C._cuda_getDevice():
        st = fn(*args, T._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    else:
        with T.cuda.device(index):
            st = fn(*args, _stream(stream))
    if st != FA_OK:
        raise FAError(st, what)


_Pair = ctypes.c_longlong * 2


def _rows(t, name: str, index):
    """(token, head) strides of new rows [T, Hkv, d]: any 16-byte multiples."""
    if t.dim() != 3 or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be [tokens, Hkv, d] on the CUDA device of the other tensors")
    st, sh, one = t.stride()
    n, H, d = t.shape
    if one != 1 and d > 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    # A dimension of one element may carry any stride; it is never stepped over.
    return (st if n > 1 else H * d, sh if H > 1 else d)


def _new_rows(k_new, v_new, index):
    """Host arrays of the new rows' strides (kept alive by the caller's reference), and FA_BF16 or FA_FP16."""
    T = _torch()
    dt = k_new.dtype
    if v_new.shape != k_new.shape or v_new.dtype is not dt:
        raise ValueError("k_new and v_new must have one shape and type")
    if dt is not T.bfloat16 and dt is not T.float16:
        raise TypeError(f"k_new and v_new must be bfloat16 or float16, got {dt}")
    return _Pair(*_rows(k_new, "k_new", index)), _Pair(*_rows(v_new, "v_new", index)), \
        FA_BF16 if dt is T.bfloat16 else FA_FP16


_ws_bytes = {}  # (device, sizes) -> bytes; what the library computes from the sizes and the SM count


def _decode_fp8_bytes(index, B, Hq, Hkv, Nq, d) -> int:
    key = (index, B, Hq, Hkv, Nq, d)
    n = _ws_bytes.get(key)
    if n is None:
        with _torch().cuda.device(index):
            n = max(fa_decode_fp8_workspace_size(B, Hq, Hkv, Nq, d), 16)
        if len(_ws_bytes) >= 4096:
            _ws_bytes.clear()
        _ws_bytes[key] = n
    return n


def attention_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, cache_seqlens=None, scale: float | None = None,
                         causal: bool = False, block_table=None, workspace=None, out=None, lse=None, stream=None):
    """Split-KV decode over an E4M3 cache: q [B,Nq,Hq,d] (bf16 or fp16) against codes (uint8 or float8_e4m3fn).

    Contiguous cache: k/v [B,Nk,Hkv,d], k/v_scale float32 [B,Hkv,ceil(Nk/128)], sequence b using its
    first cache_seqlens[b] keys (int32; all Nk when None). Paged cache (block_table int32
    [B,max_pages]): k/v [num_pages,page_size,Hkv,d], k/v_scale [num_pages,Hkv], cache_seqlens
    required. `workspace`: uint8, fa_decode_fp8_workspace_size(B,Hq,Hkv,Nq,d) bytes (one is made
    when None). Returns O [B,Nq,Hq,d] (q's type) and L float32 [B,Hq,Nq]."""
    if stream is not None:
        return _on_stream(stream, q.device, attention_decode_fp8, q, k_cache, v_cache, k_scale, v_scale, cache_seqlens,
                          scale, causal, block_table, workspace=workspace, out=out, lse=lse)
    T = _torch()
    f32, i32, dt = T.float32, T.int32, q.dtype
    index = q.get_device()
    B, Nq, Hq, d = shape = q.shape
    n0, n1, Hkv, _ = kshape = k_cache.shape
    paged = block_table is not None
    factors = (n0, Hkv) if paged else (B, Hkv, (n1 + 127) // 128)
    need = _decode_fp8_bytes(index, B, Hq, Hkv, Nq, d) if index >= 0 else 0
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = T.empty_like(q)
    if lse is None:
        lse = T.empty((B, Hq, Nq), dtype=f32, device=q.device)
    if workspace is None:
        workspace = T.empty(need, dtype=T.uint8, device=q.device)
    if not ((dt is T.bfloat16 or dt is T.float16) and index >= 0 and q.is_contiguous()
            and kshape == (n0 if paged else B, n1, Hkv, d) and v_cache.shape == kshape
            and (k_cache.dtype is T.uint8 or k_cache.dtype is T.float8_e4m3fn) and k_cache.is_contiguous()
            and (v_cache.dtype is T.uint8 or v_cache.dtype is T.float8_e4m3fn) and v_cache.is_contiguous()
            and k_cache.get_device() == index and v_cache.get_device() == index
            and k_scale.dtype is f32 and k_scale.shape == factors and k_scale.is_contiguous()
            and v_scale.dtype is f32 and v_scale.shape == factors and v_scale.is_contiguous()
            and k_scale.get_device() == index and v_scale.get_device() == index
            and out.dtype is dt and out.shape == shape and out.is_contiguous() and out.get_device() == index
            and lse.dtype is f32 and lse.shape == (B, Hq, Nq) and lse.is_contiguous() and lse.get_device() == index
            and workspace.dtype is T.uint8 and workspace.numel() >= need and workspace.is_contiguous()
            and workspace.get_device() == index
            and (not paged or cache_seqlens is not None and _fits(block_table, i32, index, (B, block_table.shape[-1])))
            and (cache_seqlens is None or _fits(cache_seqlens, i32, index, (B,)))):
        _own(q, "q", (T.bfloat16, T.float16), index, shape)
        codes = (T.uint8, T.float8_e4m3fn)
        _own(k_cache, "k_cache", codes, index, (n0 if paged else B, n1, Hkv, d))
        _own(v_cache, "v_cache", codes, index, kshape)
        _own(k_scale, "k_scale", (f32,), index, factors)
        _own(v_scale, "v_scale", (f32,), index, factors)
        _own(out, "out", (dt,), index, shape)
        _own(lse, "lse", (f32,), index, (B, Hq, Nq))
        _own(workspace, "workspace", (T.uint8,), index, workspace.shape)
        if workspace.numel() < need:
            raise ValueError(f"workspace must hold {need} bytes, got {workspace.numel()}")
        if cache_seqlens is not None:
            _own(cache_seqlens, "cache_seqlens", (i32,), index, (B,))
        if paged and cache_seqlens is None:
            raise ValueError("a paged cache needs cache_seqlens")
        _own(block_table, "block_table", (i32,), index, (B, block_table.shape[-1]))
    sl = None if cache_seqlens is None else cache_seqlens.data_ptr()
    code = FA_BF16 if dt is T.bfloat16 else FA_FP16
    if paged:
        _call(index, None, "fa_decode_paged_fp8", lib().fa_decode_paged_fp8, q.data_ptr(), k_cache.data_ptr(),
              v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), out.data_ptr(), lse.data_ptr(), sl,
              block_table.data_ptr(), workspace.data_ptr(), B, Hq, Hkv, Nq, n0, n1, block_table.shape[1], d, scale,
              bool(causal), code)
    else:
        _call(index, None, "fa_decode_fp8", lib().fa_decode_fp8, q.data_ptr(), k_cache.data_ptr(),
              v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), out.data_ptr(), lse.data_ptr(), sl,
              workspace.data_ptr(), B, Hq, Hkv, Nq, n1, d, scale, bool(causal), code)
    return out, lse


def build_block_tables(cache_seqlens, new_lens, free_pages, block_table, page_size: int, num_pages: int,
                       total_new: int, slot_map=None, cu_new=None, new_seqlens=None, pages_used=None, stream=None):
    """Pages of `free_pages` for every request's new tokens, written into block_table int32 [B,max_pages].

    cache_seqlens int32 [B] (None: every request is new), new_lens int32 [B], free_pages int32
    [num_free]. Returns slot_map int32 [total_new] (page * page_size + row of every packed new
    token, -1 for none), cu_new int32 [B+1], new_seqlens int32 [B] and pages_used int32 [1], the
    number of entries of free_pages taken."""
    if stream is not None:
        return _on_stream(stream, new_lens.device, build_block_tables, cache_seqlens, new_lens, free_pages, block_table,
                          page_size, num_pages, total_new, slot_map=slot_map, cu_new=cu_new, new_seqlens=new_seqlens,
                          pages_used=pages_used)
    T = _torch()
    i32, index = T.int32, new_lens.get_device()
    B, pages, num_free = new_lens.shape[0], block_table.shape[-1], free_pages.numel()
    if index < 0 or not _fits(new_lens, i32, index, (B,)):
        _own(new_lens, "new_lens", (i32,), index, (B,))
    if cache_seqlens is not None:
        _need(cache_seqlens, "cache_seqlens", i32, index, (B,))
    _need(free_pages, "free_pages", i32, index, (num_free,))
    _need(block_table, "block_table", i32, index, (B, pages))
    dev = new_lens.device
    slot_map = T.empty(total_new, dtype=i32, device=dev) if slot_map is None else \
        _need(slot_map, "slot_map", i32, index, (total_new,))
    cu_new = T.empty(B + 1, dtype=i32, device=dev) if cu_new is None else _need(cu_new, "cu_new", i32, index, (B + 1,))
    new_seqlens = T.empty(B, dtype=i32, device=dev) if new_seqlens is None else \
        _need(new_seqlens, "new_seqlens", i32, index, (B,))
    pages_used = T.empty(1, dtype=i32, device=dev) if pages_used is None else \
        _need(pages_used, "pages_used", i32, index, (1,))
    _call(index, None, "fa_build_block_tables", lib().fa_build_block_tables,
          None if cache_seqlens is None else cache_seqlens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
          block_table.data_ptr(), slot_map.data_ptr(), cu_new.data_ptr(), new_seqlens.data_ptr(),
          pages_used.data_ptr(), B, num_free, num_pages, page_size, pages, total_new)
    return slot_map, cu_new, new_seqlens, pages_used


def cache_append_paged(k_new, v_new, k_pages, v_pages, slot_map, stream=None):
    """Rows [T,Hkv,d] of k_new and v_new (any 16-byte strides) into the 16-bit page pools
    [num_pages,page_size,Hkv,d] at slot_map int32 [T]; slots outside the pool are skipped."""
    index = k_pages.get_device()
    ks, vs, code = _new_rows(k_new, v_new, index)
    n_new, Hkv, d = k_new.shape
    n, page = k_pages.shape[:2]
    _need(k_pages, "k_pages", k_new.dtype, index, (n, page, Hkv, d))
    _need(v_pages, "v_pages", k_new.dtype, index, (n, page, Hkv, d))
    _need(slot_map, "slot_map", _torch().int32, index, (n_new,))
    _call(index, stream, "fa_cache_append_paged", lib().fa_cache_append_paged, k_new.data_ptr(), v_new.data_ptr(), ks,
          vs, k_pages.data_ptr(), v_pages.data_ptr(), slot_map.data_ptr(), n_new, Hkv, n, page, d, code)


def cache_append_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, cu_new, cache_seqlens, new_seqlens,
                     max_new: int, block_table=None, stream=None):
    """Rows [T,Hkv,d] of k_new and v_new (bf16 or fp16, any 16-byte strides) quantised into an E4M3 cache.

    Sequence b's rows cu_new[b].. become its positions cache_seqlens[b] .. new_seqlens[b]-1 (int32
    tensors, as build_block_tables gives them), at most max_new of them. Caches and factors:
    the layouts of attention_decode_fp8 (paged with block_table), written in place."""
    T = _torch()
    f32, i32 = T.float32, T.int32
    index = k_cache.get_device()
    ks, vs, code = _new_rows(k_new, v_new, index)
    n_new, Hkv, d = k_new.shape
    B = cache_seqlens.shape[0]
    n0, n1 = k_cache.shape[:2]
    paged = block_table is not None
    kshape = (n0 if paged else B, n1, Hkv, d)
    factors = (n0, Hkv) if paged else (B, Hkv, (n1 + 127) // 128)
    if not (k_cache.shape == kshape and v_cache.shape == kshape and k_cache.is_contiguous() and v_cache.is_contiguous()
            and (k_cache.dtype is T.uint8 or k_cache.dtype is T.float8_e4m3fn)
            and (v_cache.dtype is T.uint8 or v_cache.dtype is T.float8_e4m3fn) and v_cache.get_device() == index
            and k_scale.dtype is f32 and k_scale.shape == factors and k_scale.is_contiguous()
            and v_scale.dtype is f32 and v_scale.shape == factors and v_scale.is_contiguous()
            and k_scale.get_device() == index and v_scale.get_device() == index
            and _fits(cu_new, i32, index, (B + 1,)) and _fits(cache_seqlens, i32, index, (B,))
            and _fits(new_seqlens, i32, index, (B,))
            and (not paged or _fits(block_table, i32, index, (B, block_table.shape[-1])))):
        codes = (T.uint8, T.float8_e4m3fn)
        _own(k_cache, "k_cache", codes, index, kshape)
        _own(v_cache, "v_cache", codes, index, kshape)
        _own(k_scale, "k_scale", (f32,), index, factors)
        _own(v_scale, "v_scale", (f32,), index, factors)
        _own(cu_new, "cu_new", (i32,), index, (B + 1,))
        _own(cache_seqlens, "cache_seqlens", (i32,), index, (B,))
        _own(new_seqlens, "new_seqlens", (i32,), index, (B,))
        _own(block_table, "block_table", (i32,), index, (B, block_table.shape[-1]))
    if paged:
        _call(index, stream, "fa_cache_append_paged_fp8", lib().fa_cache_append_paged_fp8, k_new.data_ptr(),
              v_new.data_ptr(), ks, vs, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
              cu_new.data_ptr(), cache_seqlens.data_ptr(), new_seqlens.data_ptr(), block_table.data_ptr(), B, n_new,
              max_new, Hkv, n0, n1, block_table.shape[1], d, code)
    else:
        _call(index, stream, "fa_cache_append_fp8", lib().fa_cache_append_fp8, k_new.data_ptr(), v_new.data_ptr(), ks,
              vs, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), cu_new.data_ptr(),
              cache_seqlens.data_ptr(), new_seqlens.data_ptr(), B, n_new, max_new, Hkv, n1, d, code)
