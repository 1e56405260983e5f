"""Thin ctypes binding of libkda (include/kda.h): the same entry-point names, argument
marshalling only.  Every step of the computation runs in the library's CUDA kernels;
there is no CPU or PyTorch fallback, and every call fails loudly when the library is
missing or returns an error.

Tensor arguments may be ``torch.Tensor`` (CUDA, contiguous), raw device addresses
(``int``) or ``None`` for the nullable ones.  ``stream`` defaults to torch's current
stream on the current device.
"""
from __future__ import annotations

import ctypes
import os

from .build_lib import LIB_PATH

KDA_F32 = 0
KDA_BF16 = 1
STATUS_NAMES = {
    0: "KDA_OK", -1: "KDA_ERR_NULL_POINTER", -2: "KDA_ERR_BAD_SHAPE", -3: "KDA_ERR_HEAD_DIM",
    -4: "KDA_ERR_CHUNK", -5: "KDA_ERR_LOWER_BOUND", -6: "KDA_ERR_MISALIGNED",
    -7: "KDA_ERR_DTYPE", -8: "KDA_ERR_LAUNCH", -9: "KDA_ERR_DEVICE", -10: "KDA_ERR_SCALE",
    -11: "KDA_ERR_TOO_LARGE", -12: "KDA_ERR_WORKSPACE", -13: "KDA_ERR_FLAGS",
    -14: "KDA_ERR_PAGE_SIZE", -15: "KDA_ERR_ROTARY", -16: "KDA_ERR_STRIDE",
}
# Exported symbols, in declaration order of include/kda.h.
EXPORTS = ("kda_chunk_fwd", "kda_chunk_fwd_varlen", "kda_chunk_fwd_workspace_size",
           "kda_chunk_fwd_varlen_workspace_size", "kda_chunk_fwd_ws", "kda_chunk_fwd_varlen_ws",
           "kda_chunk_fwd_noalloc", "kda_chunk_bwd_workspace_size", "kda_chunk_bwd",
           "kda_chunk_bwd_varlen_workspace_size", "kda_chunk_bwd_varlen",
           "kda_chunk_fwd_train_varlen", "kda_chunk_bwd_saved_varlen",
           "kda_chunk_fwd_train", "kda_chunk_bwd_saved", "kda_recurrent_attention_fwd", "kda_attention_fwd",
           "kda_attention_fwd_ws", "kda_attention_fwd_workspace_size",
           "kda_recurrent_attention_fwd_ws", "kda_recurrent_attention_fwd_workspace_size",
           "kda_decode_step", "kda_attention_step", "kda_qk_norm_rope_fwd",
           "kda_qk_norm_rope_append", "kda_qk_norm_rope_bwd_workspace_size",
           "kda_qk_norm_rope_bwd", "kda_paged_attention_fwd_workspace_size",
           "kda_paged_attention_fwd", "kda_qk_norm_rope_append_q8", "kda_paged_cache_read_q8",
           "kda_paged_attention_q8_fwd_workspace_size", "kda_paged_attention_q8_fwd",
           "kda_paged_prefix_attention_fwd_workspace_size",
           "kda_paged_prefix_attention_fwd",
           "kda_status_string",
           "kda_version", "kda_device_error", "kda_selftest_bounded_wait")
KDA_ATTN_NO_QK_L2NORM = 1
KDA_ATTN_RECURRENT = 2
KDA_ATTN_ORDER_LITERAL = 4
KDA_ROPE_INTERLEAVED = 1


class KDAError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} "
                         f"({kda_status_string(status)})")


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_LL = ctypes.c_longlong


def lib(path: str | None = None) -> ctypes.CDLL:
    """The loaded libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libkda.so is not built ({p}); run "
                           "`python -m gated_delta_rule_55_gb300.build_lib`")
    L = ctypes.CDLL(p)
    L.kda_chunk_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P,
                                _I, _I, _I, _I, _I, _I, _I, _P]
    L.kda_chunk_fwd_varlen.argtypes = [_P, _P, _P, _P, _P, _P, _P, _F, _F, _P, _I, _I,
                                       _P, _P, _P, _I, _I, _I, _I, _I, _P]
    L.kda_chunk_fwd_workspace_size.argtypes = [_I] * 7
    L.kda_chunk_fwd_varlen_workspace_size.argtypes = [_I] * 7
    L.kda_chunk_fwd_workspace_size.restype = _Z
    L.kda_chunk_fwd_varlen_workspace_size.restype = _Z
    L.kda_chunk_fwd_ws.argtypes = L.kda_chunk_fwd.argtypes[:-1] + [_P, _Z, _P]
    L.kda_chunk_fwd_varlen_ws.argtypes = L.kda_chunk_fwd_varlen.argtypes[:-1] + [_P, _Z, _P]
    L.kda_chunk_fwd_noalloc.argtypes = L.kda_chunk_fwd.argtypes
    L.kda_recurrent_attention_fwd.argtypes = ([_P] * 7 + [_F] + [_P] * 4 + [_I] * 8 + [_P])
    L.kda_recurrent_attention_fwd_ws.argtypes = ([_P] * 7 + [_F] + [_P] * 4 + [_I] * 8 +
                                                 [_P, _Z, _P])
    L.kda_recurrent_attention_fwd_workspace_size.argtypes = [_I] * 8
    L.kda_recurrent_attention_fwd_workspace_size.restype = _Z
    L.kda_chunk_bwd_workspace_size.argtypes = [_I] * 6
    L.kda_chunk_bwd_workspace_size.restype = _Z
    L.kda_chunk_bwd.argtypes = ([_P] * 7 + [_F, _F] + [_P] * 11 + [_I] * 6 + [_P, _Z, _P])
    L.kda_chunk_bwd_saved.argtypes = L.kda_chunk_bwd.argtypes
    L.kda_chunk_bwd_varlen_workspace_size.argtypes = [_I] * 6
    L.kda_chunk_bwd_varlen_workspace_size.restype = _Z
    L.kda_chunk_bwd_varlen.argtypes = ([_P] * 7 + [_F, _F, _P, _I, _I] + [_P] * 11 + [_I] * 4 +
                                       [_P, _Z, _P])
    L.kda_chunk_bwd_saved_varlen.argtypes = L.kda_chunk_bwd_varlen.argtypes
    L.kda_chunk_fwd_train_varlen.argtypes = L.kda_chunk_fwd_varlen_ws.argtypes
    L.kda_chunk_fwd_train.argtypes = L.kda_chunk_fwd_ws.argtypes
    L.kda_attention_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I,
                                    _I, _I, _P]
    L.kda_attention_fwd_ws.argtypes = L.kda_attention_fwd.argtypes[:-1] + [_P, _Z, _P]
    L.kda_attention_fwd_workspace_size.argtypes = [_I] * 8
    L.kda_attention_fwd_workspace_size.restype = _Z
    L.kda_decode_step.argtypes = [_P, _P, _P, _P, _P, _P, _P, _F, _F, _P, _P,
                                  _I, _I, _I, _I, _P]
    L.kda_attention_step.argtypes = ([_P] * 10 + [_F] + [_I] * 7 + [_LL] * 3 + [_I, _I, _P])
    L.kda_qk_norm_rope_fwd.argtypes = ([_P] * 9 + [_F] + [_I] * 6 + [_LL] * 2 + [_I, _I, _P])
    L.kda_qk_norm_rope_append.argtypes = ([_P] * 12 + [_F] + [_I] * 8 + [_LL] * 3 +
                                          [_I, _I, _P])
    L.kda_qk_norm_rope_bwd_workspace_size.argtypes = [_I] * 4
    L.kda_qk_norm_rope_bwd_workspace_size.restype = _Z
    L.kda_qk_norm_rope_bwd.argtypes = ([_P] * 13 + [_F] + [_I] * 6 + [_LL] * 2 +
                                       [_I, _I, _P, _Z, _P])
    L.kda_paged_attention_fwd_workspace_size.argtypes = [_I] * 6
    L.kda_paged_attention_fwd_workspace_size.restype = _Z
    L.kda_paged_attention_fwd.argtypes = ([_P] * 8 + [_F] + [_I] * 10 + [_LL, _I, _P, _Z, _P])
    L.kda_qk_norm_rope_append_q8.argtypes = ([_P] * 14 + [_F] + [_I] * 8 + [_LL] * 3 +
                                             [_I, _I, _P])
    L.kda_paged_cache_read_q8.argtypes = [_P] * 7 + [_I] * 6 + [_P]
    L.kda_paged_attention_q8_fwd_workspace_size.argtypes = [_I] * 6
    L.kda_paged_attention_q8_fwd_workspace_size.restype = _Z
    L.kda_paged_attention_q8_fwd.argtypes = ([_P] * 10 + [_F] + [_I] * 10 +
                                             [_LL, _I, _P, _Z, _P])
    L.kda_paged_prefix_attention_fwd_workspace_size.argtypes = [_I] * 7
    L.kda_paged_prefix_attention_fwd_workspace_size.restype = _Z
    L.kda_paged_prefix_attention_fwd.argtypes = ([_P] * 13 + [_F] + [_I] * 10 +
                                                 [_LL, _I, _P, _Z, _P])
    L.kda_device_error.argtypes = [_I]
    L.kda_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, _P]
    L.kda_selftest_bounded_wait.restype = _I
    for f in ("kda_chunk_fwd", "kda_chunk_fwd_varlen", "kda_chunk_fwd_ws",
              "kda_chunk_fwd_varlen_ws", "kda_chunk_fwd_noalloc", "kda_chunk_bwd",
              "kda_chunk_bwd_saved", "kda_chunk_fwd_train", "kda_chunk_bwd_varlen",
              "kda_chunk_fwd_train_varlen", "kda_chunk_bwd_saved_varlen",
              "kda_attention_fwd", "kda_attention_fwd_ws", "kda_recurrent_attention_fwd",
              "kda_recurrent_attention_fwd_ws",
              "kda_decode_step", "kda_attention_step", "kda_qk_norm_rope_fwd",
              "kda_qk_norm_rope_append", "kda_qk_norm_rope_bwd", "kda_paged_attention_fwd",
              "kda_qk_norm_rope_append_q8", "kda_paged_cache_read_q8",
              "kda_paged_attention_q8_fwd", "kda_paged_prefix_attention_fwd",
              "kda_version", "kda_device_error"):
        getattr(L, f).restype = _I
    L.kda_status_string.argtypes = [_I]
    L.kda_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = L
    return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous CUDA tensors")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype_code(x, dtype):
    if dtype is not None:
        return dtype
    import torch
    if x.dtype == torch.float32:
        return KDA_F32
    if x.dtype == torch.bfloat16:
        return KDA_BF16
    raise ValueError(f"unsupported q/k/v dtype {x.dtype}")


def _check(fn, status):
    if status != 0:
        raise KDAError(fn, status)


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return lib().kda_version()


def kda_device_error(reset: bool = True) -> int:
    """Bitmask of device-side errors recorded since the last reset (synchronises)."""
    r = lib().kda_device_error(int(bool(reset)))
    if r < 0:
        raise KDAError("kda_device_error", r)
    return r


def kda_selftest_bounded_wait(limit_ns: int, stream=None) -> None:
    """Launch a bounded wait of each kind that runs out (sets bit 3 of kda_device_error)."""
    _check("kda_selftest_bounded_wait", lib().kda_selftest_bounded_wait(int(limit_ns),
                                                                         _stream(stream)))


def kda_chunk_fwd(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                  initial_state, out, final_state, B, T, H, dk, dv, chunk=64, dtype=None,
                  stream=None):
    """Chunked forward over B equal-length sequences (see include/kda.h)."""
    _check("kda_chunk_fwd", lib().kda_chunk_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(out), _ptr(final_state),
        B, T, H, dk, dv, chunk, _dtype_code(q, dtype), _stream(stream)))


def kda_chunk_fwd_varlen(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                         cu_seqlens, N, total_T, initial_state, out, final_state, H, dk, dv,
                         chunk=64, dtype=None, stream=None):
    """Chunked forward over N packed sequences (see include/kda.h)."""
    _check("kda_chunk_fwd_varlen", lib().kda_chunk_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(cu_seqlens), N, total_T, _ptr(initial_state),
        _ptr(out), _ptr(final_state), H, dk, dv, chunk, _dtype_code(q, dtype),
        _stream(stream)))


def kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk=64, dtype=KDA_BF16) -> int:
    """Device workspace bytes kda_chunk_fwd_ws needs (0: none)."""
    return int(lib().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, dtype))


def kda_chunk_fwd_varlen_workspace_size(N, total_T, H, dk, dv, chunk=64, dtype=KDA_BF16) -> int:
    """Device workspace bytes kda_chunk_fwd_varlen_ws needs (0: none)."""
    return int(lib().kda_chunk_fwd_varlen_workspace_size(N, total_T, H, dk, dv, chunk, dtype))


def _ws(workspace):
    """(pointer, bytes) of a workspace given as a CUDA tensor, (address, bytes) or None."""
    if workspace is None:
        return None, 0
    if isinstance(workspace, tuple):
        return workspace
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def kda_chunk_fwd_ws(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                     initial_state, out, final_state, B, T, H, dk, dv, chunk=64, dtype=None,
                     workspace=None, stream=None):
    """kda_chunk_fwd through a caller workspace (two-launch path; see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_fwd_ws", lib().kda_chunk_fwd_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(out), _ptr(final_state),
        B, T, H, dk, dv, chunk, _dtype_code(q, dtype), wp, wb, _stream(stream)))


def kda_chunk_fwd_varlen_ws(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                            cu_seqlens, N, total_T, initial_state, out, final_state, H, dk, dv,
                            chunk=64, dtype=None, workspace=None, stream=None):
    """kda_chunk_fwd_varlen through a caller workspace (see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_fwd_varlen_ws", lib().kda_chunk_fwd_varlen_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(cu_seqlens), N, total_T, _ptr(initial_state),
        _ptr(out), _ptr(final_state), H, dk, dv, chunk, _dtype_code(q, dtype), wp, wb,
        _stream(stream)))


NOALLOC_SCRATCH_BYTES = 256 << 20  # include/kda.h KDA_NOALLOC_SCRATCH_BYTES


def kda_chunk_fwd_noalloc(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                          initial_state, out, final_state, B, T, H, dk, dv, chunk=64,
                          dtype=None, stream=None):
    """kda_chunk_fwd_ws with the library's own scratch array as the workspace (see
    include/kda.h)."""
    _check("kda_chunk_fwd_noalloc", lib().kda_chunk_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(out), _ptr(final_state),
        B, T, H, dk, dv, chunk, _dtype_code(q, dtype), _stream(stream)))


def kda_chunk_bwd_workspace_size(B, T, H, dk, dv, dtype=KDA_BF16) -> int:
    """Device workspace bytes kda_chunk_bwd needs for q/k/v of `dtype` (0: unsupported)."""
    return int(lib().kda_chunk_bwd_workspace_size(B, T, H, dk, dv, dtype))


def kda_chunk_bwd(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound, initial_state,
                  d_out, d_final_state, dq, dk, dv, dg, dbeta_logits, da_log, ddt_bias,
                  d_initial_state, B, T, H, dk_dim, dv_dim, dtype=None, workspace=None,
                  stream=None):
    """Gradients of kda_chunk_fwd (see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_bwd", lib().kda_chunk_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(d_out), _ptr(d_final_state),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta_logits), _ptr(da_log), _ptr(ddt_bias),
        _ptr(d_initial_state), B, T, H, dk_dim, dv_dim, _dtype_code(q, dtype), wp, wb,
        _stream(stream)))


def kda_chunk_bwd_varlen_workspace_size(N, total_T, H, dk, dv, dtype=KDA_BF16) -> int:
    """Device workspace bytes kda_chunk_bwd_varlen needs (0: unsupported)."""
    return int(lib().kda_chunk_bwd_varlen_workspace_size(N, total_T, H, dk, dv, dtype))


def kda_chunk_bwd_varlen(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                         cu_seqlens, N, total_T, initial_state, d_out, d_final_state, dq, dk,
                         dv, dg, dbeta_logits, da_log, ddt_bias, d_initial_state, H, dk_dim,
                         dv_dim, dtype=None, workspace=None, stream=None):
    """Gradients of kda_chunk_fwd_varlen (packed sequences; see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_bwd_varlen", lib().kda_chunk_bwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(cu_seqlens), N, total_T, _ptr(initial_state),
        _ptr(d_out), _ptr(d_final_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
        _ptr(dbeta_logits), _ptr(da_log), _ptr(ddt_bias), _ptr(d_initial_state), H, dk_dim,
        dv_dim, _dtype_code(q, dtype), wp, wb, _stream(stream)))


def kda_chunk_fwd_train_varlen(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                               cu_seqlens, N, total_T, initial_state, out, final_state, H, dk,
                               dv, chunk=64, dtype=None, workspace=None, stream=None):
    """The packed-sequence training forward (see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_fwd_train_varlen", lib().kda_chunk_fwd_train_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(cu_seqlens), N, total_T, _ptr(initial_state),
        _ptr(out), _ptr(final_state), H, dk, dv, chunk, _dtype_code(q, dtype), wp, wb,
        _stream(stream)))


def kda_chunk_bwd_saved_varlen(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                               cu_seqlens, N, total_T, initial_state, d_out, d_final_state, dq,
                               dk, dv, dg, dbeta_logits, da_log, ddt_bias, d_initial_state, H,
                               dk_dim, dv_dim, dtype=None, workspace=None, stream=None):
    """kda_chunk_bwd_varlen reading what kda_chunk_fwd_train_varlen kept in ``workspace``."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_bwd_saved_varlen", lib().kda_chunk_bwd_saved_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(cu_seqlens), N, total_T, _ptr(initial_state),
        _ptr(d_out), _ptr(d_final_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
        _ptr(dbeta_logits), _ptr(da_log), _ptr(ddt_bias), _ptr(d_initial_state), H, dk_dim,
        dv_dim, _dtype_code(q, dtype), wp, wb, _stream(stream)))


def kda_chunk_fwd_train(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                        initial_state, out, final_state, B, T, H, dk, dv, chunk=64, dtype=None,
                        workspace=None, stream=None):
    """The forward, keeping the backward's records in ``workspace`` (see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_fwd_train", lib().kda_chunk_fwd_train(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(out), _ptr(final_state),
        B, T, H, dk, dv, chunk, _dtype_code(q, dtype), wp, wb, _stream(stream)))


def kda_chunk_bwd_saved(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound,
                        initial_state, d_out, d_final_state, dq, dk, dv, dg, dbeta_logits,
                        da_log, ddt_bias, d_initial_state, B, T, H, dk_dim, dv_dim, dtype=None,
                        workspace=None, stream=None):
    """kda_chunk_bwd reading what kda_chunk_fwd_train kept in ``workspace``."""
    wp, wb = _ws(workspace)
    _check("kda_chunk_bwd_saved", lib().kda_chunk_bwd_saved(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(initial_state), _ptr(d_out), _ptr(d_final_state),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta_logits), _ptr(da_log), _ptr(ddt_bias),
        _ptr(d_initial_state), B, T, H, dk_dim, dv_dim, _dtype_code(q, dtype), wp, wb,
        _stream(stream)))


def kda_recurrent_attention_fwd(query, key, value, out, B, T, Hq, Hkv, D, g=None, g_gamma=None,
                                gk=None, gv=None, softmax_scale=None, initial_state=None,
                                final_state=None, cu_seqlens=None, N=0, reverse=False,
                                dtype=None, stream=None):
    """The recurrent page's gated linear recurrence (see include/kda.h)."""
    _check("kda_recurrent_attention_fwd", lib().kda_recurrent_attention_fwd(
        _ptr(query), _ptr(key), _ptr(value), _ptr(g), _ptr(g_gamma), _ptr(gk), _ptr(gv),
        float(softmax_scale or 0.0), _ptr(initial_state), _ptr(out), _ptr(final_state),
        _ptr(cu_seqlens), N, B, T, Hq, Hkv, D, int(bool(reverse)), _dtype_code(query, dtype),
        _stream(stream)))


KDA_REC_PACKED, KDA_REC_VALUE_GATE, KDA_REC_REVERSE = 1, 2, 4  # include/kda.h


def kda_recurrent_attention_fwd_workspace_size(B, T, Hq, Hkv, D, N=0, packed=False,
                                               value_gate=False, reverse=False,
                                               dtype=KDA_BF16):
    """Bytes of workspace kda_recurrent_attention_fwd_ws needs (0: none; see include/kda.h)."""
    flags = ((KDA_REC_PACKED if packed else 0) | (KDA_REC_VALUE_GATE if value_gate else 0) |
             (KDA_REC_REVERSE if reverse else 0))
    return int(lib().kda_recurrent_attention_fwd_workspace_size(N, B, T, Hq, Hkv, D, flags,
                                                                dtype))


def kda_recurrent_attention_fwd_ws(query, key, value, out, B, T, Hq, Hkv, D, g=None,
                                   g_gamma=None, gk=None, gv=None, softmax_scale=None,
                                   initial_state=None, final_state=None, cu_seqlens=None, N=0,
                                   reverse=False, dtype=None, workspace=None, stream=None):
    """kda_recurrent_attention_fwd through a caller workspace (chunked tensor-core path; see
    include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_recurrent_attention_fwd_ws", lib().kda_recurrent_attention_fwd_ws(
        _ptr(query), _ptr(key), _ptr(value), _ptr(g), _ptr(g_gamma), _ptr(gk), _ptr(gv),
        float(softmax_scale or 0.0), _ptr(initial_state), _ptr(out), _ptr(final_state),
        _ptr(cu_seqlens), N, B, T, Hq, Hkv, D, int(bool(reverse)), _dtype_code(query, dtype),
        wp, wb, _stream(stream)))


def kda_attention_fwd(query, key, value, beta, decay, initial_state, out, final_state, B, T, H,
                      dk, dv, softmax_scale=None, chunk=64, use_qk_l2norm=True,
                      use_chunked=True, order="decay_first", dtype=None, stream=None):
    """The kernel_delta_attention call: per-head log-decay (None: no decay), beta as given
    (see include/kda.h)."""
    flags = ((0 if use_qk_l2norm else KDA_ATTN_NO_QK_L2NORM) |
             (0 if use_chunked else KDA_ATTN_RECURRENT) |
             {"decay_first": 0, "literal": KDA_ATTN_ORDER_LITERAL}[order])
    _check("kda_attention_fwd", lib().kda_attention_fwd(
        _ptr(query), _ptr(key), _ptr(value), _ptr(beta), _ptr(decay), _ptr(initial_state),
        _ptr(out), _ptr(final_state), float(softmax_scale or 0.0), B, T, H, dk, dv, chunk,
        flags, _dtype_code(query, dtype), _stream(stream)))


def _attn_flags(use_qk_l2norm, use_chunked, order):
    return ((0 if use_qk_l2norm else KDA_ATTN_NO_QK_L2NORM) |
            (0 if use_chunked else KDA_ATTN_RECURRENT) |
            {"decay_first": 0, "literal": KDA_ATTN_ORDER_LITERAL}[order])


def kda_attention_fwd_workspace_size(B, T, H, dk, dv, chunk=64, use_qk_l2norm=True,
                                     use_chunked=True, order="decay_first", dtype=KDA_BF16):
    """Bytes of workspace kda_attention_fwd_ws needs (0: none; see include/kda.h)."""
    return int(lib().kda_attention_fwd_workspace_size(
        B, T, H, dk, dv, chunk, _attn_flags(use_qk_l2norm, use_chunked, order), dtype))


def kda_attention_fwd_ws(query, key, value, beta, decay, initial_state, out, final_state, B, T,
                         H, dk, dv, softmax_scale=None, chunk=64, use_qk_l2norm=True,
                         use_chunked=True, order="decay_first", dtype=None, workspace=None,
                         stream=None):
    """kda_attention_fwd through a caller workspace (tensor-core path; see include/kda.h)."""
    wp, wb = _ws(workspace)
    _check("kda_attention_fwd_ws", lib().kda_attention_fwd_ws(
        _ptr(query), _ptr(key), _ptr(value), _ptr(beta), _ptr(decay), _ptr(initial_state),
        _ptr(out), _ptr(final_state), float(softmax_scale or 0.0), B, T, H, dk, dv, chunk,
        _attn_flags(use_qk_l2norm, use_chunked, order), _dtype_code(query, dtype), wp, wb,
        _stream(stream)))


def kda_decode_step(q, k, v, g, beta_logits, a_log, dt_bias, scale, lower_bound, out, S,
                    B, H, dk, dv, stream=None):
    """One decode token for B requests, S updated in place (see include/kda.h)."""
    _check("kda_decode_step", lib().kda_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta_logits), _ptr(a_log), _ptr(dt_bias),
        float(scale), float(lower_bound), _ptr(out), _ptr(S), B, H, dk, dv, _stream(stream)))


class _Call:
    """What the serving calls look up once: torch's types, the current device and its stream.
    A serving step makes many small calls, so their arguments are checked in few Python
    operations each."""
    f32 = bf16 = i32 = i64 = e4m3 = u8 = None
    device = raw_stream = where = dense = address = None


def _setup():
    import torch
    _Call.bf16, _Call.i32, _Call.i64 = torch.bfloat16, torch.int32, torch.int64
    _Call.e4m3, _Call.u8 = torch.float8_e4m3fn, torch.uint8
    _Call.device = torch.cuda.current_device
    _Call.where, _Call.dense = torch.Tensor.get_device, torch.Tensor.is_contiguous
    _Call.address = torch.Tensor.data_ptr
    # the stream's address without building a stream object, where torch offers it
    _Call.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _Call.f32 = torch.float32  # last: what _begin looks at, perhaps in another thread


def _begin(x, dtype, stream):
    """(kda dtype, torch dtype, device, stream address) of a call whose first tensor is x."""
    if _Call.f32 is None:
        _setup()
    if dtype is None:
        el = x.dtype
        if el is _Call.bf16:
            dtype = KDA_BF16
        elif el is _Call.f32:
            dtype = KDA_F32
        else:
            raise ValueError(f"unsupported q/k/v dtype {el}")
    else:
        el = _Call.f32 if dtype == KDA_F32 else _Call.bf16
    if x.__class__ is not int and not x.is_cuda:
        raise ValueError("query must be a tensor of the current CUDA device")
    dev = _Call.device()
    if stream is None:
        stream = _Call.raw_stream(dev)
    elif stream.__class__ is not int:
        stream = stream.cuda_stream
    return dtype, el, dev, stream


def _dev(x, dtype, dev, what):
    """Address of a dense tensor of the given type on the current device (None and raw
    addresses pass as they are)."""
    if x is None or x.__class__ is int:
        return x
    if x.get_device() != dev or x.dtype is not dtype or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of the current CUDA device")
    return x.data_ptr()


def _devs(xs, dtypes, dev, names):
    """The addresses of several such arguments: whole lists are checked at once, and looked at
    one by one only when something is not a tensor of its kind."""
    try:
        if ([x.dtype for x in xs] == dtypes and all(map(_Call.dense, xs)) and
                set(map(_Call.where, xs)) == {dev}):
            return map(_Call.address, xs)
    except (AttributeError, TypeError):  # an address or None among them
        pass
    return [_dev(x, t, dev, n) for x, t, n in zip(xs, dtypes, names.split())]


def _rows(x, dtype, dev, heads, dim, what):
    """(address, token stride in elements) of a [tokens, heads, dim] argument: a raw address is
    taken as dense, a tensor may have any distance between its tokens."""
    if x is None or x.__class__ is int:
        return x, heads * dim
    if x.get_device() != dev or x.dtype is not dtype:
        raise ValueError(f"{what} must be a {dtype} tensor of the current CUDA device")
    shape, st = x.shape, x.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what} must have shape [tokens, {heads}, {dim}], not {list(shape)}")
    if (st[2] != 1 and dim > 1) or (st[1] != dim and heads > 1):
        raise ValueError(f"the heads of {what} must be dense")
    return x.data_ptr(), st[0] if shape[0] > 1 else heads * dim


def _scratch(workspace, dev):
    """_ws, for scratch that has to lie on the call's device."""
    p, n = _ws(workspace)
    if workspace is not None and workspace.__class__ is not tuple and workspace.get_device() != dev:
        raise ValueError("workspace must be a tensor of the current CUDA device")
    return p, n


def kda_attention_step(query, key, value, beta, decay, state, slots, out, N, T, Hk, Hv, dk, dv,
                       num_slots, out_slots=None, cu_seqlens=None, softmax_scale=None,
                       use_qk_l2norm=True, order="decay_first", dtype=None, stream=None):
    """A few new tokens of N requests against a pool of states (see include/kda.h): T tokens per
    request, or T packed tokens in all with ``cu_seqlens``."""
    flags = 0 if use_qk_l2norm and order == "decay_first" else _attn_flags(use_qk_l2norm, True,
                                                                           order)
    code, el, dev, st = _begin(query, dtype, stream)
    f32, i32 = _Call.f32, _Call.i32
    qp, qs = _rows(query, el, dev, Hk, dk, "query")
    kp, ks = _rows(key, el, dev, Hk, dk, "key")
    vp, vs = _rows(value, el, dev, Hv, dv, "value")
    bp, sp, lp, op = _devs((beta, state, slots, out), [f32, f32, i32, el], dev,
                           "beta state slots out")
    _check("kda_attention_step", lib().kda_attention_step(
        qp, kp, vp, bp, _dev(decay, f32, dev, "decay"), sp, lp,
        _dev(out_slots, i32, dev, "out_slots"), _dev(cu_seqlens, i32, dev, "cu_seqlens"), op,
        float(softmax_scale or 0.0), N, T, Hk, Hv, dk, dv, num_slots, qs, ks, vs, flags, code,
        st))


def _norm_rope_in(query_weight, key_weight, cos_table, sin_table, positions, dev):
    f32 = _Call.f32
    return _devs((query_weight, key_weight, cos_table, sin_table, positions),
                 [f32, f32, f32, f32, _Call.i32], dev,
                 "query_weight key_weight cos_table sin_table positions")


def kda_qk_norm_rope_fwd(query, key, query_weight, key_weight, cos_table, sin_table, positions,
                         query_out, key_out, T, Hq, Hkv, D, R, max_position, eps=1e-6,
                         interleaved=False, dtype=None, stream=None):
    """RMS norm of every query and key head and the position rotation (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    kp, ks = _rows(key, el, dev, Hkv, D, "key")
    _check("kda_qk_norm_rope_fwd", lib().kda_qk_norm_rope_fwd(
        qp, kp, *_norm_rope_in(query_weight, key_weight, cos_table, sin_table, positions, dev),
        *_devs((query_out, key_out), [el, el], dev, "query_out key_out"), float(eps), T, Hq, Hkv,
        D, R, max_position, qs, ks, KDA_ROPE_INTERLEAVED if interleaved else 0, code, st))


def kda_qk_norm_rope_append(query, key, value, query_weight, key_weight, cos_table, sin_table,
                            positions, slots, query_out, k_cache, v_cache, T, Hq, Hkv, D, R,
                            max_position, num_pages, page_size, eps=1e-6, interleaved=False,
                            dtype=None, stream=None):
    """kda_qk_norm_rope_fwd with keys and values written into cache pages (see
    include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    kp, ks = _rows(key, el, dev, Hkv, D, "key")
    vp, vs = _rows(value, el, dev, Hkv, D, "value")
    _check("kda_qk_norm_rope_append", lib().kda_qk_norm_rope_append(
        qp, kp, vp,
        *_norm_rope_in(query_weight, key_weight, cos_table, sin_table, positions, dev),
        *_devs((slots, query_out, k_cache, v_cache), [_Call.i64, el, el, el], dev,
               "slots query_out k_cache v_cache"), float(eps), T, Hq, Hkv, D, R, max_position,
        num_pages, page_size, qs, ks, vs, KDA_ROPE_INTERLEAVED if interleaved else 0, code, st))


def kda_qk_norm_rope_bwd_workspace_size(T, Hq, Hkv, D) -> int:
    """Bytes of workspace kda_qk_norm_rope_bwd needs."""
    return int(lib().kda_qk_norm_rope_bwd_workspace_size(T, Hq, Hkv, D))


def kda_qk_norm_rope_bwd(query, key, query_weight, key_weight, cos_table, sin_table, positions,
                         d_query_out, d_key_out, d_query, d_key, d_query_weight, d_key_weight, T,
                         Hq, Hkv, D, R, max_position, eps=1e-6, interleaved=False, dtype=None,
                         workspace=None, stream=None):
    """Gradients of kda_qk_norm_rope_fwd (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    f32 = _Call.f32
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    kp, ks = _rows(key, el, dev, Hkv, D, "key")
    wp, wb = _scratch(workspace, dev)
    _check("kda_qk_norm_rope_bwd", lib().kda_qk_norm_rope_bwd(
        qp, kp, *_norm_rope_in(query_weight, key_weight, cos_table, sin_table, positions, dev),
        *_devs((d_query_out, d_key_out, d_query, d_key, d_query_weight, d_key_weight),
               [el, el, el, el, f32, f32], dev,
               "d_query_out d_key_out d_query d_key d_query_weight d_key_weight"),
        float(eps), T, Hq, Hkv, D, R, max_position, qs, ks,
        KDA_ROPE_INTERLEAVED if interleaved else 0, code, wp, wb, st))


def kda_paged_attention_fwd_workspace_size(N, total_T, Hq, Hkv, D, dtype=KDA_BF16) -> int:
    """Bytes of workspace kda_paged_attention_fwd needs (0: none; see include/kda.h)."""
    return int(lib().kda_paged_attention_fwd_workspace_size(N, total_T, Hq, Hkv, D, dtype))


def kda_paged_attention_fwd(query, k_cache, v_cache, block_table, cu_seqlens, kv_lens, out, N,
                            total_T, Hq, Hkv, D, num_pages, page_size, max_pages, lse=None,
                            softmax_scale=None, window=0, sinks=0, dtype=None, workspace=None,
                            stream=None):
    """Attention of new tokens over a paged cache (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    i32 = _Call.i32
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    wp, wb = _scratch(workspace, dev)
    _check("kda_paged_attention_fwd", lib().kda_paged_attention_fwd(
        qp, *_devs((k_cache, v_cache, block_table, cu_seqlens, kv_lens, out),
                   [el, el, i32, i32, i32, el], dev,
                   "k_cache v_cache block_table cu_seqlens kv_lens out"),
        _dev(lse, _Call.f32, dev, "lse"), float(softmax_scale or 0.0), N, total_T, Hq, Hkv, D,
        num_pages, page_size, max_pages, window, sinks, qs, code, wp, wb, st))


def kda_qk_norm_rope_append_q8(query, key, value, query_weight, key_weight, cos_table, sin_table,
                               positions, slots, query_out, k_cache, v_cache, k_scale, v_scale, T,
                               Hq, Hkv, D, R, max_position, num_pages, page_size, eps=1e-6,
                               interleaved=False, dtype=None, stream=None):
    """kda_qk_norm_rope_append into pages of 8-bit rows: caches of torch.float8_e4m3fn, scales of
    torch.uint8 (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    kp, ks = _rows(key, el, dev, Hkv, D, "key")
    vp, vs = _rows(value, el, dev, Hkv, D, "value")
    e4m3, u8 = _Call.e4m3, _Call.u8
    _check("kda_qk_norm_rope_append_q8", lib().kda_qk_norm_rope_append_q8(
        qp, kp, vp,
        *_norm_rope_in(query_weight, key_weight, cos_table, sin_table, positions, dev),
        *_devs((slots, query_out, k_cache, v_cache, k_scale, v_scale),
               [_Call.i64, el, e4m3, e4m3, u8, u8], dev,
               "slots query_out k_cache v_cache k_scale v_scale"), float(eps), T, Hq, Hkv, D, R,
        max_position, num_pages, page_size, qs, ks, vs,
        KDA_ROPE_INTERLEAVED if interleaved else 0, code, st))


def kda_paged_cache_read_q8(k_cache, v_cache, k_scale, v_scale, slots, key_out, value_out, T, Hkv,
                            D, num_pages, page_size, dtype=None, stream=None):
    """Tokens of an 8-bit cache as dense rows of key_out's type (see include/kda.h)."""
    code, el, dev, st = _begin(key_out, dtype, stream)
    e4m3, u8 = _Call.e4m3, _Call.u8
    _check("kda_paged_cache_read_q8", lib().kda_paged_cache_read_q8(
        *_devs((k_cache, v_cache, k_scale, v_scale, slots, key_out, value_out),
               [e4m3, e4m3, u8, u8, _Call.i64, el, el], dev,
               "k_cache v_cache k_scale v_scale slots key_out value_out"), T, Hkv, D, num_pages,
        page_size, code, st))


def kda_paged_attention_q8_fwd_workspace_size(N, total_T, Hq, Hkv, D, dtype=KDA_BF16) -> int:
    """Bytes of workspace kda_paged_attention_q8_fwd needs (0: none; see include/kda.h)."""
    return int(lib().kda_paged_attention_q8_fwd_workspace_size(N, total_T, Hq, Hkv, D, dtype))


def kda_paged_attention_q8_fwd(query, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                               kv_lens, out, N, total_T, Hq, Hkv, D, num_pages, page_size,
                               max_pages, lse=None, softmax_scale=None, window=0, sinks=0,
                               dtype=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache in 8 bits (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    i32, e4m3, u8 = _Call.i32, _Call.e4m3, _Call.u8
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    wp, wb = _scratch(workspace, dev)
    _check("kda_paged_attention_q8_fwd", lib().kda_paged_attention_q8_fwd(
        qp, *_devs((k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, kv_lens, out),
                   [e4m3, e4m3, u8, u8, i32, i32, i32, el], dev,
                   "k_cache v_cache k_scale v_scale block_table cu_seqlens kv_lens out"),
        _dev(lse, _Call.f32, dev, "lse"), float(softmax_scale or 0.0), N, total_T, Hq, Hkv, D,
        num_pages, page_size, max_pages, window, sinks, qs, code, wp, wb, st))


def kda_paged_prefix_attention_fwd_workspace_size(num_groups, N, total_T, Hq, Hkv, D,
                                                  dtype=KDA_BF16) -> int:
    """Bytes of workspace kda_paged_prefix_attention_fwd needs (see include/kda.h)."""
    return int(lib().kda_paged_prefix_attention_fwd_workspace_size(num_groups, N, total_T, Hq, Hkv,
                                                                   D, dtype))


def kda_paged_prefix_attention_fwd(query, k_cache, v_cache, prefix_table, prefix_lens, cu_groups,
                                   block_table, cu_seqlens, kv_lens, out, num_groups, N, total_T,
                                   Hq, Hkv, D, num_pages, page_size, max_prefix_pages, max_pages,
                                   k_scale=None, v_scale=None, lse=None, softmax_scale=None,
                                   dtype=None, workspace=None, stream=None):
    """Attention of groups of sequences that share prefixes, over pages of query's type or, with
    scales, of 8 bits (see include/kda.h)."""
    code, el, dev, st = _begin(query, dtype, stream)
    i32, u8 = _Call.i32, _Call.u8
    kept = el if k_scale is None and v_scale is None else _Call.e4m3
    qp, qs = _rows(query, el, dev, Hq, D, "query")
    wp, wb = _scratch(workspace, dev)
    kp, vp, *rest = _devs(
        (k_cache, v_cache, prefix_table, prefix_lens, cu_groups, block_table, cu_seqlens, kv_lens,
         out), [kept, kept, i32, i32, i32, i32, i32, i32, el], dev,
        "k_cache v_cache prefix_table prefix_lens cu_groups block_table cu_seqlens kv_lens out")
    _check("kda_paged_prefix_attention_fwd", lib().kda_paged_prefix_attention_fwd(
        qp, kp, vp, _dev(k_scale, u8, dev, "k_scale"), _dev(v_scale, u8, dev, "v_scale"), *rest,
        _dev(lse, _Call.f32, dev, "lse"), float(softmax_scale or 0.0), num_groups, N, total_T, Hq,
        Hkv, D, num_pages, page_size, max_prefix_pages, max_pages, qs, code, wp, wb, st))
