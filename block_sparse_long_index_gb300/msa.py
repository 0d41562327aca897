"""ctypes binding of libmsa.so: the C ABI of include/msa.h under the same names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (bf16 as ``torch.bfloat16``, int32 as
``torch.int32``); their device pointers and the current torch stream are
passed through.  Importing this module loads ``libmsa.so`` and fails loudly if
it is missing — there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libmsa.so is not built (run __graft_entry__.build() or "
                      "python -m block_sparse_long_index_gb300.build); there is no fallback path")
_lib = ctypes.CDLL(LIB_PATH)

MSA_OK = 0
MSA_ERR_INVALID_ARGUMENT = 1
MSA_ERR_UNSUPPORTED = 2
MSA_ERR_WORKSPACE_TOO_SMALL = 3
MSA_ERR_CUDA = 4
MSA_ERR_BAD_INDEX = 5
MSA_ERR_TIMEOUT = 6
MSA_ERR_NO_PAGES = 7


class msa_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int),
                ("d_I", ctypes.c_int), ("Bk", ctypes.c_int), ("k", ctypes.c_int)]


class msa_kv4_pool_t(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("H_kv", ctypes.c_int), ("d", ctypes.c_int)]


class msa_pages_t(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("max_pages", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("n_seqs", ctypes.c_int),
                ("page_size", ctypes.c_int)]


class msa_page_pool_t(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


class msa_rope_t(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("factor", ctypes.c_float)]


class msa_kv_pool_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int)]


class msa_append_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_idx", "k_idx")] +
                [(n + "_stride", ctypes.c_int64) for n in ("q", "k", "v", "q_idx", "k_idx")] +
                [(n, ctypes.c_void_p) for n in ("q_out", "q_idx_out", "k_idx_pool", "positions")] +
                [("H_q", ctypes.c_int), ("d_I", ctypes.c_int), ("idx_f8", ctypes.c_int), ("idx_scale", ctypes.c_float)])


_P, _I64, _I, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SP = ctypes.POINTER(msa_shape_t)
_KP, _GP, _LP = ctypes.POINTER(msa_kv4_pool_t), ctypes.POINTER(msa_pages_t), ctypes.POINTER(msa_page_pool_t)
_RP, _VP, _AP = ctypes.POINTER(msa_rope_t), ctypes.POINTER(msa_kv_pool_t), ctypes.POINTER(msa_append_t)

_SIGS = {
    "msa_select_blocks_workspace": (_SZ, [_I64, _I, _I, _I, _I]),
    "msa_select_blocks": (_I, [_P, _P, _I64, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "msa_invert_blocks_workspace": (_SZ, [_I64, _I, _I, _I]),
    "msa_invert_blocks": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "msa_sparse_attn_fwd_workspace": (_SZ, [_SP]),
    "msa_sparse_attn_fwd": (_I, [_P, _P, _P, _P, _SP, _F, _P, _P, _P, _SZ, _P]),
    "msa_sparse_attn_bwd_workspace": (_SZ, [_SP]),
    "msa_sparse_attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _SP, _F, _F, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                 _P]),
    "msa_prefill_workspace": (_SZ, [_SP]),
    "msa_prefill": (_I, [_P, _P, _P, _P, _P, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_workspace": (_SZ, [_I, _SP]),
    "msa_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_paged": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _SP, _F, _P, _P, _P, _P]),
    "msa_quantize_e4m3": (_I, [_P, _I64, _F, _P, _P]),
    "msa_warmup_fwd": (_I, [_P, _P, _P, _P, _P, _SP, _F, _P, _P, _P, _P]),
    "msa_warmup_index_grad": (_I, [_P, _P, _P, _P, _P, _P, _SP, _F, _F, _P, _P, _P, _P]),
    "msa_select_blocks_varlen_workspace": (_SZ, [_I64, _I, _I, _I, _I]),
    "msa_select_blocks_varlen": (_I, [_P, _P, _P, _I, _I64, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "msa_prefill_varlen_workspace": (_SZ, [_SP]),
    "msa_prefill_varlen": (_I, [_P, _P, _P, _P, _P, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_select_blocks_fp8": (_I, [_P, _P, _I64, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "msa_prefill_fp8": (_I, [_P, _P, _P, _P, _P, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_paged_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_dense_prefill_varlen_workspace": (_SZ, [_I64, _I, _I, _I, _I]),
    "msa_dense_prefill_varlen": (_I, [_P, _P, _P, _P, _I, _I64, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "msa_kv4_workspace": (_SZ, []),
    "msa_kv4_store": (_I, [_P, _P, _I64, _P, _I, _P, _P, _I64, _KP, _P, _SZ, _P]),
    "msa_kv4_load": (_I, [_KP, _I64, _P, _I, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "msa_dense_decode_paged_kv4_workspace": (_SZ, [_I, _I, _I, _I]),
    "msa_dense_decode_paged_kv4": (_I, [_P, _KP, _P, _I64, _P, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "msa_decode_paged_kv4": (_I, [_P, _P, _P, _KP, _P, _I64, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_decode_paged_kv4_fp8": (_I, [_P, _P, _P, _KP, _P, _I64, _P, _I, _SP, _F, _P, _P, _P, _P, _SZ, _P]),
    "msa_pages_workspace": (_SZ, [_GP, _I]),
    "msa_pages_reserve": (_I, [_GP, _P, _P, _I, _P, _SZ, _P]),
    "msa_pages_fork": (_I, [_GP, _P, _P, _I, _LP, _I, _P, _SZ, _P]),
    "msa_pages_free": (_I, [_GP, _P, _I, _P, _SZ, _P]),
    "msa_pages_compact": (_I, [_GP, _LP, _I, _P, _P, _P, _SZ, _P]),
    "msa_pages_accept_workspace": (_SZ, [_GP, _I, _I]),
    "msa_pages_accept": (_I, [_GP, _P, _P, _P, _P, _I, _I, _LP, _I, _P, _SZ, _P]),
    "msa_rope": (_I, [_P, _I64, _P, _I64, _I64, _I, _I, _I, _P, _RP, _I, _P]),
    "msa_append_workspace": (_SZ, []),
    "msa_append_paged": (_I, [_AP, _I64, _P, _I, _P, _P, _I64, _VP, _RP, _RP, _P, _SZ, _P]),
    "msa_append_paged_kv4": (_I, [_AP, _I64, _P, _I, _P, _P, _I64, _KP, _RP, _RP, _P, _SZ, _P]),
    "msa_tree_decode_workspace": (_SZ, [_I, _I, _I, _I, _I]),
    "msa_tree_decode_paged": (_I, [_P, _VP, _P, _I64, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "msa_tree_decode_paged_kv4": (_I, [_P, _KP, _P, _I64, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "msa_verify_workspace": (_SZ, []),
    "msa_verify_tree": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I64, _P, _P, _P, _P, _SZ, _P]),
    "msa_check_device_error": (_I, [_P, _P]),
    "msa_status_string": (ctypes.c_char_p, [_I]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTS = tuple(_SIGS)


class MsaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, msa_status_string(status), status))


def _ptr(t):
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        return int(t)


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())  # (no Stream object: 1 us less)
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _check(status, where):
    if status != MSA_OK:
        raise MsaError(status, where)
    return status


def shape(N, H_q, H_kv, d, d_I, Bk, k):
    return msa_shape_t(int(N), int(H_q), int(H_kv), int(d), int(d_I), int(Bk), int(k))


# ---------------------------------------------------------------- same-name wrappers
def msa_status_string(status):
    return _lib.msa_status_string(int(status)).decode()


def msa_select_blocks_workspace(N, G, d_I, Bk, k):
    return int(_lib.msa_select_blocks_workspace(N, G, d_I, Bk, k))


def msa_select_blocks(q_idx, k_idx, N, G, d_I, Bk, k, block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_select_blocks(_ptr(q_idx), _ptr(k_idx), N, G, d_I, Bk, k, _ptr(block_idx),
                                         _ptr(workspace), wb, _stream(stream)), "msa_select_blocks")


def msa_invert_blocks_workspace(N, G, Bk, k):
    return int(_lib.msa_invert_blocks_workspace(N, G, Bk, k))


def msa_invert_blocks(block_idx, N, G, Bk, k, row_ptr, entries, n_entries, workspace, workspace_bytes=None,
                      stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_invert_blocks(_ptr(block_idx), N, G, Bk, k, _ptr(row_ptr), _ptr(entries),
                                         _ptr(n_entries), _ptr(workspace), wb, _stream(stream)),
                  "msa_invert_blocks")


def msa_sparse_attn_fwd_workspace(shp):
    return int(_lib.msa_sparse_attn_fwd_workspace(ctypes.byref(shp)))


def msa_sparse_attn_fwd(q, k, v, block_idx, shp, scale, out, lse, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_sparse_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(block_idx), ctypes.byref(shp),
                                           float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                           _stream(stream)), "msa_sparse_attn_fwd")


def msa_sparse_attn_bwd_workspace(shp):
    return int(_lib.msa_sparse_attn_bwd_workspace(ctypes.byref(shp)))


def msa_sparse_attn_bwd(q, k, v, q_idx, k_idx, block_idx, out, lse, dout, shp, scale, kl_weight, dq, dk, dv, dq_idx,
                        dk_idx, kl, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_sparse_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), _ptr(block_idx),
                                           _ptr(out), _ptr(lse), _ptr(dout), ctypes.byref(shp), float(scale),
                                           float(kl_weight), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dq_idx), _ptr(dk_idx),
                                           _ptr(kl), _ptr(workspace), wb, _stream(stream)), "msa_sparse_attn_bwd")


def msa_prefill_workspace(shp):
    return int(_lib.msa_prefill_workspace(ctypes.byref(shp)))


def msa_prefill(q, k, v, q_idx, k_idx, shp, scale, block_idx, out, lse, workspace, workspace_bytes=None,
                stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), ctypes.byref(shp),
                                   float(scale), _ptr(block_idx), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                   _stream(stream)), "msa_prefill")


def msa_decode_workspace(B, shp):
    return int(_lib.msa_decode_workspace(B, ctypes.byref(shp)))


def msa_decode(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, B, shp, scale, out, lse, block_idx,
               workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_cache), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(ctx_len), B, ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse),
                                  _ptr(block_idx), _ptr(workspace), wb, _stream(stream)), "msa_decode")


def msa_decode_paged(q_t, q_idx_t, k_idx_pool, k_pool, v_pool, page_table, max_pages, n_pages, page_size, ctx_len,
                     B, shp, scale, out, lse, block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode_paged(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_pool), _ptr(k_pool), _ptr(v_pool),
                                        _ptr(page_table), int(max_pages), int(n_pages), int(page_size), _ptr(ctx_len),
                                        B, ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse), _ptr(block_idx),
                                        _ptr(workspace), wb, _stream(stream)), "msa_decode_paged")


def msa_decode_noalloc(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, B, shp, scale, out, lse, block_idx,
                       stream=None):
    """msa_decode without a workspace, for callers that may not allocate device memory (the library's
    fixed 8 MiB device array is the scratch; calls on one device must not overlap)."""
    return _check(_lib.msa_decode_noalloc(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_cache), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(ctx_len), B, ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse),
                                          _ptr(block_idx), _stream(stream)), "msa_decode_noalloc")


def msa_quantize_e4m3(x, n, scale, y, stream=None):
    return _check(_lib.msa_quantize_e4m3(_ptr(x), int(n), float(scale), _ptr(y), _stream(stream)),
                  "msa_quantize_e4m3")


def msa_select_blocks_fp8(q_idx, k_idx, N, G, d_I, Bk, k, block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_select_blocks_fp8(_ptr(q_idx), _ptr(k_idx), N, G, d_I, Bk, k, _ptr(block_idx),
                                             _ptr(workspace), wb, _stream(stream)), "msa_select_blocks_fp8")


def msa_prefill_fp8(q, k, v, q_idx, k_idx, shp, scale, block_idx, out, lse, workspace, workspace_bytes=None,
                    stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_prefill_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), ctypes.byref(shp),
                                       float(scale), _ptr(block_idx), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                       _stream(stream)), "msa_prefill_fp8")


def msa_decode_fp8(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, B, shp, scale, out, lse, block_idx,
                   workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode_fp8(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_cache), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(ctx_len), B, ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse),
                                      _ptr(block_idx), _ptr(workspace), wb, _stream(stream)), "msa_decode_fp8")


def msa_decode_paged_fp8(q_t, q_idx_t, k_idx_pool, k_pool, v_pool, page_table, max_pages, n_pages, page_size,
                         ctx_len, B, shp, scale, out, lse, block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode_paged_fp8(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_pool), _ptr(k_pool),
                                            _ptr(v_pool), _ptr(page_table), int(max_pages), int(n_pages),
                                            int(page_size), _ptr(ctx_len), B, ctypes.byref(shp), float(scale),
                                            _ptr(out), _ptr(lse), _ptr(block_idx), _ptr(workspace), wb,
                                            _stream(stream)), "msa_decode_paged_fp8")


def msa_select_blocks_varlen_workspace(N, G, d_I, Bk, k):
    return int(_lib.msa_select_blocks_varlen_workspace(N, G, d_I, Bk, k))


def msa_select_blocks_varlen(q_idx, k_idx, cu_seqlens, S, N, G, d_I, Bk, k, block_idx, workspace,
                             workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_select_blocks_varlen(_ptr(q_idx), _ptr(k_idx), _ptr(cu_seqlens), int(S), N, G, d_I, Bk,
                                                k, _ptr(block_idx), _ptr(workspace), wb, _stream(stream)),
                  "msa_select_blocks_varlen")


def msa_prefill_varlen_workspace(shp):
    return int(_lib.msa_prefill_varlen_workspace(ctypes.byref(shp)))


def msa_prefill_varlen(q, k, v, q_idx, k_idx, cu_seqlens, S, shp, scale, block_idx, out, lse, workspace,
                       workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), _ptr(cu_seqlens),
                                          int(S), ctypes.byref(shp), float(scale), _ptr(block_idx), _ptr(out),
                                          _ptr(lse), _ptr(workspace), wb, _stream(stream)), "msa_prefill_varlen")


def msa_warmup_fwd(q, k, v, q_idx, k_idx, shp, scale, out, lse, lse_idx, stream=None):
    return _check(_lib.msa_warmup_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), ctypes.byref(shp),
                                      float(scale), _ptr(out), _ptr(lse), _ptr(lse_idx), _stream(stream)),
                  "msa_warmup_fwd")


def msa_warmup_index_grad(q, k, q_idx, k_idx, lse, lse_idx, shp, scale, kl_weight, dq_idx, dk_idx, kl, stream=None):
    return _check(_lib.msa_warmup_index_grad(_ptr(q), _ptr(k), _ptr(q_idx), _ptr(k_idx), _ptr(lse), _ptr(lse_idx),
                                             ctypes.byref(shp), float(scale), float(kl_weight), _ptr(dq_idx),
                                             _ptr(dk_idx), _ptr(kl), _stream(stream)), "msa_warmup_index_grad")


def msa_dense_prefill_varlen_workspace(N, S, H_q, H_kv, d):
    return int(_lib.msa_dense_prefill_varlen_workspace(int(N), int(S), H_q, H_kv, d))


def msa_dense_prefill_varlen(q, k, v, cu_seqlens, S, N, H_q, H_kv, d, scale, out, lse, workspace,
                             workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_dense_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(S), int(N), H_q, H_kv,
                                                d, float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                                _stream(stream)), "msa_dense_prefill_varlen")


def kv4_pool(k_codes, k_scales, v_codes, v_scales, n_pages, page_size, H_kv, d):
    return msa_kv4_pool_t(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), int(n_pages), int(page_size),
                          int(H_kv), int(d))


def msa_kv4_workspace():
    return int(_lib.msa_kv4_workspace())


def msa_kv4_store(k, v, N, cu_seqlens, S, pos0, page_table, max_pages, pool, workspace, workspace_bytes=None,
                  stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_kv4_store(_ptr(k), _ptr(v), int(N), _ptr(cu_seqlens), int(S), _ptr(pos0), _ptr(page_table),
                                     int(max_pages), ctypes.byref(pool), _ptr(workspace), wb, _stream(stream)),
                  "msa_kv4_store")


def msa_kv4_load(pool, N, cu_seqlens, S, pos0, page_table, max_pages, k, v, workspace, workspace_bytes=None,
                 stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_kv4_load(ctypes.byref(pool), int(N), _ptr(cu_seqlens), int(S), _ptr(pos0),
                                    _ptr(page_table), int(max_pages), _ptr(k), _ptr(v), _ptr(workspace), wb,
                                    _stream(stream)), "msa_kv4_load")


def msa_dense_decode_paged_kv4_workspace(B, H_q, H_kv, d):
    return int(_lib.msa_dense_decode_paged_kv4_workspace(int(B), H_q, H_kv, d))


def msa_dense_decode_paged_kv4(q_t, pool, page_table, max_pages, ctx_len, B, H_q, scale, out, lse, workspace,
                               workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_dense_decode_paged_kv4(_ptr(q_t), ctypes.byref(pool), _ptr(page_table), int(max_pages),
                                                  _ptr(ctx_len), int(B), H_q, float(scale), _ptr(out), _ptr(lse),
                                                  _ptr(workspace), wb, _stream(stream)), "msa_dense_decode_paged_kv4")


def msa_decode_paged_kv4(q_t, q_idx_t, k_idx_pool, pool, page_table, max_pages, ctx_len, B, shp, scale, out, lse,
                         block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode_paged_kv4(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_pool), ctypes.byref(pool),
                                            _ptr(page_table), int(max_pages), _ptr(ctx_len), int(B),
                                            ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse), _ptr(block_idx),
                                            _ptr(workspace), wb, _stream(stream)), "msa_decode_paged_kv4")


def msa_decode_paged_kv4_fp8(q_t, q_idx_t, k_idx_pool, pool, page_table, max_pages, ctx_len, B, shp, scale, out, lse,
                             block_idx, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_decode_paged_kv4_fp8(_ptr(q_t), _ptr(q_idx_t), _ptr(k_idx_pool), ctypes.byref(pool),
                                                _ptr(page_table), int(max_pages), _ptr(ctx_len), int(B),
                                                ctypes.byref(shp), float(scale), _ptr(out), _ptr(lse),
                                                _ptr(block_idx), _ptr(workspace), wb, _stream(stream)),
                  "msa_decode_paged_kv4_fp8")


def pages(page_table, ctx_len, refs, max_pages, n_pages, n_seqs, page_size):
    return msa_pages_t(_ptr(page_table), _ptr(ctx_len), _ptr(refs), int(max_pages), int(n_pages), int(n_seqs),
                       int(page_size))


def page_pools(entries):
    """A C array of (base, page_bytes) entries for the page calls."""
    entries = list(entries)
    return (msa_page_pool_t * max(1, len(entries)))(*[msa_page_pool_t(_ptr(b), int(n)) for b, n in entries])


def msa_pages_workspace(pgs, n):
    return int(_lib.msa_pages_workspace(ctypes.byref(pgs), int(n)))


def msa_pages_reserve(pgs, seqs, new_len, n, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_pages_reserve(ctypes.byref(pgs), _ptr(seqs), _ptr(new_len), int(n), _ptr(workspace), wb,
                                         _stream(stream)), "msa_pages_reserve")


def msa_pages_fork(pgs, src, dst, n, pools, n_pools, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_pages_fork(ctypes.byref(pgs), _ptr(src), _ptr(dst), int(n), pools, int(n_pools),
                                      _ptr(workspace), wb, _stream(stream)), "msa_pages_fork")


def msa_pages_free(pgs, seqs, n, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_pages_free(ctypes.byref(pgs), _ptr(seqs), int(n), _ptr(workspace), wb, _stream(stream)),
                  "msa_pages_free")


def msa_pages_compact(pgs, pools, n_pools, page_map, n_live, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_pages_compact(ctypes.byref(pgs), pools, int(n_pools), _ptr(page_map), _ptr(n_live),
                                         _ptr(workspace), wb, _stream(stream)), "msa_pages_compact")


def msa_pages_accept_workspace(pgs, n, T):
    return int(_lib.msa_pages_accept_workspace(ctypes.byref(pgs), int(n), int(T)))


def msa_pages_accept(pgs, seqs, base, path, n_path, n, T, pools, n_pools, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_pages_accept(ctypes.byref(pgs), _ptr(seqs), _ptr(base), _ptr(path), _ptr(n_path), int(n),
                                        int(T), pools, int(n_pools), _ptr(workspace), wb, _stream(stream)),
                  "msa_pages_accept")


def rope(turns, rot, interleaved, factor):
    return msa_rope_t(_ptr(turns), int(rot), int(bool(interleaved)), float(factor))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def msa_rope(x, x_stride, y, y_stride, N, H, d, f32, positions, rope, inverse, stream=None):
    return _check(_lib.msa_rope(_ptr(x), int(x_stride), _ptr(y), int(y_stride), int(N), int(H), int(d), int(bool(f32)),
                                _ptr(positions), _ref(rope), int(bool(inverse)), _stream(stream)), "msa_rope")


def kv_pool(k, v, n_pages, page_size, H_kv, d):
    return msa_kv_pool_t(_ptr(k), _ptr(v), int(n_pages), int(page_size), int(H_kv), int(d))


def msa_append_workspace():
    return int(_lib.msa_append_workspace())


def msa_append_paged(rows, N, cu_seqlens, S, pos0, page_table, max_pages, pool, rope, rope_idx, workspace,
                     workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_append_paged(ctypes.byref(rows), int(N), _ptr(cu_seqlens), int(S), _ptr(pos0),
                                        _ptr(page_table), int(max_pages), ctypes.byref(pool), _ref(rope),
                                        _ref(rope_idx), _ptr(workspace), wb, _stream(stream)), "msa_append_paged")


def msa_append_paged_kv4(rows, N, cu_seqlens, S, pos0, page_table, max_pages, pool, rope, rope_idx, workspace,
                         workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_append_paged_kv4(ctypes.byref(rows), int(N), _ptr(cu_seqlens), int(S), _ptr(pos0),
                                            _ptr(page_table), int(max_pages), ctypes.byref(pool), _ref(rope),
                                            _ref(rope_idx), _ptr(workspace), wb, _stream(stream)),
                  "msa_append_paged_kv4")


def msa_tree_decode_workspace(B, T, H_q, H_kv, d):
    return int(_lib.msa_tree_decode_workspace(int(B), int(T), int(H_q), int(H_kv), int(d)))


def msa_tree_decode_paged(q, pool, page_table, max_pages, ctx_len, tree_len, parents, B, T, H_q, scale, out, lse,
                          workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_tree_decode_paged(_ptr(q), ctypes.byref(pool), _ptr(page_table), int(max_pages),
                                             _ptr(ctx_len), _ptr(tree_len), _ptr(parents), int(B), int(T), int(H_q),
                                             float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wb, _stream(stream)),
                  "msa_tree_decode_paged")


def msa_tree_decode_paged_kv4(q, pool, page_table, max_pages, ctx_len, tree_len, parents, B, T, H_q, scale, out, lse,
                              workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_tree_decode_paged_kv4(_ptr(q), ctypes.byref(pool), _ptr(page_table), int(max_pages),
                                                 _ptr(ctx_len), _ptr(tree_len), _ptr(parents), int(B), int(T),
                                                 int(H_q), float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wb,
                                                 _stream(stream)), "msa_tree_decode_paged_kv4")


def msa_verify_workspace():
    return int(_lib.msa_verify_workspace())


def msa_verify_tree(probs, draft_probs, tokens, parents, tree_len, u, u_last, B, T, V, path, n_path, next_token,
                    workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() if workspace_bytes is None else workspace_bytes
    return _check(_lib.msa_verify_tree(_ptr(probs), _ptr(draft_probs), _ptr(tokens), _ptr(parents), _ptr(tree_len),
                                       _ptr(u), _ptr(u_last), int(B), int(T), int(V), _ptr(path), _ptr(n_path),
                                       _ptr(next_token), _ptr(workspace), wb, _stream(stream)), "msa_verify_tree")


def msa_check_device_error(workspace, stream=None):
    """Returns the device status code (raises nothing)."""
    return int(_lib.msa_check_device_error(_ptr(workspace), _stream(stream)))


def raw():
    """The loaded ctypes library (for status-code tests that bypass the wrappers)."""
    return _lib
