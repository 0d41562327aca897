"""Tensor-level entry points over the C ABI (allocation of outputs and workspaces with torch).

``MsaPrefill`` / ``MsaDecode`` own their outputs and workspace so repeated steps
allocate nothing; ``prefill`` / ``decode`` are one-shot conveniences.  All
compute is in libmsa.so.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import msa as _c


def _check_bf16(name, t, shape):
    if t.dtype is torch.bfloat16 and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA bfloat16 tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


class MsaPrefill:
    """One prefill layer step: select -> (invert + KV-outer attention + combine).

    Calling the object runs msa_prefill (both stages in one call); ``select``
    and ``attend`` run the two stages as separate calls."""

    def __init__(self, N, H_q, H_kv, d, d_I, Bk, k, device="cuda"):
        self.N, self.H_q, self.H_kv, self.d, self.d_I, self.Bk, self.k = N, H_q, H_kv, d, d_I, Bk, k
        self.G = H_kv
        self.shape = _c.shape(N, H_q, H_kv, d, d_I, Bk, k)
        ws = max(_c.msa_select_blocks_workspace(N, self.G, d_I, Bk, k), _c.msa_sparse_attn_fwd_workspace(self.shape),
                 _c.msa_prefill_workspace(self.shape))
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        self.block_idx = torch.empty((self.G, N, k), dtype=torch.int32, device=device)
        self.out = torch.empty((N, H_q, d), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((H_q, N), dtype=torch.float32, device=device)

    def select(self, q_idx, k_idx, stream=None):
        _c.msa_select_blocks(q_idx, k_idx, self.N, self.G, self.d_I, self.Bk, self.k, self.block_idx,
                             self.workspace, stream=stream)
        return self.block_idx

    def attend(self, q, k, v, block_idx=None, scale=None, stream=None, out=None, lse=None):
        """The attention stage; out / lse default to the object's own buffers."""
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        _c.msa_sparse_attn_fwd(q, k, v, self.block_idx if block_idx is None else block_idx, self.shape, scale,
                               out, lse, self.workspace, stream=stream)
        return out, lse

    def __call__(self, q, k, v, q_idx, k_idx, scale=None, stream=None):
        N, G = self.N, self.G
        _check_bf16("q", q, (N, self.H_q, self.d))
        _check_bf16("k", k, (N, self.H_kv, self.d))
        _check_bf16("v", v, (N, self.H_kv, self.d))
        _check_bf16("q_idx", q_idx, (N, G, self.d_I))
        _check_bf16("k_idx", k_idx, (N, self.d_I))
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        _c.msa_prefill(q, k, v, q_idx, k_idx, self.shape, scale, self.block_idx, self.out, self.lse, self.workspace,
                       stream=stream)
        return self.out, self.lse, self.block_idx

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class MsaDecode:
    """One decode step for B sequences over caches of capacity ctx_max."""

    def __init__(self, B, ctx_max, H_q, H_kv, d, d_I, Bk, k, device="cuda"):
        self.B, self.ctx_max = B, ctx_max
        self.H_q, self.H_kv, self.d, self.d_I, self.Bk, self.k = H_q, H_kv, d, d_I, Bk, k
        self.shape = _c.shape(ctx_max, H_q, H_kv, d, d_I, Bk, k)
        self.workspace = torch.empty(_c.msa_decode_workspace(B, self.shape), dtype=torch.uint8, device=device)
        self.out = torch.empty((B, H_q, d), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((B, H_q), dtype=torch.float32, device=device)
        self.block_idx = torch.empty((B, H_kv, k), dtype=torch.int32, device=device)

    def __call__(self, q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, scale=None, stream=None):
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        _c.msa_decode(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, self.B, self.shape, scale, self.out,
                      self.lse, self.block_idx, self.workspace, stream=stream)
        return self.out, self.lse, self.block_idx

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


def _check_tensor(name, t, dtype, shape, dev=None):
    """t: contiguous, of the type and shape, on device number dev (any CUDA device where dev is None)."""
    at = t.get_device()  # -1 on the CPU
    if t.dtype is dtype and t.shape == shape and at >= 0 and (dev is None or at == dev) and t.is_contiguous():
        return
    if t.dtype != dtype or at < 0 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA %s tensor" % (name, str(dtype).replace("torch.", "")))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if at != dev and dev is not None:
        raise ValueError("%s is on cuda:%d, the object on cuda:%d" % (name, at, dev))


def _device(t):
    """The number of t's device, which has to be the current one: launches go there."""
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError("the object is on cuda:%d, the current device is cuda:%d" % (dev, torch.cuda.current_device()))
    return dev


def _allocating_for(stream):
    """Within it tensors come from the memory of `stream` (None: the current one), so that work of the current stream
    that still uses a freed block is not overtaken by the stream's."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _settled(tensors):
    """The tensors, whose clearing on the current stream is over: the first call on them may be on another stream."""
    with torch.cuda.device(tensors[0].device):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return tensors


class MsaDensePrefill:
    """Dense causal attention over packed prompts of N rows in all, S sequences.

    A call returns the object's own ``out`` and ``lse``, which the next call overwrites; two calls in flight at once
    need two objects."""

    def __init__(self, N, H_q, H_kv, d, S, device="cuda"):
        self.N, self.H_q, self.H_kv, self.d, self.S = N, H_q, H_kv, d, S
        self.workspace = torch.empty(_c.msa_dense_prefill_varlen_workspace(N, S, H_q, H_kv, d), dtype=torch.uint8,
                                     device=device)
        self.out = torch.empty((N, H_q, d), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((H_q, N), dtype=torch.float32, device=device)

    def __call__(self, q, k, v, cu_seqlens, scale=None, stream=None):
        dev = _device(self.workspace)
        _check_tensor("q", q, torch.bfloat16, (self.N, self.H_q, self.d), dev)
        _check_tensor("k", k, torch.bfloat16, (self.N, self.H_kv, self.d), dev)
        _check_tensor("v", v, torch.bfloat16, (self.N, self.H_kv, self.d), dev)
        _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (self.S + 1,), dev)
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        _c.msa_dense_prefill_varlen(q, k, v, cu_seqlens, self.S, self.N, self.H_q, self.H_kv, self.d, scale, self.out,
                                    self.lse, self.workspace, stream=stream)
        return self.out, self.lse

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_len=None, beta_fast=32.0, beta_slow=1.0):
    """Radians a position of the rot / 2 pairs, a list of floats: base^(-2 i / rot), scaled for contexts `factor` times
    as long as those of training where `scaling` says so:

    "linear"   every frequency over factor;
    "base"     the base grown so that the lowest frequency falls by factor and the highest stays: base factor^(rot / (rot - 2));
    "parts"    a pair that turns over beta_fast times within original_len positions stays, one that turns less than
               beta_slow times is divided by factor, those between are mixed linearly in their index.
               (Attention over such rows is often sharpened by Rope's `factor` 1 + 0.1 ln factor.)"""
    rot, base, factor = int(rot), float(base), float(factor)
    if rot < 2 or rot % 2:
        raise ValueError("rot has to be even")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base has to be above 1 and factor at least 1")
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling by the base needs two pairs at least")
        base *= factor ** (rot / (rot - 2.0))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling in (None, "base"):
        return f
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling != "parts":
        raise ValueError("scaling is None, 'linear', 'base' or 'parts'")
    if not original_len or original_len < 1:
        raise ValueError("scaling by parts needs original_len")
    # the (real) index of the pair that turns n times within original_len
    index = lambda n: rot * math.log(original_len / (2.0 * math.pi * n)) / (2.0 * math.log(base))  # noqa: E731
    lo, hi = max(0.0, math.floor(index(beta_fast))), min(rot - 1.0, math.ceil(index(beta_slow)))
    mix = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
    return [x * (1.0 - m) + x / factor * m for x, m in zip(f, mix)]


class Rope:
    """Rotary positions: a table of frequencies on the device.  Calling it turns rows (or turns them back).

    ``Rope(rot, base, ...)`` takes rope_frequencies' arguments, ``Rope.from_frequencies`` any frequencies in radians a
    position.  `amplitude` multiplies the turned channels."""

    def __init__(self, rot, base=10000.0, interleaved=False, amplitude=1.0, device="cuda", **scaling):
        self._set(rope_frequencies(rot, base, **scaling), interleaved, amplitude, device)

    @classmethod
    def from_frequencies(cls, freqs, interleaved=False, amplitude=1.0, device=None):
        """freqs: a float64 tensor, or numbers; the table goes to its device, or to `device`."""
        self = cls.__new__(cls)
        if isinstance(freqs, torch.Tensor):
            device = freqs.device if device is None else device
            freqs = freqs.tolist()
        self._set(freqs, interleaved, amplitude, "cuda" if device is None else device)
        return self

    def _set(self, freqs, interleaved, amplitude, device):
        self.rot, self.interleaved, self.amplitude = 2 * len(freqs), bool(interleaved), float(amplitude)
        self.turns = torch.tensor([_turns(float(f)) for f in freqs], dtype=torch.int64, device=device)
        self.dev = self.turns.get_device()  # -1 on the CPU
        self.c = _c.rope(self.turns, self.rot, self.interleaved, self.amplitude)

    def __call__(self, x, positions, out=None, inverse=False, stream=None):
        """x [N, H, d] bf16 or fp32 turned by positions [N] int32 into `out` (x itself is allowed; a new tensor where it
        is None).  Heads are contiguous, rows may lie apart, as slices of a wider projection.  With `inverse` turned
        back: the gradient of x from that of the result."""
        dev, dtype, shape = _device(self.turns), x.dtype, x.shape
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise ValueError("x has to be bfloat16 or float32")
        if len(shape) != 3:
            raise ValueError("x has shape %s, expected [N, H, d]" % (tuple(shape),))
        N, H, d = shape
        x_stride = _check_rows("x", x, dtype, shape, dev)
        _check_tensor("positions", positions, torch.int32, (N,), dev)
        if out is None:
            out, stride = _new(x, shape, dtype, stream), H * d
        else:
            stride = _check_rows("out", out, dtype, shape, dev)
        if N:
            _c.msa_rope(x, x_stride, out, stride, N, H, d, dtype is torch.float32, positions, self.c, inverse, stream=stream)
        return out


def _turns(f):
    """f radians a position as 2^-64 turns: f / (2 pi) 2^64 rounded, modulo 2^64, as a signed integer."""
    if not math.isfinite(f):
        raise ValueError("a frequency is not finite")
    n, d = f.as_integer_ratio()
    # pi 2^132 as an integer: f / (2 pi) 2^64 = n 2^(63 + 132) / (d pi 2^132)
    pi = 0x3243F6A8885A308D313198A2E03707344A
    num, den = n << (63 + 132), d * pi
    t = (2 * num + den) // (2 * den) % (1 << 64)
    return t - (1 << 64) if t >= 1 << 63 else t


def _check_rows(name, t, dtype, shape, dev):
    """t [N, ...] of the type and shape, on device number dev; each row contiguous, rows apart by any stride that holds one.
    Returns the elements from row to row."""
    row = math.prod(shape[1:])
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return row
    if t.dtype != dtype or t.get_device() < 0:
        raise ValueError("%s must be a CUDA %s tensor" % (name, str(dtype).replace("torch.", "")))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the object on cuda:%d" % (name, t.get_device(), dev))
    step = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != step:
            raise ValueError("%s: the rows themselves must be contiguous" % name)
        step *= n
    if t.shape[0] < 2:
        return row
    if t.stride(0) < row:
        raise ValueError("%s: rows must not overlap" % name)
    return t.stride(0)


def _new(like, shape, dtype, stream):
    """An uninitialized contiguous tensor on like's device, from the memory of `stream` (see _allocating_for)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _allocating_for(stream):
        return like.new_empty(shape, dtype=dtype)


class _Append:
    """What KvPool and Kv4Pool share: new rows on their way into the pool."""

    def append(self, k, v, cu_seqlens, pos0, page_table, rope=None, positions=None, q=None, k_idx=None, k_idx_pool=None,
               q_idx=None, idx_rope=None, idx_scale=1.0, q_out=None, q_idx_out=None, stream=None):
        """Stores packed rows k (turned by `rope`) and v [N, H_kv, d] at the places of their tokens (cu_seqlens, pos0 and
        page_table as in Kv4Pool.store), index keys k_idx [N, d_I] in k_idx_pool [n_pages, page_size, d_I] (bf16, or
        uint8: E4M3 codes of idx_scale times the rows), and returns (q, q_idx) turned, None for what was not given.

        The index rows are turned by idx_rope (`rope` where it is None).  positions [N] int32: what rows are turned by
        where it is not their place in the cache.  Rows of the inputs may lie apart, as slices of a wider projection.
        See msa_append_paged."""
        N, S, dev = k.shape[0], cu_seqlens.shape[0] - 1, _device(self.workspace)
        shape, bf16 = (N, self.H_kv, self.d), torch.bfloat16
        k_stride, v_stride = _check_rows("k", k, bf16, shape, dev), _check_rows("v", v, bf16, shape, dev)
        max_pages = page_table.shape[-1]
        _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (S + 1,), dev)
        _check_tensor("pos0", pos0, torch.int32, (S,), dev)
        _check_tensor("page_table", page_table, torch.int32, (S, max_pages), dev)
        if positions is not None:
            _check_tensor("positions", positions, torch.int32, (N,), dev)
        for name, r in (("rope", rope), ("idx_rope", idx_rope)):
            if r is not None and r.dev != dev:
                raise ValueError("%s is on device %d, the object on cuda:%d" % (name, r.dev, dev))
        f8, q_stride, H_q, d_I, q_idx_stride, k_idx_stride = False, 0, 0, 0, 0, 0
        if q is not None:
            if q.dim() != 3 or q.shape[2] != self.d:
                raise ValueError("q has shape %s, expected [N, H_q, %d]" % (tuple(q.shape), self.d))
            H_q = q.shape[1]
            q_stride = _check_rows("q", q, bf16, (N, H_q, self.d), dev)
            if q_out is None:
                q_out = _new(q, q.shape, bf16, stream)
            else:
                _check_tensor("q_out", q_out, bf16, q.shape, dev)
        if k_idx is not None:
            if k_idx_pool is None:
                raise ValueError("k_idx needs k_idx_pool")
            f8, d_I = k_idx_pool.dtype is torch.uint8, k_idx.shape[-1]
            k_idx_stride = _check_rows("k_idx", k_idx, bf16, (N, d_I), dev)
            _check_tensor("k_idx_pool", k_idx_pool, torch.uint8 if f8 else bf16, (self.n_pages, self.page_size, d_I), dev)
        elif k_idx_pool is not None:
            raise ValueError("k_idx_pool needs k_idx")
        elif q_idx_out is not None:
            f8 = q_idx_out.dtype is torch.uint8
        if q_idx is not None:
            if k_idx is not None and d_I != q_idx.shape[-1]:
                raise ValueError("q_idx and k_idx differ in d_I")
            d_I, held = q_idx.shape[-1], torch.uint8 if f8 else bf16
            q_idx_stride = _check_rows("q_idx", q_idx, bf16, (N, self.H_kv, d_I), dev)
            if q_idx_out is None:
                q_idx_out = _new(q_idx, q_idx.shape, held, stream)
            else:
                _check_tensor("q_idx_out", q_idx_out, held, q_idx.shape, dev)
        if N:
            at = _c._ptr
            has_q, has_qi = q is not None, q_idx is not None
            rows = _c.msa_append_t(at(q), at(k), at(v), at(q_idx), at(k_idx), q_stride, k_stride, v_stride, q_idx_stride, k_idx_stride,
                                   at(q_out) if has_q else None, at(q_idx_out) if has_qi else None, at(k_idx_pool), at(positions), H_q,
                                   d_I, f8, idx_scale)
            idx_rope = None if k_idx is None and q_idx is None else rope if idx_rope is None else idx_rope
            self._append(rows, N, cu_seqlens, S, pos0, page_table, max_pages, self.c, None if rope is None else rope.c,
                         None if idx_rope is None else idx_rope.c, self.workspace, stream=stream)
        return q_out if q is not None else None, q_idx_out if q_idx is not None else None


class KvPool(_Append):
    """A bf16 paged K/V cache: k and v [n_pages, page_size, H_kv, d].  ``KvPool.empty`` makes one.

    What msa_decode_paged reads and MsaTreeDecode attends to.  Calls on other streams may touch other rows at the same
    time; the error word that ``device_status`` reads is one for all of them, that of the call that ran last."""

    _append = staticmethod(_c.msa_append_paged)

    def __init__(self, k, v):
        self.n_pages, self.page_size, self.H_kv, self.d = k.shape
        for name, t in (("k", k), ("v", v)):
            _check_tensor(name, t, torch.bfloat16, tuple(k.shape), k.get_device())
        self.k, self.v = k, v
        self.c = _c.kv_pool(k, v, self.n_pages, self.page_size, self.H_kv, self.d)
        self.workspace = torch.empty(_c.msa_append_workspace(), dtype=torch.uint8, device=k.device)

    @classmethod
    def empty(cls, n_pages, page_size, H_kv, d, device="cuda"):
        return cls(*_settled([torch.zeros((n_pages, page_size, H_kv, d), dtype=torch.bfloat16, device=device) for _ in range(2)]))

    def tensors(self):
        return [self.k, self.v]

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class Kv4Pool(_Append):
    """A 4-bit paged K/V cache: codes [n_pages, page_size, H_kv, d / 2] and scales [n_pages, page_size, H_kv, 4]
    of K and of V (uint8).  ``Kv4Pool.empty`` makes one.  ``append`` is ``store`` with the rotation on the way.

    Calls on other streams may touch other rows at the same time; the error word that ``device_status`` reads is one
    for all of them, that of the call that ran last."""

    _append = staticmethod(_c.msa_append_paged_kv4)

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        self.n_pages, self.page_size, self.H_kv, half = k_codes.shape
        self.d = 2 * half
        for name, t, last in (("k_codes", k_codes, half), ("k_scales", k_scales, 4), ("v_codes", v_codes, half),
                              ("v_scales", v_scales, 4)):
            _check_tensor(name, t, torch.uint8, (self.n_pages, self.page_size, self.H_kv, last), k_codes.get_device())
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.c = _c.kv4_pool(k_codes, k_scales, v_codes, v_scales, self.n_pages, self.page_size, self.H_kv, self.d)
        self.workspace = torch.empty(_c.msa_kv4_workspace(), dtype=torch.uint8, device=k_codes.device)

    @classmethod
    def empty(cls, n_pages, page_size, H_kv, d, device="cuda"):
        return cls(*_settled([torch.zeros((n_pages, page_size, H_kv, last), dtype=torch.uint8, device=device)
                              for last in (d // 2, 4, d // 2, 4)]))

    def tensors(self):
        return [self.k_codes, self.k_scales, self.v_codes, self.v_scales]

    def _rows(self, k, v, shape, cu_seqlens, pos0, page_table):
        S, dev = cu_seqlens.numel() - 1, _device(self.workspace)
        _check_tensor("k", k, torch.bfloat16, shape, dev)
        _check_tensor("v", v, torch.bfloat16, shape, dev)
        _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (S + 1,), dev)
        _check_tensor("pos0", pos0, torch.int32, (S,), dev)
        _check_tensor("page_table", page_table, torch.int32, (S, page_table.shape[-1]), dev)
        return S, page_table.shape[1]

    def store(self, k, v, cu_seqlens, pos0, page_table, stream=None):
        """Quantizes rows k, v [N, H_kv, d] into the pages of their sequences (see msa_kv4_store)."""
        N = k.shape[0]
        S, max_pages = self._rows(k, v, (N, self.H_kv, self.d), cu_seqlens, pos0, page_table)
        _c.msa_kv4_store(k, v, N, cu_seqlens, S, pos0, page_table, max_pages, self.c, self.workspace, stream=stream)

    def load(self, N, cu_seqlens, pos0, page_table, k=None, v=None, stream=None):
        """The rows' values as bf16 [N, H_kv, d] (see msa_kv4_load); rows of no sequence stay as k and v had them."""
        shape = (N, self.H_kv, self.d)
        if k is None or v is None:
            with _allocating_for(stream):
                k = torch.empty(shape, dtype=torch.bfloat16, device=self.k_codes.device) if k is None else k
                v = torch.empty(shape, dtype=torch.bfloat16, device=self.k_codes.device) if v is None else v
        S, max_pages = self._rows(k, v, shape, cu_seqlens, pos0, page_table)
        _c.msa_kv4_load(self.c, N, cu_seqlens, S, pos0, page_table, max_pages, k, v, self.workspace, stream=stream)
        return k, v

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class MsaDecodeKv4:
    """One decode token for B sequences over a Kv4Pool: ``dense`` attends to the whole context, calling the
    object runs the MSA step (select by the index branch, attend to the chosen blocks; needs d_I, Bk and k).

    The tensors that a call returns are the object's own: the next call of the same operator overwrites them, one
    of the other operator does not.  ``out`` and ``lse`` are those of the last call.  Both use one workspace, so two
    calls in flight at once need two objects."""

    def __init__(self, pool: Kv4Pool, B, max_pages, H_q, d_I=None, Bk=128, k=16, device=None):
        at = pool.k_codes.get_device()
        if device is not None and (torch.device(device).type != "cuda" or torch.device(device).index not in (None, at)):
            raise ValueError("the pool is on cuda:%d" % at)
        device = pool.k_codes.device  # ("cuda" alone would be the current one)
        self.pool, self.B, self.max_pages, self.H_q, self.d_I = pool, B, max_pages, H_q, d_I
        need = _c.msa_dense_decode_paged_kv4_workspace(B, H_q, pool.H_kv, pool.d)
        if d_I is not None:
            self.shape = _c.shape(max_pages * pool.page_size, H_q, pool.H_kv, pool.d, d_I, Bk, k)
            need = max(need, _c.msa_decode_workspace(B, self.shape))
            self.block_idx = torch.empty((B, pool.H_kv, k), dtype=torch.int32, device=device)
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self._dense, self._step = [(torch.empty((B, H_q, pool.d), dtype=torch.bfloat16, device=device),
                                    torch.empty((B, H_q), dtype=torch.float32, device=device))
                                   if wanted else None for wanted in (True, d_I is not None)]
        self.out, self.lse = self._step or self._dense

    def _check(self, q_t, page_table, ctx_len):
        dev = _device(self.workspace)
        _check_tensor("q_t", q_t, torch.bfloat16, (self.B, self.H_q, self.pool.d), dev)
        _check_tensor("page_table", page_table, torch.int32, (self.B, self.max_pages), dev)
        _check_tensor("ctx_len", ctx_len, torch.int32, (self.B,), dev)
        return dev

    def dense(self, q_t, page_table, ctx_len, scale=None, stream=None):
        self._check(q_t, page_table, ctx_len)
        scale = 1.0 / math.sqrt(self.pool.d) if scale is None else scale
        out, lse = self._dense
        _c.msa_dense_decode_paged_kv4(q_t, self.pool.c, page_table, self.max_pages, ctx_len, self.B, self.H_q, scale,
                                      out, lse, self.workspace, stream=stream)
        self.out, self.lse = out, lse
        return out, lse

    def __call__(self, q_t, q_idx_t, k_idx_pool, page_table, ctx_len, scale=None, stream=None):
        """q_idx_t [B, H_kv, d_I] and k_idx_pool [n_pages, page_size, d_I]: both bf16, or both uint8 (E4M3 codes)."""
        if self.d_I is None:
            raise ValueError("the MSA step needs d_I (and Bk, k) when the object is made")
        dev = self._check(q_t, page_table, ctx_len)
        f8 = q_idx_t.dtype == torch.uint8
        idx = torch.uint8 if f8 else torch.bfloat16
        _check_tensor("q_idx_t", q_idx_t, idx, (self.B, self.pool.H_kv, self.d_I), dev)
        _check_tensor("k_idx_pool", k_idx_pool, idx, (self.pool.n_pages, self.pool.page_size, self.d_I), dev)
        scale = 1.0 / math.sqrt(self.pool.d) if scale is None else scale
        call = _c.msa_decode_paged_kv4_fp8 if f8 else _c.msa_decode_paged_kv4
        out, lse = self._step
        call(q_t, q_idx_t, k_idx_pool, self.pool.c, page_table, self.max_pages, ctx_len, self.B, self.shape, scale,
             out, lse, self.block_idx, self.workspace, stream=stream)
        self.out, self.lse = out, lse
        return out, lse, self.block_idx

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class MsaTreeDecode:
    """Dense attention of trees of up to T drafted tokens, one for each of B sequences, over a KvPool or a Kv4Pool.

    (T = 1 is a dense decode step.)  A call returns the object's own ``out`` [B, T, H_q, d] and ``lse`` [B, T, H_q], which
    the next call overwrites, nodes past a tree's length left as they were; two calls in flight at once need two objects."""

    def __init__(self, pool, B, T, max_pages, H_q):
        device = pool.tensors()[0].device
        self.pool, self.B, self.T, self.max_pages, self.H_q = pool, B, T, max_pages, H_q
        self.workspace = torch.empty(_c.msa_tree_decode_workspace(B, T, H_q, pool.H_kv, pool.d), dtype=torch.uint8, device=device)
        self.out, self.lse = _settled([torch.zeros((B, T, H_q, pool.d), dtype=torch.bfloat16, device=device),
                                       torch.zeros((B, T, H_q), dtype=torch.float32, device=device)])
        self._call = _c.msa_tree_decode_paged_kv4 if isinstance(pool, Kv4Pool) else _c.msa_tree_decode_paged

    def __call__(self, q, page_table, ctx_len, parents, tree_len=None, scale=None, stream=None):
        """q [B, T, H_q, d]; parents [B, T] int32 (-1: a root); ctx_len [B]: tokens before the tree, whose node j is token
        ctx_len + j of the cache; tree_len [B]: nodes of each tree (T each where None)."""
        dev = _device(self.workspace)
        _check_tensor("q", q, torch.bfloat16, (self.B, self.T, self.H_q, self.pool.d), dev)
        _check_tensor("page_table", page_table, torch.int32, (self.B, self.max_pages), dev)
        _check_tensor("ctx_len", ctx_len, torch.int32, (self.B,), dev)
        _check_tensor("parents", parents, torch.int32, (self.B, self.T), dev)
        if tree_len is not None:
            _check_tensor("tree_len", tree_len, torch.int32, (self.B,), dev)
        scale = 1.0 / math.sqrt(self.pool.d) if scale is None else scale
        self._call(q, self.pool.c, page_table, self.max_pages, ctx_len, tree_len, parents, self.B, self.T, self.H_q, scale,
                   self.out, self.lse, self.workspace, stream=stream)
        return self.out, self.lse

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class DraftVerifier:
    """Verification of trees of up to T nodes, one for each of B sequences, over a vocabulary of V tokens.

    A call returns the object's own ``path`` [B, T] (accepted nodes, node 0 first, then -1), ``n_path`` [B] and
    ``next_token`` [B], int32, which the next call overwrites; PagedCache.accept takes them as they are."""

    def __init__(self, B, T, V, device="cuda"):
        self.B, self.T, self.V = B, T, V
        self.workspace = torch.empty(_c.msa_verify_workspace(), dtype=torch.uint8, device=device)
        self.path = torch.empty((B, T), dtype=torch.int32, device=device)
        self.n_path = torch.empty((B,), dtype=torch.int32, device=device)
        self.next_token = torch.empty((B,), dtype=torch.int32, device=device)

    def __call__(self, probs, tokens, parents, u, u_last, draft_probs=None, tree_len=None, stream=None):
        """probs, draft_probs [B, T, V] fp32: the target's distribution after each node, and that which its children were
        drawn from (None: the drafts were certain); u [B, T] and u_last [B] fp32 random numbers in [0, 1)."""
        dev = _device(self.workspace)
        _check_tensor("probs", probs, torch.float32, (self.B, self.T, self.V), dev)
        _check_tensor("tokens", tokens, torch.int32, (self.B, self.T), dev)
        _check_tensor("parents", parents, torch.int32, (self.B, self.T), dev)
        _check_tensor("u", u, torch.float32, (self.B, self.T), dev)
        _check_tensor("u_last", u_last, torch.float32, (self.B,), dev)
        if draft_probs is not None:
            _check_tensor("draft_probs", draft_probs, torch.float32, (self.B, self.T, self.V), dev)
        if tree_len is not None:
            _check_tensor("tree_len", tree_len, torch.int32, (self.B,), dev)
        _c.msa_verify_tree(probs, draft_probs, tokens, parents, tree_len, u, u_last, self.B, self.T, self.V, self.path,
                           self.n_path, self.next_token, self.workspace, stream=stream)
        return self.path, self.n_path, self.next_token

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


class PagedCache:
    """Page tables, lengths and reference counts of a paged cache, and the pools that they address.

    page_table [n_seqs, max_pages], ctx_len [n_seqs] and refs [n_pages] are int32 device tensors; every pool is a
    contiguous tensor of n_pages pages, at most 8 of them.  ``PagedCache.empty`` makes the tables.  A call's
    errors (MSA_ERR_NO_PAGES, MSA_ERR_BAD_INDEX) are what ``device_status`` returns after it.  Calls follow one
    another on the device: calls on other streams have to be ordered by the caller."""

    def __init__(self, page_table, ctx_len, refs, page_size, pools=()):
        n_seqs, max_pages = page_table.shape
        n_pages = refs.numel()
        dev = page_table.get_device()
        _check_tensor("page_table", page_table, torch.int32, (n_seqs, max_pages), dev)
        _check_tensor("ctx_len", ctx_len, torch.int32, (n_seqs,), dev)
        _check_tensor("refs", refs, torch.int32, (n_pages,), dev)
        for i, t in enumerate(pools):
            _check_tensor("pools[%d]" % i, t, t.dtype, (n_pages, page_size) + tuple(t.shape[2:]), dev)
        self.page_table, self.ctx_len, self.refs, self.page_size = page_table, ctx_len, refs, page_size
        self.pools, self.n_pages = list(pools), n_pages
        self.c = _c.pages(page_table, ctx_len, refs, max_pages, n_pages, n_seqs, page_size)
        self.c_pools = _c.page_pools((t, t.numel() // n_pages * t.element_size()) for t in self.pools)
        self.page_map = torch.empty((n_pages,), dtype=torch.int32, device=refs.device)
        self.n_live = torch.empty((1,), dtype=torch.int32, device=refs.device)
        need = max(_c.msa_pages_workspace(self.c, 0), _c.msa_pages_workspace(self.c, 4096),  # compact, the most entries
                   _c.msa_pages_accept_workspace(self.c, 4096, 64))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=refs.device)

    @classmethod
    def empty(cls, n_seqs, max_pages, n_pages, page_size, pools=(), device="cuda"):
        return cls(*_settled([torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device),
                              torch.zeros((n_seqs,), dtype=torch.int32, device=device),
                              torch.zeros((n_pages,), dtype=torch.int32, device=device)]), page_size, pools)

    def reserve(self, seqs, new_len, stream=None):
        n, dev = seqs.numel(), _device(self.workspace)
        _check_tensor("seqs", seqs, torch.int32, (n,), dev)
        _check_tensor("new_len", new_len, torch.int32, (n,), dev)
        _c.msa_pages_reserve(self.c, seqs, new_len, n, self.workspace, stream=stream)

    def fork(self, src, dst, stream=None):
        n, dev = src.numel(), _device(self.workspace)
        _check_tensor("src", src, torch.int32, (n,), dev)
        _check_tensor("dst", dst, torch.int32, (n,), dev)
        _c.msa_pages_fork(self.c, src, dst, n, self.c_pools, len(self.pools), self.workspace, stream=stream)

    def free(self, seqs, stream=None):
        n, dev = seqs.numel(), _device(self.workspace)
        _check_tensor("seqs", seqs, torch.int32, (n,), dev)
        _c.msa_pages_free(self.c, seqs, n, self.workspace, stream=stream)

    def accept(self, seqs, base_len, path, n_path, stream=None):
        """Of sequence seqs[i]'s tokens from base_len[i] on, those at base_len[i] + path[i][: n_path[i]] stay, in their
        order, and the sequence ends after them (path [n, T] and n_path [n] as DraftVerifier returns them; n_path 0 cuts
        the sequence off at base_len)."""
        n, dev = seqs.numel(), _device(self.workspace)
        _check_tensor("seqs", seqs, torch.int32, (n,), dev)
        _check_tensor("base_len", base_len, torch.int32, (n,), dev)
        _check_tensor("path", path, torch.int32, (n, path.shape[-1]), dev)
        _check_tensor("n_path", n_path, torch.int32, (n,), dev)
        _c.msa_pages_accept(self.c, seqs, base_len, path, n_path, n, path.shape[1], self.c_pools, len(self.pools),
                            self.workspace, stream=stream)

    def compact(self, stream=None):
        """Returns (page_map [n_pages], n_live [1]): each page's new id (-1 where it was free), and the pages held.
        Both are the object's own; the next compact overwrites them."""
        _device(self.workspace)
        _c.msa_pages_compact(self.c, self.c_pools, len(self.pools), self.page_map, self.n_live, self.workspace,
                             stream=stream)
        return self.page_map, self.n_live

    def device_status(self, stream=None):
        return _c.msa_check_device_error(self.workspace, stream)


def prefill(q, k, v, q_idx, k_idx, Bk=128, k_blocks=16, scale=None):
    """One-shot prefill: returns (out [N,H_q,d] bf16, lse [H_q,N] fp32, block_idx [G,N,k] int32)."""
    N, H_q, d = q.shape
    H_kv = k.shape[1]
    run = MsaPrefill(N, H_q, H_kv, d, q_idx.shape[2], Bk, k_blocks, device=q.device)
    out, lse, blk = run(q, k, v, q_idx, k_idx, scale)
    return out, lse, blk


def decode(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, Bk=128, k_blocks=16, scale=None):
    """One-shot decode step: returns (out [B,H_q,d], lse [B,H_q], block_idx [B,G,k])."""
    B, H_q, d = q_t.shape
    _, ctx_max, H_kv, _ = k_cache.shape
    run = MsaDecode(B, ctx_max, H_q, H_kv, d, q_idx_t.shape[2], Bk, k_blocks, device=q_t.device)
    return run(q_t, q_idx_t, k_idx_cache, k_cache, v_cache, ctx_len, scale)


def varlen_cells(lengths, Bk):
    """Block-aligned cell offsets for sequences of the given lengths: cu_seqlens [S+1] (a list of ints)
    for msa_select_blocks_varlen / msa_prefill_varlen, sequence s starting at the first block boundary
    after sequence s-1's last token; N = cu_seqlens[-1] cells hold them all."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + (int(n) + Bk - 1) // Bk * Bk)
    return cu


def prefill_from_host(run: MsaPrefill, host_inputs, dev_inputs, host_out, stream=None):
    """End-to-end step through the public API with host buffers: pinned host -> device copies,
    the prefill step, device -> pinned host copies of out and lse, all on one stream."""
    for name in ("q", "k", "v", "q_idx", "k_idx"):
        dev_inputs[name].copy_(host_inputs[name], non_blocking=True)
    out, lse, blk = run(dev_inputs["q"], dev_inputs["k"], dev_inputs["v"], dev_inputs["q_idx"], dev_inputs["k_idx"],
                        stream=stream)
    host_out["out"].copy_(out, non_blocking=True)
    host_out["lse"].copy_(lse, non_blocking=True)
    return host_out


class PrefillHostPipeline:
    """Prefill steps from pinned host buffers to pinned host buffers, with the copies overlapped.

    Copies run on two host->device and two device->host streams (each direction
    then keeps two copy engines busy, which on this GPU's host link roughly
    doubles what one stream moves while the other direction is busy too), and
    the prefill on the compute stream.  Step i's inputs land in one of two
    device input sets while step i-1 computes on the other; its index inputs
    (q_idx, k_idx) are copied first so that the select can start while q, k and
    v are still in flight.  Step i's out and lse go to one of two device output
    sets and are copied back while step i+1 computes into the other, so the
    compute stream never waits for a device->host copy of the step before.
    Every step still copies all of its inputs in and all of its outputs (out,
    lse) out."""

    NAMES = ("q_idx", "k_idx", "q", "k", "v")

    def __init__(self, run: MsaPrefill, device="cuda"):
        self.run = run
        self.dev = [{n: torch.empty(_input_shape(run, n), dtype=torch.bfloat16, device=device) for n in self.NAMES}
                    for _ in range(2)]
        self.outs = [(run.out, run.lse), (torch.empty_like(run.out), torch.empty_like(run.lse))]
        self.h2d = [torch.cuda.Stream(device=device) for _ in range(2)]
        self.d2h = [torch.cuda.Stream(device=device) for _ in range(2)]

    def __call__(self, host_inputs, host_outputs, stream=None):
        """host_inputs: list of dicts of pinned bf16 tensors (q, k, v, q_idx, k_idx), one per step;
        host_outputs: list of dicts of pinned tensors (out, lse), one per step.  Returns once the
        work is queued; it is ordered before later work on `stream` (default: the current stream)."""
        comp = torch.cuda.current_stream() if stream is None else stream
        E = torch.cuda.Event
        for st in self.h2d + self.d2h:
            st.wait_stream(comp)
        half = self.run.N // 2
        attn_done, d2h_done = {}, {}
        for i, (hin, hout) in enumerate(zip(host_inputs, host_outputs)):
            dev = self.dev[i % 2]
            idx_in, qkv_in = E(), [E(), E()]
            for j, st in enumerate(self.h2d):
                with torch.cuda.stream(st):
                    if i - 2 in attn_done:  # the attention of step i-2 has finished reading this input set
                        st.wait_event(attn_done[i - 2])
                    if j == 0:
                        for n in ("q_idx", "k_idx"):
                            dev[n].copy_(hin[n], non_blocking=True)
                        idx_in.record(st)
                        dev["q"][:half].copy_(hin["q"][:half], non_blocking=True)
                        dev["k"].copy_(hin["k"], non_blocking=True)
                    else:
                        dev["q"][half:].copy_(hin["q"][half:], non_blocking=True)
                        dev["v"].copy_(hin["v"], non_blocking=True)
                    qkv_in[j].record(st)
            comp.wait_event(idx_in)
            self.run.select(dev["q_idx"], dev["k_idx"], stream=comp)
            for ev in qkv_in:
                comp.wait_event(ev)
            for ev in d2h_done.get(i - 2, ()):  # out and lse of step i-2 (this output set) are on the host
                comp.wait_event(ev)
            out, lse = self.outs[i % 2]
            self.run.attend(dev["q"], dev["k"], dev["v"], stream=comp, out=out, lse=lse)
            attn_done[i] = E()
            attn_done[i].record(comp)
            d2h_done[i] = []
            for j, st in enumerate(self.d2h):
                with torch.cuda.stream(st):
                    st.wait_event(attn_done[i])
                    if j == 0:
                        hout["out"][:half].copy_(out[:half], non_blocking=True)
                        hout["lse"].copy_(lse, non_blocking=True)
                    else:
                        hout["out"][half:].copy_(out[half:], non_blocking=True)
                    ev = E()
                    ev.record(st)
                    d2h_done[i].append(ev)
        for st in self.h2d + self.d2h:
            comp.wait_stream(st)
        return host_outputs


def _input_shape(run: MsaPrefill, name):
    return {"q": (run.N, run.H_q, run.d), "k": (run.N, run.H_kv, run.d), "v": (run.N, run.H_kv, run.d),
            "q_idx": (run.N, run.G, run.d_I), "k_idx": (run.N, run.d_I)}[name]
