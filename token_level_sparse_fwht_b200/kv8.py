"""Caches held in 8 bits (e4m3 or int8 with a float32 scale per block of positions and kv
head): append, read, dense and sparse attention, eviction by accumulated attention weight.

Like the rest of the package this only marshals torch tensors into the C ABI of
include/adamas.h (adamas_kv8_*, adamas_evict_select, adamas_compact_rows).  Calls run on
the device of the cache's tensors, on `stream` (default: that device's current stream);
tensors made here (outputs, workspaces) belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from token_level_sparse_fwht_b200 import (ERR_INVALID_ARG, HEAD_DIM, OK, AdamasError, lib, _c_f,
                                          _c_i, _c_i64, _c_p, _c_sz, _dev, _dtype_code)

_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}


class _CCache(ctypes.Structure):
    """adamas_kv8_cache."""
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_scale", _c_p), ("v_scale", _c_p), ("codes", _c_p),
                ("block_table", _c_p), ("Lmax", _c_i64), ("num_pages", _c_i64),
                ("format", ctypes.c_int32), ("block_size", ctypes.c_int32), ("B", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _typed(t, name, dtype, shape=None):
    """Device pointer of a contiguous CUDA tensor of this type (and shape)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return _dev(t, name)


class KV8Cache:
    """The tensors of an 8-bit cache.

    Contiguous: k, v [B,Hkv,Lmax,128] (torch.float8_e4m3fn or torch.int8), k_scale, v_scale
    [B,Hkv,Lmax/block_size] float32, codes (optional) [B,Hkv,Lmax,32] uint8.  Paged, with
    block_table [B,max_blocks] int32: k, v [P,Hkv,page,128], scales
    [P,Hkv,page/block_size], codes [P,Hkv,page,32]; max_seq_len (default: what the table
    holds) bounds every sequence."""

    def __init__(self, k, v, k_scale, v_scale, block_size: int, codes=None, block_table=None,
                 max_seq_len: int | None = None):
        if k.dtype not in _FORMATS:
            raise TypeError(f"unsupported cache dtype {k.dtype} (float8_e4m3fn or int8)")
        if k.dim() != 4 or k.shape[-1] != HEAD_DIM:
            raise ValueError(f"k must be [B, Hkv, Lmax, {HEAD_DIM}] or [P, Hkv, page, {HEAD_DIM}]")
        if block_size < 1 or k.shape[2] % block_size:
            raise ValueError("rows per unit or page must be a multiple of block_size")
        P, Hkv, rows, d = k.shape
        c = _CCache()
        c.k = _typed(k, "k", k.dtype)
        c.v = _typed(v, "v", k.dtype, k.shape)
        sc = (P, Hkv, rows // block_size)
        c.k_scale = _typed(k_scale, "k_scale", torch.float32, sc)
        c.v_scale = _typed(v_scale, "v_scale", torch.float32, sc)
        if codes is not None:
            c.codes = _typed(codes, "codes", torch.uint8, (P, Hkv, rows, d // 4))
        if block_table is None:
            self.B, self.Lmax = P, rows
            if max_seq_len is not None and max_seq_len != rows:
                raise ValueError("a contiguous cache's max_seq_len is its Lmax")
        else:
            if block_table.dim() != 2:
                raise ValueError("block_table must be [B, max_blocks]")
            c.block_table = _typed(block_table, "block_table", torch.int32)
            self.B, c.max_blocks_per_seq = block_table.shape
            self.Lmax = c.max_blocks_per_seq * rows if max_seq_len is None else int(max_seq_len)
            c.page_size, c.num_pages = rows, P
        self.Hkv, self.block_size = Hkv, block_size
        c.Lmax, c.format, c.block_size = self.Lmax, _FORMATS[k.dtype], block_size
        c.B, c.Hkv, c.d = self.B, Hkv, d
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.codes, self.block_table = codes, block_table
        self.device = k.device
        for t in (v, k_scale, v_scale, codes, block_table):
            if t is not None and t.device != self.device:
                raise ValueError("the cache's tensors must be on one device")
        self._c = c

    @property
    def ptr(self):
        return ctypes.byref(self._c)


def kv8_cache(B: int, Hkv: int, Lmax: int, block_size: int = 64, dtype=torch.float8_e4m3fn,
              codes: bool = False, device="cuda") -> KV8Cache:
    """An empty contiguous cache (zero rows; Lmax is rounded up to whole blocks)."""
    rows = -(-Lmax // block_size) * block_size
    byte = torch.zeros((2, B, Hkv, rows, HEAD_DIM), dtype=torch.uint8, device=device).view(dtype)
    scale = torch.zeros((2, B, Hkv, rows // block_size), dtype=torch.float32, device=device)
    c = torch.zeros((B, Hkv, rows, HEAD_DIM // 4), dtype=torch.uint8, device=device) if codes else None
    return KV8Cache(byte[0], byte[1], scale[0], scale[1], block_size, codes=c)


# ------------------------------------------------------------------ calls
class _Call:
    """One C call bound to its buffers: name, arguments, the device it runs on."""

    def __init__(self, name, args, keep, device):
        self._name, self._args, self._keep, self._device = name, args, keep, device
        self._fn = getattr(lib(), name)

    def __call__(self):
        # launches go to the current device, which need not be the tensors' own
        if torch.cuda.current_device() == self._device:
            status = self._fn(*self._args)
        else:
            with torch.cuda.device(self._device):
                status = self._fn(*self._args)
        if status != OK:
            raise AdamasError(status, self._name)


def _where(device, stream):
    """(device index, stream handle) of a call on tensors of `device`."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    if stream is None:
        stream = torch.cuda.current_stream(index)
    return index, int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


@contextlib.contextmanager
def _owner(device, stream):
    """Tensors made inside belong to the call's device and stream."""
    index, handle = _where(device, stream)
    with contextlib.ExitStack() as stack:
        if torch.cuda.current_device() != index:
            stack.enter_context(torch.cuda.device(index))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(handle, index)
            stack.enter_context(torch.cuda.stream(stream))
        yield


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _ws(ws, device):
    _same_device(device, workspace=ws)
    if ws.dtype != torch.uint8:
        raise TypeError("workspace must be uint8")
    return _c_p(_dev(ws, "workspace")), _c_sz(ws.numel())


def _new_workspace(n, name, device, stream):
    if n == 0:
        raise AdamasError(ERR_INVALID_ARG, name)
    device = torch.device(device)
    with _owner(device, stream):
        return torch.zeros(int(n), dtype=torch.uint8, device=device)


def kv8_workspace(device="cuda", stream=None):
    """A workspace of the calls that only need an error word (append, read, evict)."""
    return _new_workspace(256, "kv8_workspace", device, stream)


def kv8_attention_workspace(B: int, Hq: int, Hkv: int, Lmax: int, weights: bool = False,
                            device="cuda", stream=None):
    """A zero-filled workspace of kv8_attention (and of the calls above)."""
    with torch.cuda.device(torch.device(device)):
        n = lib().adamas_kv8_attention_workspace_bytes(B, Hq, Hkv, HEAD_DIM, Lmax,
                                                       int(bool(weights)))
    return _new_workspace(n, "adamas_kv8_attention_workspace_bytes", device, stream)


def kv8_sparse_attention_workspace(B: int, Hq: int, Hkv: int, k: int, shared: bool = False,
                                   weights: bool = False, device="cuda", stream=None):
    """A zero-filled workspace of kv8_sparse_attention for lists of k positions."""
    with torch.cuda.device(torch.device(device)):
        n = lib().adamas_kv8_sparse_attention_workspace_bytes(
            B, Hq, Hkv, HEAD_DIM, k, int(bool(shared)), int(bool(weights)))
    return _new_workspace(n, "adamas_kv8_sparse_attention_workspace_bytes", device, stream)


def _lens(cache, t, name):
    return _c_p(_typed(t, name, torch.int32, (cache.B,)))


# --------------------------------------------------------------- append, read
class PreparedKV8Append(_Call):
    """kv8_append bound to fixed buffers (a serving loop refills them between calls)."""

    def __init__(self, cache: KV8Cache, k_new, v_new, starts, ws, counts=None, t=None, ratio=None,
                 stream=None):
        B, Hkv, n, d = k_new.shape
        if (B, Hkv, d) != (cache.B, cache.Hkv, HEAD_DIM):
            raise ValueError("k_new must be [B, Hkv, n, 128] of the cache's B and Hkv")
        # a dimension of one element may have any stride: it is never stepped
        sb, sh, sn, sd = (0 if w == 1 else x for w, x in zip(k_new.shape, k_new.stride()))
        v_strides = tuple(0 if w == 1 else x for w, x in zip(v_new.shape, v_new.stride()))
        if v_new.shape != k_new.shape or v_strides != (sb, sh, sn, sd) or v_new.dtype != k_new.dtype:
            raise ValueError("v_new must have k_new's shape, strides and dtype")
        if not k_new.is_cuda or not v_new.is_cuda:
            raise ValueError("k_new and v_new must be CUDA tensors")
        if sd != 1:
            raise ValueError("rows of k_new must be contiguous")
        size = k_new.element_size()
        if any(x * size % 16 for x in (sb, sh, sn)) or k_new.data_ptr() % 16 or v_new.data_ptr() % 16:
            raise ValueError("rows of k_new and v_new must start at multiples of 16 bytes")
        _same_device(cache.device, k_new=k_new, v_new=v_new, starts=starts, counts=counts)
        if cache.codes is not None and (t is None) == (ratio is None):
            raise ValueError("a cache with codes needs a threshold t or a ratio")
        if ratio is not None and not ratio > 0:
            raise ValueError("ratio must be in (0, 1]")
        index, handle = _where(cache.device, stream)
        args = (cache.ptr, _c_p(k_new.data_ptr()), _c_p(v_new.data_ptr()), _c_i(_dtype_code(k_new)),
                _c_i64(n), _c_i64(sb), _c_i64(sh), _c_i64(sn), _lens(cache, starts, "starts"),
                None if counts is None else _lens(cache, counts, "counts"),
                _c_f(0.0 if t is None else t), _c_f(0.0 if ratio is None else ratio),
                *_ws(ws, cache.device), _c_p(handle))
        super().__init__("adamas_kv8_append", args, (cache, k_new, v_new, starts, counts, ws), index)


def _starts(cache, starts, stream):
    if isinstance(starts, int):
        with _owner(cache.device, stream):
            return torch.full((cache.B,), starts, dtype=torch.int32, device=cache.device)
    return starts


def kv8_append(cache: KV8Cache, k_new, v_new, starts, ws, counts=None, t=None, ratio=None,
               stream=None):
    """Quantises rows k_new, v_new [B,Hkv,n,128] (bf16 or float32, the same strides for both; rows
    contiguous, each starting at a multiple of 16 bytes) into positions starts[b] .. of every
    sequence (starts: int32 [B], or one int for all); counts [B] int32: how many of the n rows
    (n at most the cache's Lmax) each sequence takes (default: all).  A cache with codes gets the new keys' codes (threshold t, or ratio of each key's absmax)."""
    PreparedKV8Append(cache, k_new, v_new, _starts(cache, starts, stream), ws, counts, t, ratio,
                      stream)()
    return cache


class PreparedKV8Read(_Call):
    """kv8_read bound to fixed buffers."""

    def __init__(self, cache: KV8Cache, starts, n: int, k_out, v_out, ws, stream=None):
        _same_device(cache.device, starts=starts, k_out=k_out, v_out=v_out)
        shape = (cache.B, cache.Hkv, n, HEAD_DIM)
        index, handle = _where(cache.device, stream)
        args = (cache.ptr, _lens(cache, starts, "starts"), _c_i64(n), _c_i(_dtype_code(k_out)),
                _c_p(_typed(k_out, "k_out", k_out.dtype, shape)),
                _c_p(_typed(v_out, "v_out", k_out.dtype, shape)), *_ws(ws, cache.device),
                _c_p(handle))
        super().__init__("adamas_kv8_read", args, (cache, starts, k_out, v_out, ws), index)


def kv8_read(cache: KV8Cache, starts, n: int, ws, dtype=torch.bfloat16, stream=None):
    """Values of positions starts[b] .. starts[b] + n - 1: (k, v) [B,Hkv,n,128]."""
    with _owner(cache.device, stream):
        k, v = (torch.empty((cache.B, cache.Hkv, n, HEAD_DIM), dtype=dtype, device=cache.device)
                for _ in range(2))
    PreparedKV8Read(cache, _starts(cache, starts, stream), n, k, v, ws, stream)()
    return k, v


# ------------------------------------------------------------------ attention
def _attention_args(cache, q, out, weights, weights_out):
    B, Hq, d = q.shape
    if (B, d) != (cache.B, HEAD_DIM):
        raise ValueError("q must be [B, Hq, 128] of the cache's B")
    _same_device(cache.device, q=q, out=out, weights=weights, weights_out=weights_out)
    if weights_out is None:
        weights_out = weights
    shape = (B, cache.Hkv, cache.Lmax)
    w = [None if x is None else _c_p(_typed(x, "weights", torch.float32, shape))
         for x in (weights, weights_out)]
    return (_c_p(_dev(q, "q")), _c_i(_dtype_code(q))), (
        *w, _c_p(_typed(out, "out", torch.float32, (B, Hq, HEAD_DIM)))), Hq


class PreparedKV8Attention(_Call):
    """kv8_attention bound to fixed buffers."""

    def __init__(self, q, cache: KV8Cache, seq_lens, ws, out, weights=None, weights_out=None,
                 stream=None):
        first, last, Hq = _attention_args(cache, q, out, weights, weights_out)
        _same_device(cache.device, seq_lens=seq_lens)
        index, handle = _where(cache.device, stream)
        lens = None if seq_lens is None else _lens(cache, seq_lens, "seq_lens")
        args = (*first, cache.ptr, _c_i(Hq), lens, *_ws(ws, cache.device), *last, _c_p(handle))
        super().__init__("adamas_kv8_attention", args,
                         (q, cache, seq_lens, ws, out, weights, weights_out), index)


def kv8_attention(q, cache: KV8Cache, seq_lens, ws, weights=None, weights_out=None, out=None,
                  stream=None):
    """Dense attention of q [B,Hq,128] over the first seq_lens[b] positions (int32 [B], None: all)
    of an 8-bit cache: out [B,Hq,128] float32.  weights [B,Hkv,Lmax] float32: every position's
    attention weight (summed over its query heads) is added, into weights_out or in place."""
    if out is None:
        with _owner(cache.device, stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=cache.device)
    PreparedKV8Attention(q, cache, seq_lens, ws, out, weights, weights_out, stream)()
    return out


class PreparedKV8SparseAttention(_Call):
    """kv8_sparse_attention bound to fixed buffers."""

    def __init__(self, q, cache: KV8Cache, idx, ws, out, shared: bool = False, weights=None,
                 weights_out=None, stream=None):
        first, last, Hq = _attention_args(cache, q, out, weights, weights_out)
        _same_device(cache.device, idx=idx)
        k = idx.shape[-1]
        index, handle = _where(cache.device, stream)
        lists = _typed(idx, "idx", torch.int32, (cache.B, cache.Hkv if shared else Hq, k))
        args = (*first, cache.ptr, _c_i(Hq), _c_p(lists), _c_i(k), _c_i(int(bool(shared))),
                *_ws(ws, cache.device), *last, _c_p(handle))
        super().__init__("adamas_kv8_sparse_attention", args,
                         (q, cache, idx, ws, out, weights, weights_out), index)


def kv8_sparse_attention(q, cache: KV8Cache, idx, ws, shared: bool = False, weights=None,
                         weights_out=None, out=None, stream=None):
    """Attention of q [B,Hq,128] over positions idx [B,Hq,k] (shared: [B,Hkv,k]) int32 of an 8-bit
    cache; entries below 0 are skipped.  weights as in kv8_attention."""
    if out is None:
        with _owner(cache.device, stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=cache.device)
    PreparedKV8SparseAttention(q, cache, idx, ws, out, shared, weights, weights_out, stream)()
    return out


# ------------------------------------------------------------------- eviction
class PreparedKV8Evict(_Call):
    """kv8_evict bound to fixed buffers."""

    def __init__(self, cache: KV8Cache, dst: KV8Cache, weights, weights_out, seq_lens, lens_out, keep,
                 budget: int, sink: int, recent: int, ws, stream=None):
        _same_device(cache.device, dst=dst.k, weights=weights, weights_out=weights_out,
                     seq_lens=seq_lens, lens_out=lens_out, keep=keep)
        index, handle = _where(cache.device, stream)
        f32, unit = torch.float32, (cache.B, cache.Hkv)
        args = (cache.ptr, dst.ptr,
                _c_p(_typed(weights, "weights", f32, (*unit, cache.Lmax))),
                _c_p(_typed(weights_out, "weights_out", f32, (*unit, dst.Lmax))),
                _lens(cache, seq_lens, "seq_lens"), _lens(cache, lens_out, "lens_out"),
                _c_i(budget), _c_i(sink), _c_i(recent),
                _c_p(_typed(keep, "keep", torch.int32, (*unit, budget))), *_ws(ws, cache.device),
                _c_p(handle))
        super().__init__("adamas_kv8_evict", args,
                         (cache, dst, weights, weights_out, seq_lens, lens_out, keep, ws), index)


def kv8_evict(cache: KV8Cache, weights, seq_lens, budget: int, ws, sink: int = 0, recent: int = 0,
              dst: KV8Cache | None = None, weights_out=None, lens_out=None, keep=None, stream=None):
    """Cuts every sequence to at most `budget` rows per kv head: the first `sink`, the last `recent`
    and the largest weights between.  Rows, scales, codes and weights move to the front, in
    place (dst None) or into dst.  Returns (keep [B,Hkv,budget] int32, new lengths [B])."""
    if dst is None:
        dst = cache
        weights_out = weights if weights_out is None else weights_out
        lens_out = seq_lens if lens_out is None else lens_out
    with _owner(cache.device, stream):
        if weights_out is None:
            weights_out = torch.zeros((dst.B, dst.Hkv, dst.Lmax), dtype=torch.float32,
                                      device=cache.device)
        if lens_out is None:
            lens_out = torch.empty_like(seq_lens)
        if keep is None:
            keep = torch.empty((cache.B, cache.Hkv, budget), dtype=torch.int32, device=cache.device)
    PreparedKV8Evict(cache, dst, weights, weights_out, seq_lens, lens_out, keep, budget, sink, recent,
                     ws, stream)()
    return keep, lens_out


def evict_select(weights, seq_lens, budget: int, ws, sink: int = 0, recent: int = 0,
                 weights_out=None, keep=None, stream=None):
    """The positions kv8_evict would keep, for any cache: keep [B,Hkv,budget] int32, ascending, then -1.
    weights_out (optional, may be `weights`) receives the kept weights."""
    B, Hkv, Lmax = weights.shape
    device = weights.device
    if keep is None:
        with _owner(device, stream):
            keep = torch.empty((B, Hkv, budget), dtype=torch.int32, device=device)
    _same_device(device, seq_lens=seq_lens, weights_out=weights_out, keep=keep)
    index, handle = _where(device, stream)
    out, top = None, 0
    if weights_out is not None:
        top = weights_out.shape[-1]
        out = _c_p(_typed(weights_out, "weights_out", torch.float32, (B, Hkv, top)))
    args = (_c_p(_typed(weights, "weights", torch.float32)), _c_i(B), _c_i(Hkv), _c_i64(Lmax),
            _c_p(_typed(seq_lens, "seq_lens", torch.int32, (B,))), _c_i(budget), _c_i(sink),
            _c_i(recent), _c_p(_typed(keep, "keep", torch.int32, (B, Hkv, budget))), out, _c_i64(top),
            *_ws(ws, device), _c_p(handle))
    _Call("adamas_evict_select", args, (weights, seq_lens, keep, weights_out, ws), index)()
    return keep


def compact_rows(src, keep, seq_lens, ws, dst=None, block_table=None, max_seq_len=None, stream=None):
    """Moves row keep[b,h,i] of a cache to row i (i < min(seq_lens[b], keep's length)), in place or into
    dst: rows of 32 (codes), 256 (bf16) or 512 (float32) bytes, src [B,Hkv,Lmax,.] or, with a
    block_table, [P,Hkv,page,.]."""
    dst = src if dst is None else dst
    B, Hkv, n = keep.shape
    row_bytes = src.shape[-1] * src.element_size()
    if dst.shape != src.shape or dst.dtype != src.dtype or src.dim() != 4 or src.shape[1] != Hkv:
        raise ValueError("src and dst must be one cache's [B or P, Hkv, rows, .] tensors")
    _same_device(src.device, dst=dst, keep=keep, seq_lens=seq_lens, block_table=block_table)
    page = pages = blocks = 0
    Lmax = src.shape[2]
    table = None
    if block_table is not None:
        table = _c_p(_typed(block_table, "block_table", torch.int32))
        pages, page, blocks = src.shape[0], src.shape[2], block_table.shape[1]
        Lmax = blocks * page if max_seq_len is None else max_seq_len
    if (B if block_table is None else block_table.shape[0]) != (src.shape[0] if block_table is None else B):
        raise ValueError("keep's batch must be the cache's")
    index, handle = _where(src.device, stream)
    args = (_c_p(_dev(src, "src")), _c_p(_dev(dst, "dst")), _c_i(row_bytes), _c_i(B), _c_i(Hkv),
            _c_i64(Lmax), _c_i(page), _c_i64(pages), table, _c_i(blocks),
            _c_p(_typed(keep, "keep", torch.int32)), _c_i(n),
            _c_p(_typed(seq_lens, "seq_lens", torch.int32, (B,))), *_ws(ws, src.device),
            _c_p(handle))
    _Call("adamas_compact_rows", args, (src, dst, keep, seq_lens, block_table, ws), index)()
    return dst
