"""The paged key/value cache: handles over a cache and its calls.

A decode step with attention, for a batch of sequences of a cache:

  kv_resize     once: room for the step's new tokens (lengths then count them)
  kv_append     per layer: the heads of the fused q|k|v projection are normed and
                rotated, the keys and values go to their places in the cache
  kv_attention  per layer: the new tokens' queries over the cache

and kv_free, kv_fork, kv_copy and kv_compact to manage the pages. The handles
(PagedKV, KVPool) check their tensors once and keep them alive; a program makes
them when it makes the tensors, and the tensors' contents -- lengths, page
tables -- change from step to step on the device.
"""
from __future__ import annotations

import ctypes
import operator

from . import REGIME_NAMES, _check, lib

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class _View(ctypes.Structure):
    _fields_ = [("cache", _P), ("page_stride", _I64), ("pages", _I32), ("heads", _I32),
                ("page_size", _I32), ("dim", _I32), ("table", _P), ("table_stride", _I64),
                ("width", _I32), ("table_rows", _I32), ("rows", _P), ("cu_q", _P), ("kv_len", _P),
                ("batch", _I32), ("max_q", _I32)]


class _Pool(ctypes.Structure):
    _fields_ = [("data", _P), ("layer_stride", _I64), ("page_stride", _I64), ("page_bytes", _I64),
                ("layers", _I32), ("pages", _I32), ("page_size", _I32), ("refs", _P), ("table", _P),
                ("table_stride", _I64), ("width", _I32), ("lens", _P), ("seqs", _I32),
                ("info", _P)]


def _same(what, device, t, dtype, dims=None, shape=None, row_stride=False):
    """Reject a tensor the C ABI would misread; row_stride: rows may be further
    apart than their length (columns contiguous)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch tensor, got %s" % (what, type(t).__name__))
    if t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if dims is not None and t.dim() != dims:
        raise ValueError("%s: expected %d dimensions, got shape %s" % (what, dims, tuple(t.shape)))
    if row_stride:
        if t.stride(-1) != 1:
            raise ValueError("%s: needs unit column stride" % what)
    elif not t.is_contiguous():
        raise ValueError("%s: must be contiguous" % what)
    if t.device.type != "cuda":
        raise ValueError("%s: expected a CUDA tensor, got one on %s" % (what, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s: on %s, the other operands on %s" % (what, t.device, device))
    return t


def _rows(what, h, t, dtype):
    """A matrix whose rows may be further apart than their length: its rows,
    row length and row stride. (The calls of a decode step are short: what they
    pass is looked over in few steps, and _same says what is wrong with it.)"""
    try:
        if t.dtype is dtype and t.get_device() == h._index:
            n, width = t.shape
            ld, one = t.stride()
            if one == 1:
                # a single row's stride says nothing
                return n, width, (ld if n > 1 else width)
    except (AttributeError, ValueError):
        pass
    _same(what, h.device, t, dtype, dims=2, row_stride=True)
    raise ValueError("%s: needs unit column stride" % what)  # a column of length 1


def _list(what, h, t, dtype, n=None):
    """A contiguous vector (of n elements); its length."""
    try:
        if (t.dtype is dtype and t.get_device() == h._index and t.dim() == 1
                and t.is_contiguous() and (n is None or t.shape[0] == n)):
            return t.shape[0]
    except AttributeError:
        pass
    _same(what, h.device, t, dtype, dims=1, shape=None if n is None else (n,))


class _Handle:
    """What both handles keep: the device, and torch's names that the calls use."""

    def _bind(self, device):
        import torch

        self.device, self._index = device, device.index
        self._bf16, self._f32, self._i32 = torch.bfloat16, torch.float32, torch.int32
        self._empty, self._current = torch.empty, torch._C._cuda_getCurrentRawStream

    def _stream(self, stream):
        return self._current(self._index) if stream is None else stream.cuda_stream


def _int32(what, n):
    """An integer that the C ABI's 32 bits hold (ctypes would cut it to them)."""
    n = operator.index(n)
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError("%s: %d does not fit 32 bits" % (what, n))
    return n


def _row_stride(t):
    """Elements between rows (a single row's stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


class PagedKV(_Handle):
    """One layer's cache and the batch of sequences that calls work on.

    cache [pages, 2, heads, page_size, dim] bf16 (pages may be further apart
    than their size); table [rows, width] int32; cu_q [batch+1] int32; kv_len
    [rows] int32, the new tokens included; rows: optional [batch] int32, the
    table row of each sequence of the batch (default: row b for sequence b).
    max_q: the most new tokens of one sequence as far as the caller knows; it may
    be set anew between calls. It chooses the kernel, not the result: give 1 for
    a step of one token a sequence, as 0 (unknown) is taken as all of the call's
    tokens and sends such a step to the kernel for chunks (8 sequences over 2000
    positions 28 us instead of 14, 64 over 4000 102 instead of 86).
    """

    def __init__(self, cache, table, cu_q, kv_len, rows=None, max_q=0):
        import torch

        i32 = torch.int32
        if not isinstance(cache, torch.Tensor):
            raise TypeError("cache: expected a torch tensor, got %s" % type(cache).__name__)
        if cache.dim() != 5 or cache.shape[1] != 2:
            raise ValueError("cache: expected [pages, 2, heads, page_size, dim], got shape %s"
                             % (tuple(cache.shape),))
        if cache.shape[0] and not cache[0].is_contiguous():
            raise ValueError("cache: a page must be contiguous")
        _same("cache", None, cache, torch.bfloat16, row_stride=True)
        dev = cache.device
        _same("table", dev, table, i32, dims=2, row_stride=True)
        _same("cu_q", dev, cu_q, i32, dims=1)
        if rows is not None:
            _same("rows", dev, rows, i32, shape=(cu_q.shape[0] - 1,))
        elif table.shape[0] < cu_q.shape[0] - 1:
            raise ValueError("table: %d rows for a batch of %d" % (table.shape[0],
                                                                   cu_q.shape[0] - 1))
        _same("kv_len", dev, kv_len, i32, shape=(table.shape[0],))
        self.cache, self.table, self.cu_q, self.kv_len, self.rows = cache, table, cu_q, kv_len, rows
        self._bind(dev)
        pages, _, self.heads, self.page_size, self.dim = cache.shape
        page = 2 * self.heads * self.page_size * self.dim
        self._view = _View(
            cache.data_ptr(), cache.stride(0) if pages > 1 else page, pages, self.heads,
            self.page_size, self.dim, table.data_ptr(), _row_stride(table), table.shape[1],
            table.shape[0], None if rows is None else rows.data_ptr(), cu_q.data_ptr(),
            kv_len.data_ptr(), cu_q.shape[0] - 1, _int32("max_q", int(max_q)))
        self._ref = ctypes.byref(self._view)

    @property
    def max_q(self):
        return self._view.max_q

    @max_q.setter
    def max_q(self, n):
        self._view.max_q = _int32("max_q", int(n))


class KVPool(_Handle):
    """The pages of all layers of a cache and the state of its sequences.

    data [layers, pages, ...] of any type (a page of a layer is contiguous;
    layers and pages may be any distance apart); refs [pages], table
    [seqs, width] (-1: unused), lens [seqs] int32; info: optional int32 of at
    least 3 elements that the calls write: pages lacking (0: done), pages free,
    pages copied. page_size: positions of a page (default: the last but one
    dimension of data, as in [layers, pages, 2, heads, page_size, dim]).
    """

    def __init__(self, data, refs, table, lens, info=None, page_size=None):
        import torch

        i32 = torch.int32
        if not isinstance(data, torch.Tensor):
            raise TypeError("data: expected a torch tensor, got %s" % type(data).__name__)
        if data.dim() < 3 or not data.numel():
            raise ValueError("data: expected [layers, pages, ...], got shape %s"
                             % (tuple(data.shape),))
        if data.device.type != "cuda":
            raise ValueError("data: expected a CUDA tensor, got one on %s" % data.device)
        if not data[0, 0].is_contiguous():
            raise ValueError("data: a page must be contiguous")
        dev, (layers, pages) = data.device, data.shape[:2]
        _same("refs", dev, refs, i32, shape=(pages,))
        _same("table", dev, table, i32, dims=2, row_stride=True)
        _same("lens", dev, lens, i32, shape=(table.shape[0],))
        if info is not None:
            _same("info", dev, info, i32, dims=1)
            if info.shape[0] < 3:
                raise ValueError("info: expected 3 elements or more")
        self.data, self.refs, self.table, self.lens, self.info = data, refs, table, lens, info
        self._bind(dev)
        size = data.element_size()
        page = data[0, 0].numel() * size
        self._pool = _Pool(
            data.data_ptr(), data.stride(0) * size if layers > 1 else page,
            data.stride(1) * size if pages > 1 else page, page, layers, pages,
            _int32("page_size", int(data.shape[-2] if page_size is None else page_size)), refs.data_ptr(),
            table.data_ptr(), _row_stride(table), table.shape[1], lens.data_ptr(), table.shape[0],
            None if info is None else info.data_ptr())
        self._ref = ctypes.byref(self._pool)

    def layer(self, l, cu_q, rows=None, max_q=0):
        """PagedKV of one layer for a batch whose sequences have table rows ``rows``."""
        return PagedKV(self.data[l], self.table, cu_q, self.lens, rows=rows, max_q=max_q)


# ---------------------------------------------------------------- the hot path
def kv_append(qkv, kv, rope, wq=None, wk=None, eps=1e-6, q=None, positions=None,
              interleaved=False, stream=None):
    """Norm and rotation of the new tokens' heads, and the append of their keys
    and values to the cache. qkv [T, (Hq + 2*heads)*dim] bf16 (rows may be
    further apart): query heads, key heads, value heads. rope [positions, rot]
    fp32: rot/2 cosines, then rot/2 sines. wq, wk: [dim] bf16 norm weights, or
    both None. Returns q [T, Hq*dim] bf16 (a new tensor if None; may be
    qkv[:, :Hq*dim])."""
    dim, bf = kv.dim, kv._bf16
    T, width, ld = _rows("qkv", kv, qkv, bf)
    hq = width // dim - 2 * kv.heads
    if hq < 1 or width % dim:
        raise ValueError("qkv: expected [T, (Hq + %d)*%d], got shape %s"
                         % (2 * kv.heads, dim, tuple(qkv.shape)))
    positions_at, rot, ld_rope = _rows("rope", kv, rope, kv._f32)
    if ld_rope != rot:
        raise ValueError("rope: must be contiguous")
    wqp = wkp = pos = None
    if wq is not None and wk is not None:
        _list("wq", kv, wq, bf, dim)
        _list("wk", kv, wk, bf, dim)
        wqp, wkp = wq.data_ptr(), wk.data_ptr()
    elif wq is not wk:
        raise ValueError("wq and wk: give both or neither")
    if positions is not None:
        _list("positions", kv, positions, kv._i32, T)
        pos = positions.data_ptr()
    if q is None:
        q = kv._empty((T, hq * dim), dtype=bf, device=kv.device)
        ldq = hq * dim
    else:
        rows, cols, ldq = _rows("q", kv, q, bf)
        if rows != T or cols != hq * dim:
            raise ValueError("q: expected shape %s, got %s" % ((T, hq * dim), tuple(q.shape)))
    if T:
        rc = lib().kv_append(kv._ref, qkv.data_ptr(), ld, wqp, wkp, eps, rope.data_ptr(),
                             positions_at, rot, 1 if interleaved else 0, pos, q.data_ptr(), ldq, T,
                             hq, kv._stream(stream))
        if rc:
            _check(rc, "kv_append")
    return q


def kv_attention(q, kv, out=None, lse=None, scale=None, window=0, stream=None):
    """Attention of the new tokens over the cache: each token sees the positions
    up to its own (the last ``window`` of them if window > 0). q [T, Hq*dim]
    bf16 (rows may be further apart); scale: 1/sqrt(dim) by default; lse:
    optional [T, Hq] fp32 output. Returns out [T, Hq*dim] bf16."""
    dim, bf = kv.dim, kv._bf16
    T, width, ldq = _rows("q", kv, q, bf)
    hq = width // dim
    if hq < 1 or width % dim or hq % kv.heads:
        raise ValueError("q: expected [T, Hq*%d] with Hq a multiple of %d, got shape %s"
                         % (dim, kv.heads, tuple(q.shape)))
    if out is None:
        out = kv._empty((T, width), dtype=bf, device=kv.device)
        ldo = width
    else:
        rows, cols, ldo = _rows("out", kv, out, bf)
        if rows != T or cols != width:
            raise ValueError("out: expected shape %s, got %s" % ((T, width), tuple(out.shape)))
    lsep = None
    if lse is not None:
        rows, cols, ld = _rows("lse", kv, lse, kv._f32)
        if rows != T or cols != hq or ld != hq:
            raise ValueError("lse: expected contiguous of shape %s, got %s" % ((T, hq),
                                                                            tuple(lse.shape)))
        lsep = lse.data_ptr()
    if T:
        rc = lib().kv_attention(kv._ref, q.data_ptr(), ldq, out.data_ptr(), ldo, lsep, T, hq,
                                dim ** -0.5 if scale is None else scale,
                                window and _int32("window", window),
                                kv._stream(stream))
        if rc:
            _check(rc, "kv_attention")
    return out


def last_attention() -> str:
    """The kernel regime of this thread's last kv_attention call."""
    return REGIME_NAMES.get(lib().kv_last_attention(), "?")


# ---------------------------------------------------------------- the pages
def kv_resize(pool, seqs, lens, stream=None):
    """Set the lengths of sequences ``seqs`` to ``lens`` (int32 on the device):
    pages are taken (the lowest free ones, in order) or given back. All or
    nothing: pool.info[0] is the number of pages that were lacking."""
    n = _list("seqs", pool, seqs, pool._i32)
    _list("lens", pool, lens, pool._i32, n)
    if n:
        _check(lib().kv_resize(pool._ref, seqs.data_ptr(), lens.data_ptr(), n,
                               pool._stream(stream)), "kv_resize")


def kv_free(pool, seqs, stream=None):
    """Give back every page of sequences ``seqs``; their lengths become 0."""
    n = _list("seqs", pool, seqs, pool._i32)
    if n:
        _check(lib().kv_free(pool._ref, seqs.data_ptr(), n, pool._stream(stream)),
               "kv_free")


def kv_fork(pool, src, dst, stream=None):
    """Sequence dst[i] becomes a copy of src[i]: full pages are shared, a last
    page that is partly filled is copied. What dst[i] held is given back."""
    n = _list("src", pool, src, pool._i32)
    _list("dst", pool, dst, pool._i32, n)
    if n:
        _check(lib().kv_fork(pool._ref, src.data_ptr(), dst.data_ptr(), n,
                             pool._stream(stream)), "kv_fork")


def kv_copy(pool, src, dst, stream=None):
    """Copy page src[i] to page dst[i] in every layer."""
    n = _list("src", pool, src, pool._i32)
    _list("dst", pool, dst, pool._i32, n)
    if n:
        _check(lib().kv_copy(pool._ref, src.data_ptr(), dst.data_ptr(), n,
                             pool._stream(stream)), "kv_copy")


def kv_compact(pool, stream=None):
    """Move pages so that the n pages in use are pages 0 .. n-1; the table and
    the reference counts follow."""
    _check(lib().kv_compact(pool._ref, pool._stream(stream)), "kv_compact")
