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


def _row_stride(t):
    """Elements between rows (a single row's stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


def _raw_stream(device, stream):
    import torch

    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


class PagedKV:
    """One layer's cache and the batch of sequences that calls work on.

    cache [pages, 2, heads, page_size, dim] bf16 (pages may be further apart
    than their size); table [rows, width] int32; cu_q [batch+1] int32; kv_len
    [rows] int32, the new tokens included; rows: optional [batch] int32, the
    table row of each sequence of the batch (default: row b for sequence b).
    max_q: the most new tokens of one sequence as far as the caller knows (it
    chooses the kernel); it may be set anew between calls.
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
        self.device = dev
        pages, _, self.heads, self.page_size, self.dim = cache.shape
        page = 2 * self.heads * self.page_size * self.dim
        self._view = _View(
            cache.data_ptr(), cache.stride(0) if pages > 1 else page, pages, self.heads,
            self.page_size, self.dim, table.data_ptr(), _row_stride(table), table.shape[1],
            table.shape[0], None if rows is None else rows.data_ptr(), cu_q.data_ptr(),
            kv_len.data_ptr(), cu_q.shape[0] - 1, int(max_q))
        self._ref = ctypes.byref(self._view)

    @property
    def max_q(self):
        return self._view.max_q

    @max_q.setter
    def max_q(self, n):
        self._view.max_q = int(n)


class KVPool:
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
        self.device = dev
        size = data.element_size()
        page = data[0, 0].numel() * size
        self._pool = _Pool(
            data.data_ptr(), data.stride(0) * size if layers > 1 else page,
            data.stride(1) * size if pages > 1 else page, page, layers, pages,
            int(data.shape[-2] if page_size is None else page_size), refs.data_ptr(),
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
    import torch

    dev, dim = kv.device, kv.dim
    bf = torch.bfloat16
    _same("qkv", dev, qkv, bf, dims=2, row_stride=True)
    T, width = qkv.shape
    hq = width // dim - 2 * kv.heads
    if hq < 1 or width % dim:
        raise ValueError("qkv: expected [T, (Hq + %d)*%d], got shape %s"
                         % (2 * kv.heads, dim, tuple(qkv.shape)))
    _same("rope", dev, rope, torch.float32, dims=2)
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk: give both or neither")
    if wq is not None:
        _same("wq", dev, wq, bf, shape=(dim,))
        _same("wk", dev, wk, bf, shape=(dim,))
    if positions is not None:
        _same("positions", dev, positions, torch.int32, shape=(T,))
    if q is None:
        q = torch.empty((T, hq * dim), dtype=bf, device=dev)
    else:
        _same("q", dev, q, bf, shape=(T, hq * dim), row_stride=True)
    if T == 0:
        return q
    _check(lib().kv_append(
        kv._ref, qkv.data_ptr(), _row_stride(qkv), None if wq is None else wq.data_ptr(),
        None if wk is None else wk.data_ptr(), eps, rope.data_ptr(), rope.shape[0], rope.shape[1],
        1 if interleaved else 0, None if positions is None else positions.data_ptr(), q.data_ptr(),
        _row_stride(q), T, hq, _raw_stream(dev, stream)), "kv_append")
    return q


def kv_attention(q, kv, out=None, lse=None, scale=None, window=0, stream=None):
    """Attention of the new tokens over the cache: each token sees the positions
    up to its own (the last ``window`` of them if window > 0). q [T, Hq*dim]
    bf16 (rows may be further apart); scale: 1/sqrt(dim) by default; lse:
    optional [T, Hq] fp32 output. Returns out [T, Hq*dim] bf16."""
    import torch

    dev, dim = kv.device, kv.dim
    _same("q", dev, q, torch.bfloat16, dims=2, row_stride=True)
    T, width = q.shape
    hq = width // dim
    if hq < 1 or width % dim or hq % kv.heads:
        raise ValueError("q: expected [T, Hq*%d] with Hq a multiple of %d, got shape %s"
                         % (dim, kv.heads, tuple(q.shape)))
    if out is None:
        out = torch.empty((T, width), dtype=torch.bfloat16, device=dev)
    else:
        _same("out", dev, out, torch.bfloat16, shape=(T, width), row_stride=True)
    if lse is not None:
        _same("lse", dev, lse, torch.float32, shape=(T, hq))
    if T == 0:
        return out
    _check(lib().kv_attention(
        kv._ref, q.data_ptr(), _row_stride(q), out.data_ptr(), _row_stride(out),
        None if lse is None else lse.data_ptr(), T, hq, dim ** -0.5 if scale is None else scale,
        window, _raw_stream(dev, stream)), "kv_attention")
    return out


def last_attention() -> str:
    """The kernel regime of this thread's last kv_attention call."""
    return REGIME_NAMES.get(lib().kv_last_attention(), "?")


# ---------------------------------------------------------------- the pages
def _list(pool, what, t, n=None):
    import torch

    return _same(what, pool.device, t, torch.int32, dims=1, shape=None if n is None else (n,))


def kv_resize(pool, seqs, lens, stream=None):
    """Set the lengths of sequences ``seqs`` to ``lens`` (int32 on the device):
    pages are taken (the lowest free ones, in order) or given back. All or
    nothing: pool.info[0] is the number of pages that were lacking."""
    n = _list(pool, "seqs", seqs).shape[0]
    _list(pool, "lens", lens, n)
    if n:
        _check(lib().kv_resize(pool._ref, seqs.data_ptr(), lens.data_ptr(), n,
                               _raw_stream(pool.device, stream)), "kv_resize")


def kv_free(pool, seqs, stream=None):
    """Give back every page of sequences ``seqs``; their lengths become 0."""
    n = _list(pool, "seqs", seqs).shape[0]
    if n:
        _check(lib().kv_free(pool._ref, seqs.data_ptr(), n, _raw_stream(pool.device, stream)),
               "kv_free")


def kv_fork(pool, src, dst, stream=None):
    """Sequence dst[i] becomes a copy of src[i]: full pages are shared, a last
    page that is partly filled is copied. What dst[i] held is given back."""
    n = _list(pool, "src", src).shape[0]
    _list(pool, "dst", dst, n)
    if n:
        _check(lib().kv_fork(pool._ref, src.data_ptr(), dst.data_ptr(), n,
                             _raw_stream(pool.device, stream)), "kv_fork")


def kv_copy(pool, src, dst, stream=None):
    """Copy page src[i] to page dst[i] in every layer."""
    n = _list(pool, "src", src).shape[0]
    _list(pool, "dst", dst, n)
    if n:
        _check(lib().kv_copy(pool._ref, src.data_ptr(), dst.data_ptr(), n,
                             _raw_stream(pool.device, stream)), "kv_copy")


def kv_compact(pool, stream=None):
    """Move pages so that the n pages in use are pages 0 .. n-1; the table and
    the reference counts follow."""
    _check(lib().kv_compact(pool._ref, _raw_stream(pool.device, stream)), "kv_compact")
