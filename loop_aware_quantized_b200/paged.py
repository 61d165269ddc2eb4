"""Paged cells: a key-value cache whose tokens live in pages.

``page_map`` makes room for a step's new tokens (block tables and slot map from
the request lengths), ``paged_append`` writes their keys and values,
``paged_decode`` is the attention of each request's newest token over its
pages, ``page_release`` gives pages back.  All state is in device tensors, so a
step of these calls can be captured into a CUDA graph and replayed.
``PagedCache`` keeps the tensors of one cache together.

Argument marshalling only, as in ``loopkv``: the work runs in ``libloopkv.so``
(``include/loopkv.h``, "Paged cells").  Checks here raise LoopKVError with
LOOPKV_ERR_INVALID_ARG and launch nothing; what only the device data can show
(no free page, a page id outside the pool) sets bits in ``status`` (int32 [1]).

Shapes: pages [cells, pages, KV heads, page size, head dim] (bf16, fp16, or
uint8 codes with ``meta`` fp32 [cells, pages, KV heads, page size, 4]); table
int32 [batch, pages of the longest request]; slot = page * page size + offset.
Vectors (q, k, v, cur_k, cur_v) are [listed cells, rows, heads, head dim] with
contiguous channels; their other strides are free (multiples of 8 elements), so
slices of a fused projection's output can be given as they are.
"""

import ctypes
import functools

import numpy as np
import torch

from . import _paged
from . import loopkv as _lk
from .loopkv import _check, _invalid

# Page dtype -> (format, dtype of the vectors)
_FORMATS = {torch.bfloat16: (_lk.LOOPKV_PAGE_BF16, torch.bfloat16),
            torch.float16: (_lk.LOOPKV_PAGE_F16, torch.float16),
            torch.uint8: (_lk.LOOPKV_PAGE_Q8, torch.bfloat16)}
_I32, _F32 = torch.int32, torch.float32

# A decode step's calls are a few microseconds of device time each, so a call in
# its plain form (the current device and its current stream, nothing wrong with
# the arguments) is checked and launched by _paged (csrc/paged_binding.cpp).  It
# returns _NOT_PLAIN, having done nothing, for the rest, which goes the way
# written here: a stream that is given, another device, what to tell the caller.
_NOT_PLAIN = -1
_paged.bind(*(ctypes.cast(getattr(_lk._lib, name), ctypes.c_void_p).value for name in (
    "loopkv_page_map", "loopkv_page_release", "loopkv_paged_append", "loopkv_paged_workspace",
    "loopkv_paged_decode")))


def _place(where, index, stream):
    """(stream handle, context or None) of a launch on device ``index``: the
    stream given, or the device's current one, with the device made current if
    it is not."""
    if stream is None:
        # the handle alone: a torch.cuda.Stream object takes 2 us to make
        handle = torch._C._cuda_getCurrentRawStream(index)
        return handle, None if torch.cuda.current_device() == index else torch.cuda.device(index)
    if stream.device_index != index:
        raise _invalid(where, "the stream is on %s, the tensors on cuda:%d" % (stream.device, index))
    return stream.cuda_stream, torch.cuda.stream(stream)


def _wrong(t, where, name, dtype, index, shape):
    """What a tensor argument that failed its check lacks."""
    if not isinstance(t, torch.Tensor):
        return _invalid(where, "%s must be a torch tensor, not %s" % (name, type(t).__name__))
    if index < 0 or t.get_device() != index:
        return _invalid(where, "%s must be on %s, not %s" % (
            name, "a CUDA device" if index < 0 else "cuda:%d" % index, t.device))
    if t.dtype != dtype:
        return _invalid(where, "%s must be %s, not %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        return _invalid(where, "%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    return _invalid(where, "%s must be contiguous" % name)


def _full(t, where, name, dtype, index, shape):
    """Pointer of a contiguous tensor of a given type and shape on a device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and \
            t.shape == shape and index >= 0 and t.is_contiguous():
        return t.data_ptr()
    raise _wrong(t, where, name, dtype, index, shape)


def _ints(t, where, name, index, shape):
    return _full(t, where, name, _I32, index, shape)


def _size(value, where, name):
    if isinstance(value, bool) or int(value) != value or not 0 <= value < 1 << 31:
        raise _invalid(where, "%s must be a count, not %r" % (name, value))
    return int(value)


def _shape(t, where, name, ndim):
    if not isinstance(t, torch.Tensor):
        raise _invalid(where, "%s must be a torch tensor, not %s" % (name, type(t).__name__))
    shape = t.shape
    if len(shape) != ndim:
        raise _invalid(where, "%s must have %d dimensions, not %d" % (name, ndim, len(shape)))
    return shape


def _launch(fn, context, *args):
    if context is None:
        rc = fn(*args)
    else:
        with context:
            rc = fn(*args)
    if rc:
        _check(rc, fn.__name__)


def page_map(lengths, n_new, table, free, free_count, page_size, slots, starts, newest=None,
             lengths_out=None, free_count_out=None, status=None, stream=None):
    """Room for ``n_new`` [batch] new tokens of requests that hold ``lengths``
    [batch]: pages from the end of ``free`` [pages of the pool] (the first
    ``free_count`` [1] are free) are entered in ``table`` [batch, width];
    ``slots`` [rows] gets the slot of every new token, request after request
    (-1 behind the last and for refused requests), ``starts`` [batch + 1] the
    first row of every request, ``newest`` [batch] (optional) the slot of its
    last new token (-1: none).  New lengths and free count go to
    ``lengths_out`` / ``free_count_out`` (None: in place).  A request that does
    not fit (pages, table width, rows) is refused whole: its length stays and
    ``status`` gets a bit.  Returns (slots, starts)."""
    where = "page_map"
    if stream is None:
        rc = _paged.page_map(lengths, n_new, table, free, free_count, page_size, slots, starts, newest,
                             lengths_out, free_count_out, status)
        if rc != _NOT_PLAIN:
            if rc:
                _check(rc, "loopkv_page_map")
            return slots, starts
    batch, width = _shape(table, where, "table", 2)
    (n_pages,), (rows,) = _shape(free, where, "free", 1), _shape(slots, where, "slots", 1)
    page_size = _size(page_size, where, "page_size")
    index, per_request, one = table.get_device(), (batch,), (1,)
    d_len = _ints(lengths, where, "lengths", index, per_request)
    d_count = _ints(free_count, where, "free_count", index, one)
    d_new = _ints(n_new, where, "n_new", index, per_request)
    d_table = _ints(table, where, "table", index, (batch, width))
    d_free = _ints(free, where, "free", index, (n_pages,))
    d_slots = _ints(slots, where, "slots", index, (rows,))
    d_starts = _ints(starts, where, "starts", index, (batch + 1,))
    d_newest = None if newest is None else _ints(newest, where, "newest", index, per_request)
    d_len_out = d_len if lengths_out is None else _ints(lengths_out, where, "lengths_out", index, per_request)
    d_count_out = d_count if free_count_out is None else _ints(free_count_out, where, "free_count_out", index, one)
    d_status = None if status is None else _ints(status, where, "status", index, one)
    handle, context = _place(where, index, stream)
    _launch(_lk.loopkv_page_map, context, batch, page_size, width, n_pages, rows, d_len, d_new, d_table,
            d_free, d_count, d_slots, d_starts, d_newest, d_len_out, d_count_out, d_status, handle)
    return slots, starts


def page_release(lengths, new_lengths, table, free, free_count, page_size, lengths_out=None,
                 free_count_out=None, status=None, stream=None):
    """Cut requests from ``lengths`` [batch] to ``new_lengths`` [batch] tokens
    (0: the request ended) and push the pages they no longer need to the end
    of ``free``, request after request.  New lengths and free count go to
    ``lengths_out`` / ``free_count_out`` (None: in place); the table stays as
    it is.  A request whose new length is not in 0 .. its length keeps it."""
    where = "page_release"
    if stream is None:
        rc = _paged.page_release(lengths, new_lengths, table, free, free_count, page_size, lengths_out,
                                 free_count_out, status)
        if rc != _NOT_PLAIN:
            if rc:
                _check(rc, "loopkv_page_release")
            return
    batch, width = _shape(table, where, "table", 2)
    (n_pages,) = _shape(free, where, "free", 1)
    page_size = _size(page_size, where, "page_size")
    index, per_request, one = table.get_device(), (batch,), (1,)
    d_len = _ints(lengths, where, "lengths", index, per_request)
    d_count = _ints(free_count, where, "free_count", index, one)
    d_new = _ints(new_lengths, where, "new_lengths", index, per_request)
    d_table = _ints(table, where, "table", index, (batch, width))
    d_free = _ints(free, where, "free", index, (n_pages,))
    d_len_out = d_len if lengths_out is None else _ints(lengths_out, where, "lengths_out", index, per_request)
    d_count_out = d_count if free_count_out is None else _ints(free_count_out, where, "free_count_out", index, one)
    d_status = None if status is None else _ints(status, where, "status", index, one)
    handle, context = _place(where, index, stream)
    _launch(_lk.loopkv_page_release, context, batch, page_size, width, n_pages, d_len, d_new, d_table, d_free,
            d_count, d_len_out, d_count_out, d_status, handle)


def _pool(k_pages, v_pages, meta, where):
    """(loopkv_page_pool, dtype of the vectors, device index) of the page tensors."""
    shape = _shape(k_pages, where, "k_pages", 5)
    page_dtype, index = k_pages.dtype, k_pages.get_device()
    if page_dtype not in _FORMATS:
        raise _invalid(where, "k_pages must be torch.bfloat16, torch.float16 or torch.uint8, not %s"
                       % page_dtype)
    fmt, dtype = _FORMATS[page_dtype]
    d_k = _full(k_pages, where, "k_pages", page_dtype, index, shape)
    d_v = _full(v_pages, where, "v_pages", page_dtype, index, shape)
    if (meta is None) != (fmt != _lk.LOOPKV_PAGE_Q8):
        raise _invalid(where, "meta belongs to uint8 pages, and to no others")
    d_meta = None if meta is None else _full(meta, where, "meta", _F32, index, shape[:4] + (4,))
    cells, pages, heads, page_size, dim = shape
    return _lk.loopkv_page_pool(cells, pages, page_size, heads, dim, fmt, d_k, d_v, d_meta), dtype, index


def _rows(t, where, name, dtype, index, shape):
    """loopkv_rows of a [cells, rows, heads, head dim] tensor (heads None: any)."""
    got = _shape(t, where, name, 4)
    if t.dtype is not dtype or t.get_device() != index or got[:2] != shape[:2] or got[3] != shape[3] or \
            (got[2] != shape[2] and shape[2] is not None):
        raise _wrong(t, where, name, dtype, index, tuple(g if w is None else w for w, g in zip(shape, got)))
    strides, at = t.stride(), t.data_ptr()
    cell, row, head = (0 if n <= 1 else s for n, s in zip(got, strides[:3]))
    if strides[3] != 1 or (cell | row | head) & 7 or at & 15:
        raise _invalid(where, "%s must have contiguous channels, strides that are multiples of 8 "
                              "and start on a 16-byte boundary; its strides are %s" % (name, strides))
    return _lk.loopkv_rows(at, cell, row, head)


def _to_int32(given, where):
    """The numbers as int32, none of them changed by it (2^32 is not cell 0)."""
    try:
        if given.dtype.kind in "iu":
            a = given.astype(np.int32)
            same = a.astype(given.dtype).tobytes() == given.tobytes()  # (a third of the time of a comparison)
        else:
            with np.errstate(invalid="ignore"):
                a = given.astype(np.int32)
            same = bool((a == given).all())
    except (TypeError, ValueError, OverflowError):
        same = False
    if not same:
        raise _invalid(where, "cells must be numbers of cells, not %r" % (given,))
    return a


def _cells(cells, where):
    """Host int32 array of a list of cells."""
    a = np.asarray(cells)
    if a.dtype != np.int32:
        a = _to_int32(a, where)
    a = np.ascontiguousarray(a).reshape(-1)
    if not 1 <= a.size <= _lk.LOOPKV_MAX_CELLS_PER_CALL:
        raise _invalid(where, "1 to %d cells in a call, not %d" % (
            _lk.LOOPKV_MAX_CELLS_PER_CALL, a.size))
    return a


def paged_append(cells, k, v, slots, k_pages, v_pages, meta=None, status=None, stream=None):
    """Write k, v [listed cells, rows, KV heads, head dim] of new tokens to
    slots ``slots`` [rows] of pool cells ``cells`` (host; distinct; -1: nothing
    is stored of that input).  Rows with slot -1 are skipped.  uint8 pages get
    codes and ``meta`` their scales and zero points."""
    where = "paged_append"
    if stream is None:
        rc = _paged.paged_append(cells, k, v, slots, k_pages, v_pages, meta, status)
        if rc != _NOT_PLAIN:
            if rc:
                _check(rc, "loopkv_paged_append")
            return
    pool, dtype, index = _pool(k_pages, v_pages, meta, where)
    cells = _cells(cells, where)
    (rows,) = _shape(slots, where, "slots", 1)
    shape = (cells.size, rows, pool.n_kv_heads, pool.head_dim)
    kr = _rows(k, where, "k", dtype, index, shape)
    vr = _rows(v, where, "v", dtype, index, shape)
    d_slots = _ints(slots, where, "slots", index, (rows,))
    d_status = None if status is None else _ints(status, where, "status", index, (1,))
    handle, context = _place(where, index, stream)
    _launch(_lk.loopkv_paged_append, context, pool, cells.tobytes(), cells.size, rows, d_slots, kr, vr, d_status, handle)


@functools.lru_cache(maxsize=256)
def _work_bytes(batch, width, group, cells, pages, page_size, heads, dim, fmt):
    """Workspace of a decode, which its sizes alone decide."""
    some = 16  # an aligned address that nothing reads
    rc, nbytes = _lk.loopkv_paged_workspace(
        _lk.loopkv_page_pool(cells, pages, page_size, heads, dim, fmt, some, some,
                             some if fmt == _lk.LOOPKV_PAGE_Q8 else None),
        _lk.loopkv_paged_desc(batch, width, group, 0.0))
    _check(rc, "loopkv_paged_workspace")
    return nbytes


def paged_decode(cells, q, k_pages, v_pages, table, lengths, meta=None, cur_k=None, cur_v=None,
                 current=None, out=None, lse=None, sm_scale=0.0, status=None, stream=None):
    """Attention of one new token per request: q [listed cells, batch, query
    heads, head dim] over the ``lengths`` [batch] tokens of each request's
    pages in pool cells ``cells`` (host; a cell may be listed more than once).
    Query head h * g + r reads KV head h (g = query heads / KV heads, 1 to 16).
    With cur_k, cur_v [listed cells, batch, KV heads, head dim], the last token
    of every request is read from them instead of its page, for all listed
    cells or those where ``current`` (host, one truth value per listed cell) is
    true.  Returns out in q's dtype and shape; ``lse`` (fp32 [listed cells,
    batch, query heads]) receives the natural-log sum of exponentials.  A
    request without tokens gives zeros and -infinity."""
    where = "paged_decode"
    if stream is None:
        got = _paged.paged_decode(cells, q, k_pages, v_pages, table, lengths, meta, cur_k, cur_v, current, out,
                                  lse, sm_scale, status)
        if type(got) is not int:
            return got
        if got != _NOT_PLAIN:
            _check(got, "loopkv_paged_decode")
    pool, dtype, index = _pool(k_pages, v_pages, meta, where)
    cells = _cells(cells, where)
    batch, width = _shape(table, where, "table", 2)
    n_cells, heads, dim = cells.size, pool.n_kv_heads, pool.head_dim
    qr = _rows(q, where, "q", dtype, index, (n_cells, batch, None, dim))
    q_heads = q.shape[2]
    if heads < 1 or q_heads % heads or not 1 <= q_heads // heads <= _lk.LOOPKV_MAX_PAGED_GROUP:
        raise _invalid(where, "%d query heads on %d KV heads: 1 to %d each" % (
            q_heads, heads, _lk.LOOPKV_MAX_PAGED_GROUP))
    d_table = _ints(table, where, "table", index, (batch, width))
    d_len = _ints(lengths, where, "lengths", index, (batch,))
    kr = vr = flags = None
    if (cur_k is None) != (cur_v is None):
        raise _invalid(where, "cur_k and cur_v come together")
    if current is not None:
        flags = np.asarray(current).astype(bool).reshape(-1)  # (not by way of 8 bits: 256 is true)
        if flags.size != n_cells:
            raise _invalid(where, "current must hold %d values, not %d" % (n_cells, flags.size))
        if cur_k is None and flags.any():
            raise _invalid(where, "cur_k and cur_v are required where current is true")
        flags = flags.tobytes()
    if cur_k is not None:
        kr = _rows(cur_k, where, "cur_k", dtype, index, (n_cells, batch, heads, dim))
        vr = _rows(cur_v, where, "cur_v", dtype, index, (n_cells, batch, heads, dim))
        if flags is None:
            flags = b"\1" * n_cells
    group = q_heads // heads
    desc = _lk.loopkv_paged_desc(batch, width, group, float(sm_scale))
    if sm_scale > 0 and desc.sm_scale == 0:  # (0 would mean 1 / sqrt(head dim))
        raise _invalid(where, "sm_scale %r is 0 in fp32" % sm_scale)
    d_status = None if status is None else _ints(status, where, "status", index, (1,))
    d_out = None if out is None else _full(out, where, "out", dtype, index, q.shape)
    d_lse = None if lse is None else _full(lse, where, "lse", _F32, index, q.shape[:3])
    nbytes = _work_bytes(batch, width, group, pool.n_cells, pool.n_pages, pool.page_size, heads, dim, pool.format)
    handle, context = _place(where, index, stream)

    def launch():  # memory made here belongs to the stream of the launch
        work = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        got = torch.empty(q.shape, dtype=dtype, device=q.device) if out is None else out
        rc = _lk.loopkv_paged_decode(
            pool, desc, cells.tobytes(), flags, n_cells, d_table, d_len, qr, kr, vr,
            got.data_ptr() if d_out is None else d_out, d_lse, work.data_ptr(), nbytes, d_status, handle)
        if rc:
            _check(rc, "loopkv_paged_decode")
        return got

    if context is None:
        return launch()
    with context:
        return launch()


class PagedCache:
    """The pages, block table, lengths and free list of one looped model's
    cache.  Cells are loop-major (cell = loop * n_layers + layer); those in
    ``shared`` (non-final loops only) store nothing and read the final loop's
    pages of their layer with their own current token.  ``dtype``: torch
    dtype of the pages (torch.uint8: 8-bit codes with scales)."""

    def __init__(self, n_loops, n_layers, n_kv_heads, head_dim, n_pages, page_size, max_batch,
                 max_pages, shared=(), dtype=None, sm_scale=0.0, device="cuda"):
        where = "PagedCache"
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _FORMATS:
            raise _invalid(where, "pages of %s" % dtype)
        if n_loops < 1 or n_layers < 1:
            raise _invalid(where, "%d loops of %d layers" % (n_loops, n_layers))
        if not 1 <= max_batch <= _lk.LOOPKV_MAX_PAGED_BATCH or max_pages < 1 or \
                max_pages * page_size > _lk.LOOPKV_MAX_PAGED_TOKENS:
            raise _invalid(where, "%d requests of %d pages of %d tokens" % (
                max_batch, max_pages, page_size))
        self.n_loops, self.n_layers, self.n_cells = n_loops, n_layers, n_loops * n_layers
        self.page_size, self.sm_scale = page_size, float(sm_scale)
        self.shared = np.zeros(self.n_cells, bool)
        shared = np.asarray(list(shared))
        if shared.dtype.kind == "b":
            raise _invalid(where, "shared must be a list of cells, not of truth values")
        for cell in _to_int32(shared, where):
            if not 0 <= cell < self.n_cells - n_layers:
                raise _invalid(where, "cell %d cannot share: only cells of non-final loops" % cell)
            self.shared[cell] = True
        # the pool cell of every cell: its own, or its layer's in the final loop
        stored = np.cumsum(~self.shared, dtype=np.int32) - 1
        final = np.tile(stored[self.n_cells - n_layers:], n_loops)
        self.pool_cell = np.where(self.shared, final, stored).astype(np.int32)
        self.store_cell = np.where(self.shared, -1, stored).astype(np.int32)
        shape = (int(stored[-1]) + 1, n_pages, n_kv_heads, page_size, head_dim)
        self.k_pages = torch.zeros(shape, dtype=dtype, device=device)
        self.v_pages = torch.zeros(shape, dtype=dtype, device=device)
        self.meta = None
        if dtype == torch.uint8:
            self.meta = torch.zeros(shape[:4] + (4,), dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((max_batch, max_pages), -1, **i32)
        self.lengths = torch.zeros(max_batch, **i32)
        self.free = torch.arange(n_pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), n_pages, **i32)
        self.starts = torch.zeros(max_batch + 1, **i32)
        self.newest = torch.full((max_batch,), -1, **i32)
        self.status = torch.zeros(1, **i32)

    def _listed(self, cells, where):
        cells = _cells(cells, where)
        if cells.min() < 0 or cells.max() >= self.n_cells:
            raise _invalid(where, "cells are 0 .. %d" % (self.n_cells - 1))
        return cells

    def grow(self, n_new, slots, stream=None):
        """Room for n_new (int32 [max_batch] on the device) tokens per request;
        fills slots (int32 [rows] on the device), ``starts`` and ``newest``;
        returns slots."""
        return page_map(self.lengths, n_new, self.table, self.free, self.free_count,
                        self.page_size, slots, self.starts, newest=self.newest,
                        status=self.status, stream=stream)[0]

    def cut(self, new_lengths, stream=None):
        """Cut every request to new_lengths (int32 [max_batch] on the device)."""
        page_release(self.lengths, new_lengths, self.table, self.free, self.free_count,
                     self.page_size, status=self.status, stream=stream)

    def append(self, cells, k, v, slots, stream=None):
        """k, v [cells, rows, KV heads, head dim] to ``slots``; shared cells keep nothing."""
        cells = self._listed(cells, "PagedCache.append")
        paged_append(self.store_cell[cells], k, v, slots, self.k_pages, self.v_pages, self.meta,
                     status=self.status, stream=stream)

    def decode(self, cells, q, cur_k=None, cur_v=None, out=None, lse=None, stream=None):
        """q [cells, max_batch, query heads, head dim]; cur_k, cur_v [cells,
        max_batch, KV heads, head dim] are needed if a listed cell is shared."""
        where = "PagedCache.decode"
        cells = self._listed(cells, where)
        current = self.shared[cells]
        if current.any() and (cur_k is None or cur_v is None):
            raise _invalid(where, "shared cells read their current token: cur_k and cur_v")
        return paged_decode(self.pool_cell[cells], q, self.k_pages, self.v_pages, self.table,
                            self.lengths, meta=self.meta, cur_k=cur_k, cur_v=cur_v,
                            current=current, out=out, lse=lse, sm_scale=self.sm_scale,
                            status=self.status, stream=stream)

    def check(self, stream=None):
        """Wait for ``stream``, read and clear the status word; raises
        LoopKVError (LOOPKV_ERR_CAPACITY if requests were refused for want of
        room, else LOOPKV_ERR_DEVICE) when it is not 0."""
        with torch.cuda.stream(stream):
            bits = int(self.status.item())
            if bits:
                self.status.zero_()
        if bits:
            room = _lk.LOOPKV_PAGE_NO_TABLE | _lk.LOOPKV_PAGE_NO_ROWS | _lk.LOOPKV_PAGE_NO_PAGES
            raise _lk.LoopKVError(6 if bits & ~room else 3, "PagedCache status 0x%x" % bits)
