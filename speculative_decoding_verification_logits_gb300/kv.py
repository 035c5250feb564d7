"""Binding of the page operators of a paged KV cache (C ABI in ``include/sd_kv.h``): forking and
extending block tables, giving pages back, copying pages and moving the pages in use to the
front of the pool.  kv_rollback truncates the same tables.

A pool of N pages is refs [N] (int32): how many table entries hold each page; 0 is a free page.
Like the rest of the package this module only checks and marshals arguments; every call takes
stream= as well, and runs on the current stream without it.

  kv_fork(...), kv_extend(...)   sd_kv_fork
  kv_free(...)                   sd_kv_free
  kv_compact(...)                sd_kv_compact
  kv_copy(...)                   sd_kv_copy
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
from typing import NamedTuple

import torch

from . import _P, _check, _need
from .logits import _lib, _stream_of, _written

SD_STATUS_BAD_PARENT, SD_STATUS_BAD_PAGE, SD_STATUS_NO_PAGE = 0x10, 0x20, 0x40
SD_MAX_ROWS, SD_MAX_PAGES, SD_MAX_CACHES = 16384, 1 << 24, 256

_I32, _U8 = torch.int32, torch.uint8


class ForkArgs(ctypes.Structure):
    """Mirror of ``sd_kv_fork_args`` in include/sd_kv.h."""
    _fields_ = [
        *((n, ctypes.c_int32) for n in ("rows_in", "R", "groups", "max_pages", "page_size",
                                        "append", "keep", "N")),
        ("parents", _P), ("table", _P), ("kv_len", _P), ("refs", _P), ("table_out", _P),
        ("len_out", _P), ("src", _P), ("dst", _P), ("fill", _P), ("count", _P), ("status", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
    ]


class CopyArgs(ctypes.Structure):
    """Mirror of ``sd_kv_copy_args`` in include/sd_kv.h."""
    _fields_ = [
        *((n, ctypes.c_int32) for n in ("n_caches", "layers", "N", "parts", "page_size")),
        ("entry_bytes", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
        ("page_stride", ctypes.c_int64), ("caches", _P), ("pairs", ctypes.c_int32), ("src", _P),
        ("dst", _P), ("fill", _P), ("count", _P), ("status", _P),
    ]


class KVFork(NamedTuple):
    """Outputs that a call makes lie, with its scratch, in one block of memory: who keeps one of them
    keeps the block.  So do those of KVMoves and KVCompact."""
    block_table: torch.Tensor   # [R][max_pages] int32
    kv_len: torch.Tensor        # [R] int32
    src: torch.Tensor           # [R] int32: pages to copy from, -1 after the last
    dst: torch.Tensor           # [R] int32: and to
    fill: torch.Tensor          # [R] int32: entries of each to copy
    count: torch.Tensor         # [1] int32: how many pairs


class KVMoves(NamedTuple):
    src: torch.Tensor
    dst: torch.Tensor
    fill: torch.Tensor
    count: torch.Tensor


class KVCompact(NamedTuple):
    src: torch.Tensor           # [N // 2] int32: pages that move, -1 after the last
    dst: torch.Tensor           # [N // 2] int32: where to
    count: torch.Tensor         # [1] int32: how many
    new_ids: torch.Tensor       # [N] int32: where each page in use is now, -1: free
    live: torch.Tensor          # [1] int32: pages in use, now [0, live)


def _bind(L):
    """Argument types of the entry points, and the structs' layouts."""
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.sd_kv_fork.argtypes = [ctypes.POINTER(ForkArgs), _P]
    L.sd_kv_copy.argtypes = [ctypes.POINTER(CopyArgs), _P]
    L.sd_kv_free.argtypes = [i64, i64, _P, _P, _P, i32, i32, _P, _P, _P]
    L.sd_kv_compact.argtypes = [i32, _P, i64, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]
    for fn in (L.sd_kv_fork, L.sd_kv_copy, L.sd_kv_free, L.sd_kv_compact):
        fn.restype = ctypes.c_int
    L.sd_kv_fork_workspace_size.argtypes = [i32, i32, i32]
    L.sd_kv_compact_workspace_size.argtypes = [i32]
    L.sd_kv_fork_workspace_size.restype = L.sd_kv_compact_workspace_size.restype = sz
    for fn, mirror in ((L.sd_kv_fork_args_size, ForkArgs), (L.sd_kv_copy_args_size, CopyArgs)):
        fn.argtypes, fn.restype = [], sz
        if fn() != ctypes.sizeof(mirror):
            raise RuntimeError(f"{mirror.__name__} layout differs between library and binding")


_device = torch._C._cuda_getDevice   # the current one's index


def _on_device(fn):
    """Runs a wrapper with the device of its first parameter, however that is passed, as the current
    one, and with `stream` (when given) as the current stream: what it allocates belongs to the
    stream that it launches on."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        t = args[0] if args else kwargs.get(first)
        if t is not None and not isinstance(t, (torch.Tensor, list, tuple)):
            t = tuple(t)   # looked at here and by the wrapper
            if args:
                args = (t, *args[1:])
            else:
                kwargs[first] = t
        while isinstance(t, (list, tuple)) and t:
            t = t[0]
        there = isinstance(t, torch.Tensor) and t.is_cuda   # if not, the wrapper says what is wrong
        if stream is not None:
            if there and stream.device != t.device:
                raise ValueError(f"stream is on {stream.device}, expected {t.device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kwargs)
        if there and t.get_device() != _device():
            with torch.cuda.device(t.device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return call


def _i32(t, name, shape, device):
    """The address of a contiguous int32 array; what is wrong with it is said by _need."""
    if t is None or t.dtype is not _I32 or t.device != device or t.shape != shape \
            or not t.is_contiguous():
        _need(t, name, _I32, shape, device)
    return t.data_ptr()


def _span(t):
    """The addresses that a tensor reaches over, or none."""
    n, at = t.numel(), t.data_ptr()
    if not n:
        return 0, 0
    if not t.is_contiguous():
        n = 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return at, at + t.element_size() * n


def _meet(a, b):
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _rows_meet(a, b, lead):
    """Whether two tensors whose rows (all dimensions from `lead` on) are contiguous share a byte:
    rows of one may lie between those of the other."""
    if not _meet(a, b):
        return False

    def starts(t):   # the rows' addresses, and their bytes
        at = torch.tensor(t.data_ptr(), device="cpu")
        for n, s in zip(t.shape[:lead], t.stride()[:lead]):
            at = at[..., None] + torch.arange(n, device="cpu") * (s * t.element_size())
        return at.flatten().sort().values, math.prod(t.shape[lead:]) * t.element_size()

    (x, nx), (y, ny) = starts(a), starts(b)
    return bool((torch.searchsorted(y, x + nx) > torch.searchsorted(y, x - ny, right=True)).any())


def _lie_apart(size, *dims):
    """Whether pieces of `size` bytes, (how many, bytes between them) along each dimension, share no
    byte with one another."""
    reach = size
    for s, n in sorted((s, n) for n, s in dims if n > 1):
        if s < reach:
            break
        reach += s * (n - 1)
    else:
        return True
    at = torch.zeros((), dtype=torch.int64, device="cpu")
    for n, s in dims:   # dimensions that lie between one another
        at = at[..., None] + torch.arange(n, device="cpu") * s
    return not bool((at.flatten().sort().values.diff() < size).any())


def _all_apart(outs, *inputs):
    """Refuses outputs that share memory with an input or with one another (contiguous ones)."""
    for i, t in enumerate(outs):
        if any(_meet(t, x) for x in inputs if x is not None):
            raise ValueError("out overlaps the input")
        if any(_meet(t, x) for x in outs[:i]):
            raise ValueError("outputs overlap")


def _pool(refs, device):
    shape = refs.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError("refs must be [N], with N >= 1")
    return _i32(refs, "refs", shape, device), shape[0]


def _table(block_table, kv_len):
    dev, shape = block_table.device, block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [rows][max_pages]")
    return (*shape, _i32(block_table, "block_table", shape, dev if block_table.is_cuda else None),
            _i32(kv_len, "kv_len", shape[:1], dev), dev)


@functools.lru_cache(256)
def _scratch(which, device, *sizes):
    """int32s of scratch that a call needs on a device (by index).  It lies beside the call's
    outputs, in one block of the allocator's (an allocation less per array, 1.5 to 3 us on the host
    each): calls and captured graphs share none."""
    n = getattr(_lib(), which)(*sizes)
    if n == 0:
        raise ValueError("sizes out of range")
    return (n + 15) // 16 * 4


def _small(*numbers):
    """Refuses numbers that would wrap around on their way into the library's int32."""
    for n in numbers:
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{n} is out of range")


def _apart(what, at, n, *others):
    """Refuses n int32s at an address, which a call writes, where they share memory with other
    arguments: (address or None, bytes)."""
    if at is None or not n:
        return
    end = at + 4 * n
    for other, size in others:
        if other is not None and size and other < end and at < other + size:
            raise ValueError(f"{what} overlaps another argument")


def _fork(a, refs, status, dev, sizes):
    """Runs sd_kv_fork with new outputs of these sizes (in the struct's order) where there are
    any; returns them."""
    ref, N = _pool(refs, dev)
    a.refs, a.N = ref, N
    st = None
    if status is not None:
        a.status = st = _i32(status, "status", (1,), dev)
    table, slots, parents = a.table, a.rows_in * a.max_pages, a.parents
    read = (a.kv_len, 4 * a.rows_in), (parents, 4 * a.R)
    _apart("refs", ref, N, (table, 4 * slots), (st, 4), *read)
    _apart("status", st, 1, (table, 4 * slots), *read)
    if parents is None:   # the table is written
        _apart("block_table", table, slots, *read)
    n = _scratch("sd_kv_fork_workspace_size", dev.index, a.rows_in, a.R, a.N)
    sizes = (n, *sizes)
    buf = torch.empty(sum(sizes), dtype=_I32, device=dev)
    at = buf.data_ptr()
    a.workspace, a.workspace_bytes = at, 4 * n
    if len(sizes) > 1:
        at += 4 * n
        if len(sizes) == 7:
            a.table_out, a.len_out = at, at + 4 * sizes[1]
            at += 4 * (sizes[1] + sizes[2])
        R = 4 * a.R
        a.src, a.dst, a.fill, a.count = at, at + R, at + 2 * R, at + 3 * R
    rc = _lib().sd_kv_fork(a, _stream_of(dev))
    if rc:
        _check(rc, "sd_kv_fork")
    _written(refs)
    return buf.unsafe_split_with_sizes(sizes)   # for autograd arrays of their own, in one block


@_on_device
def kv_fork(block_table, kv_len, parents, refs, page_size: int, *, append: int = 0,
            keep: bool = False, out: KVFork | None = None, status=None) -> KVFork:
    """New rows from the rows of block_table [rows][max_pages] and kv_len [rows] (int32): row r
    shares the pages of its parent and has room for `append` more entries; refs [N] is brought
    up to date.  parents: int32 [R], rows of the table, or [B][k] relative to each of B groups of
    rows (beam_select's, for a table of B W rows); -1 makes an empty row.

    The old rows end with the call: pages that no new row holds are given back, and the first
    row of each parent takes over what is the parent's own.  keep=True leaves the old rows as
    they are.  Either way the partly filled last page of every new row is its own: kv_copy(caches,
    f.src, f.dst, count=f.count, fill=f.fill) must follow before the rows are read.

    Where the pool runs out (status: SD_STATUS_NO_PAGE) slots without a page are -1, but the first
    row of a parent that ends keeps a shared last page, to be copied by kv_extend once pages are
    free."""
    rows, M, table, lens, dev = _table(block_table, kv_len)
    shape = parents.shape
    if len(shape) not in (1, 2):
        raise ValueError("parents must be [R] or [B][k]")
    R = parents.numel()
    if R == 0:
        raise ValueError("parents must name at least one row")
    _small(page_size, append)
    groups = shape[0] if len(shape) == 2 else 0
    if groups and rows % groups:
        raise ValueError(f"{rows} rows are not {groups} groups")
    a = ForkArgs(rows, R, groups, M, page_size, append, bool(keep))
    a.parents, a.table, a.kv_len = _i32(parents, "parents", shape, dev), table, lens
    if out is None:
        _, t, n, src, dst, fill, count = _fork(a, refs, status, dev, (R * M, R, R, R, R, 1))
        return KVFork(t.view(R, M), n, src, dst, fill, count)
    a.table_out = _i32(out.block_table, "out.block_table", (R, M), dev)
    a.len_out = _i32(out.kv_len, "out.kv_len", (R,), dev)
    a.src, a.dst, a.fill = (_i32(getattr(out, n), "out." + n, (R,), dev)
                            for n in ("src", "dst", "fill"))
    a.count = _i32(out.count, "out.count", (1,), dev)
    _all_apart(out, block_table, kv_len, parents, refs, status)
    _fork(a, refs, status, dev, ())
    for t in out:
        _written(t)
    return out


@_on_device
def kv_extend(block_table, kv_len, refs, page_size: int, append: int, *, status=None) -> KVMoves:
    """Room for `append` more entries in every row of block_table, in place: its rows get free
    pages, and a partly filled last page that others hold too becomes the row's own (kv_copy of
    the returned pairs must follow where rows may share one).  Where the pool runs out (status:
    SD_STATUS_NO_PAGE) rows keep what they hold: give pages back and call again before they
    are written."""
    rows, M, table, lens, dev = _table(block_table, kv_len)
    _small(page_size, append)
    a = ForkArgs(rows, rows, 0, M, page_size, append, 0)
    a.table = a.table_out = table
    a.kv_len = lens
    m = _fork(a, refs, status, dev, (rows, rows, rows, 1))
    _written(block_table)
    return KVMoves(*m[1:])


@_on_device
def kv_free(pages, refs, *, which=None, count=None, clear: bool = False,
            status=None) -> torch.Tensor:
    """Gives pages back to refs [N], in place: the ids in pages (int32, any shape; -1 is passed
    over), as kv_rollback lists them (pages=freed, count=free_offsets[-1:]), or the rows of a
    block table (which [rows] uint8: those whose flag is set).  clear=True makes the entries that
    are taken -1."""
    dev, shape = pages.device, pages.shape
    p = _i32(pages, "pages", shape, dev if pages.is_cuda else None)
    ref, N = _pool(refs, dev)
    size = pages.numel()
    rows, cols, w, n, st = 1, size, None, None, None
    if which is not None:
        if len(shape) != 2:
            raise ValueError("which needs pages [rows][max_pages]")
        rows, cols = shape
        _need(which, "which", _U8, (rows,), dev)
        w = which.data_ptr() if rows else None
    if count is not None:
        n = _i32(count, "count", (1,), dev)
    if status is not None:
        st = _i32(status, "status", (1,), dev)
    read = (w, rows), (n, 4)
    _apart("refs", ref, N, (p, 4 * size), (st, 4), *read)
    _apart("status", st, 1, (p, 4 * size), *read)
    if clear:
        _apart("pages", p, size, *read)
    rc = _lib().sd_kv_free(rows, cols, p, w, n, bool(clear), N, ref, st, _stream_of(dev))
    if rc:
        _check(rc, "sd_kv_free")
    _written(refs)
    if clear:
        _written(pages)
    return refs


@_on_device
def kv_compact(refs, block_table=None, *, status=None) -> KVCompact:
    """Moves the pages in use to the front of the pool: refs [N] and the entries of block_table
    (int32, any shape) are brought up to date in place; kv_copy(caches, c.src, c.dst,
    count=c.count) must follow before the pages are read.  Other tables of the same pool take
    their ids from new_ids."""
    dev = refs.device
    ref, N = _pool(refs, dev if refs.is_cuda else None)
    table, n_table, st = None, 0, None
    if block_table is not None:
        p = _i32(block_table, "block_table", block_table.shape, dev)
        n_table = block_table.numel()
        table = p if n_table else None
    if status is not None:
        st = _i32(status, "status", (1,), dev)
    _apart("refs", ref, N, (table, 4 * n_table), (st, 4))
    _apart("status", st, 1, (table, 4 * n_table))
    n, h = _scratch("sd_kv_compact_workspace_size", dev.index, N), N // 2
    sizes = (n, h, h, 1, 1, N)
    buf = torch.empty(sum(sizes), dtype=_I32, device=dev)
    ws = buf.data_ptr()
    src = ws + 4 * n
    count = src + 8 * h
    rc = _lib().sd_kv_compact(N, ref, n_table, table, src, src + 4 * h, count, count + 4,
                              count + 8, st, ws, 4 * n, _stream_of(dev))
    if rc:
        _check(rc, "sd_kv_compact")
    _written(refs)
    if n_table:
        _written(block_table)
    _, src, dst, count, live, new = buf.unsafe_split_with_sizes(sizes)
    return KVCompact(src, dst, count, new, live)


def _page_shape(shape, strides, size, first, name):
    """Whether the dimensions from `first` on lie contiguous."""
    want = 1
    for n, s in zip(reversed(shape[first:]), reversed(strides[first:])):
        if n > 1 and s != want:
            raise ValueError(f"{name}: a page must be contiguous")
        want *= n
    return want * size


@_on_device
def kv_copy(caches, src, dst, *, count=None, fill=None, heads_first: bool = False,
            status=None) -> None:
    """Copies page src[i] to page dst[i] (int32 [pairs], the first count [1] of them; -1, -1 is
    passed over) in every cache, in place.  caches: one tensor [layers][N][...] or a sequence of
    [N][...] of one shape (keys and values of every layer), any type.  fill [pairs]: only the
    first fill[i] entries of each page, for pages [page_size][...], or with heads_first
    [heads][page_size][...].  No page may be both a source and a destination, and none twice a
    destination."""
    one = isinstance(caches, torch.Tensor)
    if one:
        base, lead, tensors = caches, 1, (caches,)
    else:
        tensors = tuple(caches)
        if not tensors:
            return
        if len(tensors) > SD_MAX_CACHES:
            raise ValueError(f"at most {SD_MAX_CACHES} caches")
        base, lead = tensors[0], 0
    dev, shape, strides, size = base.device, base.shape, base.stride(), base.element_size()
    if len(shape) < lead + 2:
        raise ValueError("caches must be [layers][N][...], or each of a sequence [N][...]")
    layers = shape[0] if one else 1
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("caches must be CUDA tensors")
        if t is not base and (t.device != dev or t.shape != shape or t.stride() != strides
                              or t.dtype != base.dtype):
            raise ValueError("caches must be alike in shape, type, strides and device")
    if base.is_contiguous():
        page = size * math.prod(shape[lead + 1:])
    else:
        page = _page_shape(shape, strides, size, lead + 1, "caches")
        if not _lie_apart(page, *((shape[d], strides[d] * size) for d in range(lead + 1))):
            raise ValueError("pages of a cache overlap")
    at = lead + 2 if heads_first else lead + 1
    if fill is not None and len(shape) <= at:
        raise ValueError("fill needs pages of [page_size][...], or [heads][page_size][...]")
    parts, entries = 1, 1
    if fill is not None:
        entries = shape[at]
        parts = shape[lead + 1] if heads_first else 1
    if page == 0 or shape[lead] == 0 or layers == 0:
        return
    a = CopyArgs(len(tensors), layers, shape[lead], parts, entries, page // (parts * entries),
                 strides[0] * size if one else 0, strides[lead] * size)
    pointers = (_P * len(tensors))(*(t.data_ptr() for t in tensors))
    a.caches = ctypes.addressof(pointers)
    pairs = src.shape
    if len(pairs) != 1:
        raise ValueError("src must be [pairs]")
    a.pairs = pairs[0]
    a.src, a.dst = _i32(src, "src", pairs, dev), _i32(dst, "dst", pairs, dev)
    if fill is not None:
        a.fill = _i32(fill, "fill", pairs, dev)
    if count is not None:
        a.count = _i32(count, "count", (1,), dev)
    if status is not None:
        a.status = _i32(status, "status", (1,), dev)
    rc = _lib().sd_kv_copy(a, _stream_of(dev))
    if rc:
        _check(rc, "sd_kv_copy")
    for t in tensors:
        _written(t)
