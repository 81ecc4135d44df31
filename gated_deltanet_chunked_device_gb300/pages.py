"""Pages of a cache: reserve, fork, free, compact and copy, without a host round trip.

A page is one row of every buffer of the cache: of the state pools that ``state_indices`` addresses, or of a key/value
cache's blocks of tokens.  ``table`` [sequences, max_pages] int32 names each sequence's pages (-1: none; one column for
states), ``refcounts`` [pages] int32 counts the entries that name a page (0: free), ``lengths`` [sequences] int32 holds
tokens.  All of it is device memory that the caller owns.  The calls marshal arguments for the C ABI
(``include/gdn_pages.h``), which fixes every choice: free pages are given out lowest first, in the list's order.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch
from torch.autograd.graph import increment_version

from . import GdnError, lib, on_device

__all__ = ["cache_reserve", "cache_fork", "cache_free", "cache_compact", "cache_copy", "PAGES_ERR", "PagesBook", "PagesBuffer"]

PAGES_ERR = {"SEQ": 1 << 8, "CHILD": 1 << 9, "PAGE": 1 << 10, "NO_PAGES": 1 << 11}
MAX_BUFFERS = 128


class PagesBook(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("refcounts", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


class PagesBuffer(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("row_bytes", ctypes.c_int64)]


_pack_book = struct.Struct("@PPPiii4x").pack  # the bytes of a PagesBook
_buffer_packs = [struct.Struct("@" + "Pqq" * n).pack for n in range(MAX_BUFFERS + 1)]  # and of n PagesBuffers


def _register(L):
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L.gdn_pages_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.gdn_pages_workspace_bytes.restype = sz
    L.gdn_pages_reserve_run.argtypes = [vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.gdn_pages_fork_run.argtypes = [vp, vp, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
    L.gdn_pages_free_run.argtypes = [vp, vp, i32, vp, vp]
    L.gdn_pages_compact_run.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gdn_pages_copy_run.argtypes = [vp, i32, vp, i32, i32, vp, vp, i32, vp, vp]
    for fn in (L.gdn_pages_reserve_run, L.gdn_pages_fork_run, L.gdn_pages_free_run, L.gdn_pages_compact_run, L.gdn_pages_copy_run):
        fn.restype = ctypes.c_int


def _int32(name, t, shape, device):
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)} on cuda:{device}")
    return t.data_ptr()


def _book(table, refcounts, lengths):
    """Checks the bookkeeping; returns (device, packed book, sequences, pages a sequence, pages)."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor: this library has no CPU path")
    if table.dim() != 2 or refcounts.dim() != 1:
        raise ValueError("table must be [sequences, max_pages] and refcounts [pages]")
    device = table.get_device()
    S, M = table.shape
    P, = refcounts.shape
    return device, _pack_book(_int32("table", table, (S, M), device), _int32("refcounts", refcounts, (P,), device),
                              0 if lengths is None else _int32("lengths", lengths, (S,), device), S, M, P), S, M, P


def _as_list(pools):
    return (pools,) if isinstance(pools, torch.Tensor) else pools


def _buffers(name, pools, n_pages, device):
    """Checks the buffers; returns them packed, and how many."""
    pools = _as_list(pools)
    if len(pools) > MAX_BUFFERS:
        raise ValueError(f"at most {MAX_BUFFERS} buffers")
    out = []
    for t in pools:
        if t.get_device() != device or t.dim() < 1 or t.shape[0] != n_pages:
            raise ValueError(f"{name} must be [{n_pages}, ...] on cuda:{device}")
        size = t.element_size()
        if t.is_contiguous():
            row = stride = t.numel() // n_pages * size if n_pages else 0
        else:
            row = 1
            for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
                if n > 1 and s != row:
                    raise ValueError(f"{name} must have contiguous rows")
                row *= n
            if n_pages > 1 and t.stride(0) < row:
                raise ValueError(f"{name}'s rows must not overlap")
            stride, row = max(t.stride(0), row) * size, row * size
        out += (t.data_ptr(), stride, row)
    return _buffer_packs[len(pools)](*out), len(pools)


def _status(device_status, device):
    if device_status is None:
        return 0
    if not device_status.numel():
        raise ValueError("device_status must have an element")
    return _int32("device_status", device_status, device_status.shape, device)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(bounds):
    return lib().gdn_pages_workspace_bytes(*bounds)


def _call(name, like, args, workspace=None):
    """Calls an entry point on `like`'s device and the caller's stream; workspace: the bounds to take one for.  What it changes
    in place its caller tells autograd (increment_version), so that a backward pass that saved it refuses to go on."""
    with on_device(like.get_device()) as stream:
        if workspace is None:
            st = getattr(lib(), name)(*args, stream)
        else:
            n = _workspace_bytes(workspace)
            ws = torch.empty(n, dtype=torch.uint8, device=like.device)
            st = getattr(lib(), name)(*args, ws.data_ptr(), n, stream)
    if st != 0:
        raise GdnError(st, name)


def cache_reserve(table, refcounts, seqs, counts, device_status=None):
    """Gives sequence ``seqs[k]`` pages for its table entries 0 .. ``counts[k]`` - 1 that have none.  Returns the
    sequences' table rows [n, max_pages] (with one page a sequence: the new ``state_indices``).  The first sequence for
    which the free pages do not suffice, and those after it, get nothing (PAGES_ERR["NO_PAGES"])."""
    device, book, S, M, P = _book(table, refcounts, None)
    n = seqs.numel()
    rows = torch.empty(n, M, dtype=torch.int32, device=table.device)
    _call("gdn_pages_reserve_run", table, (book, _int32("seqs", seqs, (n,), device), _int32("counts", counts, (n,), device), n,
                                           rows.data_ptr(), _status(device_status, device)), (S, M, P, n))
    increment_version((table, refcounts))
    return rows


def cache_fork(pools, table, refcounts, parents, children, page_tokens=0, lengths=None, device_status=None):
    """Makes ``children[k]``, which has no pages, a copy of ``parents[k]``.  With ``page_tokens`` (tokens of a page, which
    do not change once written) the pages that ``lengths`` says are full are shared and a partly filled last one is copied;
    with 0 (states, which every step overwrites) every page is copied, in every buffer of ``pools``.  ``lengths``, when
    given, is carried over.  Returns the children's table rows [n, max_pages]."""
    device, book, S, M, P = _book(table, refcounts, lengths)
    if page_tokens and lengths is None:
        raise ValueError("page_tokens needs lengths")
    if page_tokens > 0x7fffffff:
        raise ValueError("page_tokens must fit 32 bits")
    n = children.numel()
    bufs, nb = _buffers("pools", pools, P, device)
    rows = torch.empty(n, M, dtype=torch.int32, device=table.device)
    _call("gdn_pages_fork_run", table, (book, bufs, nb, _int32("parents", parents, (n,), device),
                                        _int32("children", children, (n,), device), n, int(page_tokens), rows.data_ptr(),
                                        _status(device_status, device)), (S, M, P, n))
    increment_version((table, refcounts, *_as_list(pools)) if lengths is None else (table, refcounts, lengths, *_as_list(pools)))
    return rows


def cache_free(table, refcounts, seqs, lengths=None, device_status=None):
    """Drops the sequences: a reference less on each of their pages, table entries -1, lengths 0."""
    device, book, _, _, _ = _book(table, refcounts, lengths)
    n = seqs.numel()
    _call("gdn_pages_free_run", table, (book, _int32("seqs", seqs, (n,), device), n, _status(device_status, device)))
    increment_version((table, refcounts) if lengths is None else (table, refcounts, lengths))


def cache_compact(pools, table, refcounts, table_out=None, refcounts_out=None, device_status=None):
    """Moves the live pages into the first rows of every buffer.  Returns ``(remap, n_live)``: each page's new index (-1
    for a free one) and the number of live pages [1], both on the device.  The bookkeeping is changed in place, or written
    to ``table_out`` and ``refcounts_out``: then the old one stays valid, since only free pages are written."""
    device, book, S, M, P = _book(table, refcounts, None)
    table_out = table if table_out is None else table_out
    refcounts_out = refcounts if refcounts_out is None else refcounts_out
    bufs, nb = _buffers("pools", pools, P, device)
    remap = torch.empty_like(refcounts)
    n_live = torch.empty(1, dtype=torch.int32, device=refcounts.device)
    _call("gdn_pages_compact_run", table, (book, bufs, nb, _int32("table_out", table_out, (S, M), device),
                                           _int32("refcounts_out", refcounts_out, (P,), device), remap.data_ptr(),
                                           n_live.data_ptr(), _status(device_status, device)), (S, M, P, 0))
    increment_version((table_out, refcounts_out, *_as_list(pools)))
    return remap, n_live


def cache_copy(src_pools, dst_pools, src, dst, device_status=None):
    """Row ``src[i]`` of each buffer of ``src_pools`` to row ``dst[i]`` of the buffer of the same place in ``dst_pools``
    (checkpoints into a state pool, for one); pairs with a negative index are skipped.  No row is named twice in ``dst``,
    and none is both read and written."""
    src_pools, dst_pools = _as_list(src_pools), _as_list(dst_pools)
    if len(src_pools) != len(dst_pools):
        raise ValueError("src_pools and dst_pools must have as many buffers")
    if not src_pools:
        return
    device = src_pools[0].get_device()
    if device < 0:
        raise ValueError("the pools must be CUDA tensors: this library has no CPU path")
    for s, d in zip(src_pools, dst_pools):
        if s.dtype is not d.dtype or s.shape[1:] != d.shape[1:]:
            raise ValueError("a source and its destination must have rows of one type and shape")
    n_src, n_dst, n = src_pools[0].shape[0], dst_pools[0].shape[0], src.numel()
    sb, nb = _buffers("src_pools", src_pools, n_src, device)
    db, _ = _buffers("dst_pools", dst_pools, n_dst, device)
    _call("gdn_pages_copy_run", src_pools[0], (sb, n_src, db, n_dst, nb, _int32("src", src, (n,), device),
                                               _int32("dst", dst, (n,), device), n, _status(device_status, device)))
    increment_version(dst_pools)
