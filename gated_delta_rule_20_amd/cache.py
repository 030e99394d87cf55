"""Pages of a state cache (``kda_cache_*``): copying, forking, freeing and compacting.

A page is one entry along the first axis of every pool (a recurrent state, its
convolution state, ...; any dtype and page shape).  ``refcount`` [n_pages] int32
counts how many page-table entries hold each page (a page is free when it is not
above 0); ``table`` [rows, per_row] int32 lists each sequence's pages in order, -1
where there is none.  The last page of a row is the one still being written, those
before it are read only.

Every call also takes ``stream`` (a torch.cuda.Stream; None: the current one).
"""
from __future__ import annotations

import torch

from . import CACHE_MAX_POOLS, CachePool, _dev
from .linear import _call, _check_tensors, _on_stream, _required


def _pools(dst, src=None):
    """ctypes view of a tensor or a list of tensors [n_pages, ...]; with src, pairs of pools with equal pages.
    Returns (array, count, n_dst_pages, n_src_pages, device)."""
    dst = [dst] if isinstance(dst, torch.Tensor) else list(dst)
    src = dst if src is None else [src] if isinstance(src, torch.Tensor) else list(src)
    if not 1 <= len(dst) <= CACHE_MAX_POOLS or len(src) != len(dst):
        raise ValueError(f"need 1..{CACHE_MAX_POOLS} pools and as many sources, got {len(dst)} and {len(src)}")
    arr = (CachePool * len(dst))()
    for i, (d, s) in enumerate(zip(dst, src)):
        if d is None or s is None:
            raise ValueError(f"pool {i} must be a device tensor")
        _dev(d, "pool")
        if d.device != dst[0].device:
            raise ValueError(f"pool {i} is on another device than the first")
        if s is not d:
            _check_tensors(d.device, d.dtype, source_pool=s)
        if d.dim() < 1 or s.dim() < 1 or d.shape[1:] != s.shape[1:]:
            raise ValueError(f"pool {i}: pages of {tuple(d.shape[1:])} and {tuple(s.shape[1:])}")
        if d.shape[0] != dst[0].shape[0] or s.shape[0] != src[0].shape[0]:
            raise ValueError("all pools of a call must have the same number of pages")
        page = d.element_size()
        for n in d.shape[1:]:
            page *= n
        if page == 0:
            raise ValueError(f"pool {i} has empty pages")
        arr[i].dst, arr[i].src, arr[i].page_bytes = d.data_ptr(), s.data_ptr(), page
    n_dst, n_src = dst[0].shape[0], src[0].shape[0]
    if n_dst == 0 or n_src == 0:
        raise ValueError("pools without pages")
    return arr, len(dst), n_dst, n_src, dst[0].device


def _list(t, name, device):
    _required(device, torch.int32, **{name: t})
    if t.dim() != 1:
        raise ValueError(f"{name} must be a 1-d int32 tensor")
    return t.shape[0]


def _tables(table, refcount, device, n_pages=None):
    _required(device, torch.int32, table=table, refcount=refcount)
    if table.dim() != 2:
        raise ValueError(f"table must be [rows, per_row], got {tuple(table.shape)}")
    if refcount.dim() != 1 or (n_pages is not None and refcount.shape[0] != n_pages):
        raise ValueError(f"refcount must be [n_pages]{'' if n_pages is None else f' = [{n_pages}]'}, "
                         f"got {tuple(refcount.shape)}")


@_on_stream
def cache_copy(pools, src_pools, dst_pages, src_pages) -> None:
    """Copy page src_pages[i] of every source pool to page dst_pages[i] of its pool.

    pools / src_pools: a tensor or a list of tensors [n_pages, ...] (src_pools None: within the pools).  Pairs with
    a page out of range are skipped; of several pairs with one destination the last counts.  Within one pool a page
    must not be both a source and a destination."""
    arr, n_pools, n_dst, n_src, device = _pools(pools, src_pools)
    n = _list(dst_pages, "dst_pages", device)
    if _list(src_pages, "src_pages", device) != n:
        raise ValueError("dst_pages and src_pages must have the same length")
    _call("kda_cache_copy", (arr, n_pools, n_dst, n_src, dst_pages.data_ptr(), src_pages.data_ptr(), n), device)


@_on_stream
def cache_fork(pools, table, refcount, parents, children):
    """Make row children[i] of the table a continuation of row parents[i].

    The child shares the parent's pages except the last, which is copied to a free page of its own (the i-th fork
    that needs a page takes the i-th lowest free one).  The child's old row is overwritten: free it first.  table and
    refcount are updated in place.  Returns new_pages [n] int32: each child's own page, or -1 where there is none (an
    empty parent, no page left, a row out of range, a child that is a parent or named before)."""
    arr, n_pools, n_pages, _, device = _pools(pools)
    _tables(table, refcount, device, n_pages)
    n = _list(parents, "parents", device)
    if _list(children, "children", device) != n:
        raise ValueError("parents and children must have the same length")
    pages = torch.empty((2, n), dtype=torch.int32, device=device)
    _call("kda_cache_fork", (arr, n_pools, n_pages, table.data_ptr(), table.shape[0], table.shape[1], refcount.data_ptr(),
                             parents.data_ptr(), children.data_ptr(), n, pages.data_ptr(), pages.data_ptr() + 4 * n), device)
    return pages[1]


@_on_stream
def cache_free(table, refcount, rows) -> None:
    """Give up the pages of the named rows: their counts fall by one (not below 0) and the rows become -1."""
    if table is None:
        raise ValueError("table must be a device tensor")
    _dev(table, "table", torch.int32)
    _tables(table, refcount, table.device)
    n = _list(rows, "rows", table.device)
    _call("kda_cache_free", (table.data_ptr(), table.shape[0], table.shape[1], refcount.data_ptr(), refcount.shape[0], rows.data_ptr(),
                             n), table.device)


@_on_stream
def cache_compact(pools, table, refcount):
    """Move the live pages to the front of the pools; table and refcount follow, in place.

    Live pages below their number stay, and the i-th live page behind it moves to the i-th free page before it.
    Returns (moved_to [n_pages] int32: each page's new place, -1 for a free one; n_live [1] int32), both on the
    device."""
    arr, n_pools, n_pages, _, device = _pools(pools)
    _tables(table, refcount, device, n_pages)
    buf = torch.empty(2 * n_pages + 2, dtype=torch.int32, device=device)
    at = buf.data_ptr()
    _call("kda_cache_compact", (arr, n_pools, n_pages, table.data_ptr(), table.shape[0], table.shape[1], refcount.data_ptr(), at,
                                at + 4 * n_pages, at + 8 * n_pages), device)
    return buf[:n_pages], buf[2 * n_pages:2 * n_pages + 1]
