"""Python calls that manage the pages of a cache: copy, fork (beams, samples,
rows that end, grow or begin) and compact.

As in ``_serving``: arguments are checked, then handed to the library; every
call runs on the device its tensors are on, on ``stream`` or that device's
current stream.  ``pools`` are all tensors whose first dimension is the page --
K and V of every layer, scale bytes, block bounds -- in any dtype.
"""
from __future__ import annotations

from array import array
from typing import Optional, Sequence, Tuple

import torch

from ._serving import (_DEVICES, _I32, _NOT_SO, _U8, _Place, _device_of, _int32, _status,
                       _tensor, _vector)


def _check_pools(pools, num_pages: Optional[int], dev: int):
    """The pools one by one."""
    for i, t in enumerate(pools):
        name = f"pools[{i}]"
        if _device_of(t, name) != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the other tensors on "
                             f"cuda:{dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dim() < 2:
            raise ValueError(f"{name} must have pages of some size")
        if t.shape[0] != num_pages and num_pages is not None or t.shape[0] == 0:
            raise ValueError(f"{name} has {t.shape[0]} pages, expected {num_pages}")
        num_pages = t.shape[0]


def _pool_args(pools: Sequence[torch.Tensor], num_pages: Optional[int], dev: int):
    """(pointers, bytes of a page, how many, pages) of the pools, as arrays for the
    library (to be kept until the call returns)."""
    try:
        n = num_pages if num_pages is not None or not pools else pools[0].shape[0]
        sizes = array("Q", [t.nbytes // n for t in pools if t.shape[0] == n and t.dim() > 1
                            and t.is_contiguous() and t.get_device() == dev])
        if len(sizes) == len(pools):
            return array("Q", [t.data_ptr() for t in pools]), sizes, len(pools), n
    except (*_NOT_SO, ZeroDivisionError, IndexError):
        pass
    _check_pools(pools, num_pages, dev)
    raise ValueError("pools must be a sequence of tensors of the same number of pages")


_SIZES: dict = {}  # workspace bytes, by function and sizes: the last few hundred asked for
_SIZES_MOST = 256


def _workspace(given, at: _Place, name: str, *sizes: int) -> Optional[torch.Tensor]:
    """The caller's workspace or a new one; None where none is needed (or the sizes are
    wrong, which the call itself says)."""
    if given is not None:
        _tensor(given, "workspace", (_U8,), 1, at.dev)
        return given
    need = _SIZES.get((name, sizes))
    if need is None:
        need = at.call(name, *sizes)
        if len(_SIZES) >= _SIZES_MOST:
            _SIZES.clear()
        _SIZES[name, sizes] = need
    if need == 0:
        return None
    if at.stream is None:
        return torch.empty(need, dtype=_U8, device=_DEVICES[at.dev])
    return at.empty(need, _U8)


def kv_copy_pages(pools, src, dst, *, count=None, status=None, stream=None) -> None:
    """Copy page src[k] of every pool to its page dst[k].

    src, dst int32 [n] (a pair with a -1 is skipped); no page may be a dst twice,
    or a src and a dst.  count: int32 tensor of one element, only the first
    min(count, n) pairs.
    """
    dev = _device_of(src, "src")
    _tensor(src, "src", (_I32,), 1, dev)
    _vector(dst, "dst", src.shape[0], dev)
    if count is not None:
        _vector(count, "count", 1, dev)
    ptrs, sizes, n_pools, num_pages = _pool_args(pools, None, dev)
    if n_pools == 0:
        return
    _Place(dev, stream).run("tree_kv_copy_pages", ptrs.buffer_info()[0], sizes.buffer_info()[0],
                            n_pools, src.data_ptr(), dst.data_ptr(),
                            None if count is None else count.data_ptr(), src.shape[0], num_pages,
                            _status(status, dev))


def _out(t, name: str, like: torch.Tensor, shape, at: _Place) -> torch.Tensor:
    """An output given by the caller (not the input of its kind), or a new one."""
    if t is None:
        if at.stream is None:
            return torch.empty(shape, dtype=_I32, device=_DEVICES[at.dev])
        return at.empty(shape, _I32)
    _tensor(t, name, (_I32,), len(shape), at.dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.data_ptr() == like.data_ptr() and t.numel() > 0:
        raise ValueError(f"{name} must not be the input of its kind")
    return t


def kv_fork(pools, block_table, seq_lens, page_refs, src, page_size: int, *, reserve=0,
            block_table_out=None, seq_lens_out=None, page_refs_out=None, workspace=None,
            status=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The rows of the next step from the rows of this one.

    Row i of the results continues row src[i] of block_table int32 [rows][max_pages]
    (-1 where there is no page) and seq_lens int32 [rows]; src int32 [rows_out], -2: a
    new row without tokens, -1: no row.  Whole pages are shared; the last one stays with the
    first row that continues a row and is copied, in every pool, for the others;
    every row is mapped for ``reserve`` more tokens (a number, or int32
    [rows_out]).  page_refs int32 [num_pages] counts the table entries (and other
    uses) of each page, 0: free; rows that nobody continues give theirs back.
    Returns (block_table, seq_lens, page_refs) of the new rows; status 6: there
    were not enough free pages.
    """
    try:
        dev = block_table.get_device()
        rows, width = block_table.shape
        (n,), (num_pages,) = src.shape, page_refs.shape
        sound = (dev >= 0 and block_table.dtype is _I32 and seq_lens.dtype is _I32
                 and page_refs.dtype is _I32 and src.dtype is _I32 and seq_lens.shape == (rows,)
                 and seq_lens.get_device() == dev and page_refs.get_device() == dev
                 and src.get_device() == dev and block_table.is_contiguous()
                 and seq_lens.is_contiguous() and page_refs.is_contiguous()
                 and src.is_contiguous())
    except _NOT_SO:
        sound = False
    if not sound:
        dev = _device_of(block_table, "block_table")
        _tensor(block_table, "block_table", (_I32,), 2, dev)
        rows, width = block_table.shape
        _vector(seq_lens, "seq_lens", rows, dev)
        _tensor(page_refs, "page_refs", (_I32,), 1, dev)
        _tensor(src, "src", (_I32,), 1, dev)
        n, num_pages = src.shape[0], page_refs.shape[0]
    more, each = 0, None
    if type(reserve) is int:
        more = reserve
        if more < 0:
            raise ValueError("reserve must not be negative")
    else:
        _vector(reserve, "reserve", n, dev)
        each = reserve.data_ptr()
    _int32(page_size, more)
    ptrs, sizes, n_pools, _ = _pool_args(pools, num_pages, dev)
    at = _Place(dev, stream)
    table = _out(block_table_out, "block_table_out", block_table, (n, width), at)
    lens = _out(seq_lens_out, "seq_lens_out", seq_lens, (n,), at)
    refs = _out(page_refs_out, "page_refs_out", page_refs, (num_pages,), at)
    workspace = _workspace(workspace, at, "tree_kv_fork_workspace_size", rows, n, num_pages)
    at.run("tree_kv_fork", ptrs.buffer_info()[0], sizes.buffer_info()[0], n_pools,
           block_table.data_ptr(), width, seq_lens.data_ptr(), page_refs.data_ptr(),
           src.data_ptr(), each, more, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), rows, n,
           page_size, num_pages, None if workspace is None else workspace.data_ptr(),
           0 if workspace is None else workspace.numel(), None if status is None else _status(status, dev))
    return table, lens, refs


def kv_compact(pools, block_table, page_refs, *, block_table_out=None, page_refs_out=None,
               n_used=None, workspace=None, status=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Move the used pages (page_refs > 0) to the front of every pool.

    block_table int32 [rows][max_pages] (-1 where there is no page), page_refs
    int32 [num_pages].  Returns (block_table, page_refs, n_used): pages n_used ..
    num_pages - 1 are free then (n_used: int32 tensor of one element).
    """
    try:
        dev = block_table.get_device()
        rows, width = block_table.shape
        (num_pages,) = page_refs.shape
        sound = (dev >= 0 and block_table.dtype is _I32 and page_refs.dtype is _I32
                 and page_refs.get_device() == dev and block_table.is_contiguous()
                 and page_refs.is_contiguous())
    except _NOT_SO:
        sound = False
    if not sound:
        dev = _device_of(block_table, "block_table")
        _tensor(block_table, "block_table", (_I32,), 2, dev)
        _tensor(page_refs, "page_refs", (_I32,), 1, dev)
        rows, width = block_table.shape
        num_pages = page_refs.shape[0]
    ptrs, sizes, n_pools, _ = _pool_args(pools, num_pages, dev)
    at = _Place(dev, stream)
    if block_table_out is None:
        block_table_out = _out(None, "", block_table, (rows, width), at)
    else:  # (may be block_table)
        _tensor(block_table_out, "block_table_out", (_I32,), 2, dev)
        if block_table_out.shape != block_table.shape:
            raise ValueError("block_table_out must have block_table's shape")
    refs = _out(page_refs_out, "page_refs_out", page_refs, (num_pages,), at)
    n_used = _out(n_used, "n_used", page_refs, (1,), at)
    workspace = _workspace(workspace, at, "tree_kv_compact_workspace_size", num_pages)
    at.run("tree_kv_compact", ptrs.buffer_info()[0], sizes.buffer_info()[0], n_pools,
           block_table.data_ptr(), width, page_refs.data_ptr(), block_table_out.data_ptr(),
           refs.data_ptr(), n_used.data_ptr(), rows, num_pages,
           None if workspace is None else workspace.data_ptr(),
           0 if workspace is None else workspace.numel(), None if status is None else _status(status, dev))
    return block_table_out, refs, n_used
