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

from ._lib import load
from ._serving import _I32, _NOT_SO, _Place, _device_of, _status, _tensor, _vector


def _pool_args(pools: Sequence[torch.Tensor], num_pages: Optional[int], dev: int):
    """(pointers, bytes of a page, how many, pages) of the pools, as arrays for the
    library (to be kept until the call returns)."""
    ptrs, sizes = array("Q"), array("Q")
    for i, t in enumerate(pools):
        try:
            sound = (t.get_device() == dev and t.is_contiguous() and t.dim() >= 2
                     and (num_pages is None or t.shape[0] == num_pages) and t.shape[0] > 0)
        except _NOT_SO:
            sound = False
        if not sound:
            name = f"pools[{i}]"
            if _device_of(t, name) != dev:
                raise ValueError(f"{name} is on cuda:{t.get_device()}, the other tensors on "
                                 f"cuda:{dev}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.dim() < 2:
                raise ValueError(f"{name} must have pages of some size")
            raise ValueError(f"{name} has {t.shape[0]} pages, expected {num_pages}")
        num_pages = t.shape[0]
        ptrs.append(t.data_ptr())
        sizes.append(t.nbytes // num_pages)
    return ptrs, sizes, len(ptrs), num_pages


def _workspace(workspace, need: int, dev: int, at: _Place) -> torch.Tensor:
    if workspace is None:
        return at.empty(max(need, 256), torch.uint8)
    _tensor(workspace, "workspace", (torch.uint8,), 1, dev)
    return workspace


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
    if t is None:
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
    dev = _device_of(block_table, "block_table")
    _tensor(block_table, "block_table", (_I32,), 2, dev)
    rows, width = block_table.shape
    _vector(seq_lens, "seq_lens", rows, dev)
    _tensor(page_refs, "page_refs", (_I32,), 1, dev)
    _tensor(src, "src", (_I32,), 1, dev)
    n = src.shape[0]
    num_pages = page_refs.shape[0]
    more, each = 0, None
    if isinstance(reserve, torch.Tensor):
        _vector(reserve, "reserve", n, dev)
        each = reserve.data_ptr()
    else:
        more = int(reserve)
        if more < 0:
            raise ValueError("reserve must not be negative")
    ptrs, sizes, n_pools, _ = _pool_args(pools, num_pages, dev)
    at = _Place(dev, stream)
    table = _out(block_table_out, "block_table_out", block_table, (n, width), at)
    lens = _out(seq_lens_out, "seq_lens_out", seq_lens, (n,), at)
    refs = _out(page_refs_out, "page_refs_out", page_refs, (num_pages,), at)
    workspace = _workspace(workspace, load().tree_kv_fork_workspace_size(rows, n, num_pages), dev,
                           at)
    at.run("tree_kv_fork", ptrs.buffer_info()[0], sizes.buffer_info()[0], n_pools,
           block_table.data_ptr(), width, seq_lens.data_ptr(), page_refs.data_ptr(),
           src.data_ptr(), each, more, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), rows, n,
           page_size, num_pages, workspace.data_ptr(), workspace.numel(), _status(status, dev))
    return table, lens, refs


def kv_compact(pools, block_table, page_refs, *, block_table_out=None, page_refs_out=None,
               n_used=None, workspace=None, status=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Move the used pages (page_refs > 0) to the front of every pool.

    block_table int32 [rows][max_pages] (-1 where there is no page), page_refs
    int32 [num_pages].  Returns (block_table, page_refs, n_used): pages n_used ..
    num_pages - 1 are free then (n_used: int32 tensor of one element).
    """
    dev = _device_of(block_table, "block_table")
    _tensor(block_table, "block_table", (_I32,), 2, dev)
    _tensor(page_refs, "page_refs", (_I32,), 1, dev)
    rows, width = block_table.shape
    num_pages = page_refs.shape[0]
    ptrs, sizes, n_pools, _ = _pool_args(pools, num_pages, dev)
    at = _Place(dev, stream)
    if block_table_out is None:
        block_table_out = at.empty((rows, width), _I32)
    else:
        _tensor(block_table_out, "block_table_out", (_I32,), 2, dev)
        if block_table_out.shape != block_table.shape:
            raise ValueError("block_table_out must have block_table's shape")
    refs = _out(page_refs_out, "page_refs_out", page_refs, (num_pages,), at)
    if n_used is None:
        n_used = at.empty((1,), _I32)
    else:
        _vector(n_used, "n_used", 1, dev)
    workspace = _workspace(workspace, load().tree_kv_compact_workspace_size(num_pages), dev, at)
    at.run("tree_kv_compact", ptrs.buffer_info()[0], sizes.buffer_info()[0], n_pools,
           block_table.data_ptr(), width, page_refs.data_ptr(), block_table_out.data_ptr(),
           refs.data_ptr(), n_used.data_ptr(), rows, num_pages, workspace.data_ptr(),
           workspace.numel(), _status(status, dev))
    return block_table_out, refs, n_used
