"""Python calls for attention over selected pages of a long cache: bounds of the
pages' keys, selection by them, attention (see ``_serving`` for the conventions).
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from ._lib import _BITS64
from ._serving import (_BF16, _CODES, _DEVICES, _F32, _I32, _NOT_SO, _U8, _Place, _device_of,
                       _int32, _status, _tensor, _vector)

_I8 = torch.int8


def _cache_arg(pages, scales, name: str, dev: int, shape=None):
    """Checks one pool of a bf16 cache (scales None) or of an 8-bit one."""
    try:
        if (pages.get_device() == dev and pages.dim() == 4 and pages.is_contiguous()
                and (shape is None or pages.shape == shape)
                and (pages.dtype is _BF16 if scales is None else
                     pages.dtype in _CODES and scales.dtype is _U8
                     and scales.shape == pages.shape[:3] and scales.get_device() == dev
                     and scales.is_contiguous())):
            return
    except _NOT_SO:
        pass
    _tensor(pages, f"{name}_pages", (_BF16,) if scales is None else _CODES, 4, dev)
    if scales is not None:
        _tensor(scales, f"{name}_scales", (_U8,), 3, dev)
        if scales.shape != pages.shape[:3]:
            raise ValueError(f"{name}_scales must have shape {tuple(pages.shape[:3])}")
    raise ValueError(f"{name}_pages has shape {tuple(pages.shape)}, expected {tuple(shape)}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_bounds(bounds, bounds_exp, n, H, d, dev: int):
    _tensor(bounds, "bounds", (_I8,), 4, dev)
    _tensor(bounds_exp, "bounds_exp", (_U8,), 2, dev)
    if tuple(bounds.shape) != (n, H, 2, d) or tuple(bounds_exp.shape) != (n, H):
        raise ValueError(f"bounds and bounds_exp must have shapes {(n, H, 2, d)} and {(n, H)}")


def kv_block_bounds(k_pages, block_table, seq_lens, *, k_scales=None, starts=None, bounds=None,
                    bounds_exp=None, status=None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Bounds of each page's keys, per KV head and channel, in 8 bits.

    k_pages [num_pages][Hkv][P][d], bf16 or (with k_scales) 8-bit codes.  Writes the
    pages that hold positions starts[b] (None: 0) .. seq_lens[b] - 1, over their
    committed tokens (the same ones in all sequences that share a page); call it after
    tokens were appended or committed, with the lengths before as ``starts``.  Returns
    (bounds int8 [num_pages][Hkv][2][d], bounds_exp uint8 [num_pages][Hkv]); rows of
    other pages keep what they held (are uninitialised when the call makes them).
    """
    try:
        dev = k_pages.get_device()
        B, width = block_table.shape
        sound = (dev >= 0 and block_table.dtype is _I32 and seq_lens.dtype is _I32
                 and seq_lens.shape == (B,) and block_table.get_device() == dev
                 and seq_lens.get_device() == dev and block_table.is_contiguous()
                 and seq_lens.is_contiguous())
    except _NOT_SO:
        sound = False
    if not sound:
        dev = _device_of(k_pages, "k_pages")
        _tensor(block_table, "block_table", (_I32,), 2, dev)
        B, width = block_table.shape
        _vector(seq_lens, "seq_lens", B, dev)
    _cache_arg(k_pages, k_scales, "k", dev)
    n, H, P, d = k_pages.shape
    if starts is not None:
        _vector(starts, "starts", B, dev)
    if (bounds is None) != (bounds_exp is None):
        raise ValueError("give both of bounds and bounds_exp or neither")
    at = _Place(dev, stream)
    if bounds is None:
        bounds, bounds_exp = at.empty((n, H, 2, d), _I8), at.empty((n, H), _U8)
    else:
        _check_bounds(bounds, bounds_exp, n, H, d, dev)
    at.run("tree_kv_block_bounds", k_pages.data_ptr(), _ptr(k_scales), block_table.data_ptr(),
           width, _ptr(starts), seq_lens.data_ptr(), bounds.data_ptr(), bounds_exp.data_ptr(), B,
           H, d, P, n, None if status is None else _status(status, dev))
    return bounds, bounds_exp


def select_blocks(q, bounds, bounds_exp, block_table, seq_lens, n_select: int, page_size: int, *,
                  n_first: int = 1, n_last: int = 1, out=None, status=None,
                  stream=None) -> torch.Tensor:
    """For every query the n_select pages whose bounds allow the largest scores.

    q bf16 [B][T][Hq][d]; the heads that share a KV head choose together.  The first
    n_first and the last n_last pages of a sequence are always among them.  Returns
    int32 [B][T][Hkv][n_select]: pages of the sequence in ascending order, then -1.
    """
    k = n_select
    try:
        dev = q.get_device()
        B, T, Hq, d = q.shape
        n, H = bounds_exp.shape
        width = block_table.shape[1]
        sound = (dev >= 0 and q.dtype is _BF16 and bounds.dtype is _I8 and bounds_exp.dtype is _U8
                 and block_table.dtype is _I32 and seq_lens.dtype is _I32
                 and bounds.shape == (n, H, 2, d) and block_table.shape == (B, width)
                 and seq_lens.shape == (B,) and bounds.get_device() == dev
                 and bounds_exp.get_device() == dev and block_table.get_device() == dev
                 and seq_lens.get_device() == dev and q.is_contiguous()
                 and bounds.is_contiguous() and bounds_exp.is_contiguous()
                 and block_table.is_contiguous() and seq_lens.is_contiguous())
    except (*_NOT_SO, IndexError):
        sound = False
    if not sound:
        dev = _device_of(q, "q")
        _tensor(q, "q", (_BF16,), 4, dev)
        B, T, Hq, d = q.shape
        _tensor(bounds, "bounds", (_I8,), 4, dev)
        n, H = bounds.shape[:2]
        _check_bounds(bounds, bounds_exp, n, H, d, dev)
        _tensor(block_table, "block_table", (_I32,), 2, dev)
        if block_table.shape[0] != B:
            raise ValueError(f"block_table must have {B} rows, got {block_table.shape[0]}")
        _vector(seq_lens, "seq_lens", B, dev)
        width = block_table.shape[1]
    _int32(k, page_size, n_first, n_last)
    at = _Place(dev, stream)
    if out is None and at.stream is None and k > 0:
        out = torch.empty((B, T, H, k), dtype=_I32, device=_DEVICES[dev])
    elif out is None:
        out = at.empty((B, T, H, max(k, 0)), _I32)
    else:
        _tensor(out, "out", (_I32,), 4, dev)
        if tuple(out.shape) != (B, T, H, k):
            raise ValueError(f"out must have shape {(B, T, H, k)}")
    at.run("tree_select_blocks", q.data_ptr(), bounds.data_ptr(), bounds_exp.data_ptr(),
           block_table.data_ptr(), width, seq_lens.data_ptr(), out.data_ptr(), B, Hq, H, d, T,
           page_size, n, k, n_first, n_last, None if status is None else _status(status, dev))
    return out


def _check_verify(q, tree_k, tree_v, block_table, seq_lens, blocks, mask, parents, dev, H, d):
    """verify_blocks' arguments one by one."""
    for t, name in ((q, "q"), (tree_k, "tree_k"), (tree_v, "tree_v")):
        _tensor(t, name, (_BF16,), 4, dev)
    B, T = q.shape[:2]
    _tensor(block_table, "block_table", (_I32,), 2, dev)
    _vector(seq_lens, "seq_lens", B, dev)
    _tensor(blocks, "blocks", (_I32,), 4, dev)
    if (q.shape[3] != d or tuple(tree_k.shape) != (B, T, H, d) or tree_v.shape != tree_k.shape
            or block_table.shape[0] != B or tuple(blocks.shape[:3]) != (B, T, H)):
        raise ValueError("inconsistent tensor shapes")
    if (mask is None) == (parents is None):
        raise ValueError("give exactly one of mask and parents")
    tree, dtypes, name = (mask, _BITS64, "mask") if parents is None else (parents, (_I32,), "parents")
    _tensor(tree, name, dtypes, tree.dim() if isinstance(tree, torch.Tensor) else 1, dev)
    if tuple(tree.shape) not in ((T,), (B, T)):
        raise ValueError(f"{name} must have shape [T] or [B][T]")


def verify_blocks(q, k_pages, v_pages, block_table, seq_lens, blocks, tree_k, tree_v, *, mask=None,
                  parents=None, k_scales=None, v_scales=None, out=None, lse=None, status=None,
                  softmax_scale: Optional[float] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Split tree attention over selected pages (T = 1: plain decoding).

    As ``verify`` (bf16 cache) or, with k_scales and v_scales, ``verify_fp8``, where
    token t of sequence b sees through KV head h only the committed tokens of pages
    blocks[b][t][h] (``select_blocks``; -1: none), and the tree tokens by ``mask`` or
    ``parents``.  Returns (out, lse).
    """
    dev = _device_of(k_pages, "k_pages")
    if (k_scales is None) != (v_scales is None):
        raise ValueError("give both of k_scales and v_scales or neither")
    _cache_arg(k_pages, k_scales, "k", dev)
    n, H, P, d = shape = k_pages.shape
    _cache_arg(v_pages, v_scales, "v", dev, shape)
    tree = mask if parents is None else parents
    try:
        B, T, Hq, _ = q.shape
        sound = (q.dtype is _BF16 and tree_k.dtype is _BF16 and tree_v.dtype is _BF16
                 and seq_lens.dtype is _I32 and block_table.dtype is _I32
                 and blocks.dtype is _I32 and q.shape[3] == d and blocks.dim() == 4
                 and tree_k.shape == (B, T, H, d) and tree_v.shape == (B, T, H, d)
                 and seq_lens.shape == (B,) and block_table.dim() == 2
                 and block_table.shape[0] == B and blocks.shape[:3] == (B, T, H)
                 and (parents is None or mask is None) and tree.shape in ((T,), (B, T))
                 and (tree.dtype is _I32 if mask is None else tree.dtype in _BITS64)
                 and q.get_device() == dev and tree_k.get_device() == dev
                 and tree_v.get_device() == dev and seq_lens.get_device() == dev
                 and tree.get_device() == dev and block_table.get_device() == dev
                 and blocks.get_device() == dev and q.is_contiguous()
                 and tree_k.is_contiguous() and tree_v.is_contiguous()
                 and seq_lens.is_contiguous() and tree.is_contiguous()
                 and block_table.is_contiguous() and blocks.is_contiguous())
    except _NOT_SO:
        sound = False
    if not sound:
        _check_verify(q, tree_k, tree_v, block_table, seq_lens, blocks, mask, parents, dev, H, d)
        B, T, Hq, _ = q.shape
    stride = T if tree.dim() == 2 else 0
    at = _Place(dev, stream)
    if out is None and lse is None and at.stream is None:
        out = torch.empty_like(q)
        lse = torch.empty((B, T, Hq), dtype=_F32, device=_DEVICES[dev])
    else:
        if out is None:
            out = at.empty(q.shape, _BF16)
        else:
            _tensor(out, "out", (_BF16,), 4, dev)
        if lse is None:
            lse = at.empty((B, T, Hq), _F32)
        else:
            _tensor(lse, "lse", (_F32,), 3, dev)
        if out.shape != q.shape or tuple(lse.shape) != (B, T, Hq):
            raise ValueError("out and lse must have shapes [B][T][Hq][d] and [B][T][Hq]")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    at.run("tree_attn_verify_blocks", q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
           _ptr(k_scales), _ptr(v_scales), block_table.data_ptr(), block_table.shape[1],
           seq_lens.data_ptr(), blocks.data_ptr(), blocks.shape[3], tree_k.data_ptr(),
           tree_v.data_ptr(), _ptr(mask), stride if parents is None else 0, _ptr(parents),
           0 if parents is None else stride, out.data_ptr(), lse.data_ptr(), B, Hq, H, d, T, P, n,
           float(softmax_scale), None if status is None else _status(status, dev))
    return out, lse
