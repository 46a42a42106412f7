"""Python calls around verification: the 8-bit paged cache (write, commit, read
back), verification over it, and causal attention over whole prompts.

As in ``_lib``: arguments are checked, then handed to the library; there is no
fallback.  Every call runs on the device its tensors are on (all on one), on
``stream`` or that device's current stream.  Results and workspaces that a call
makes itself belong to the stream it runs on.

A step of a server makes these calls for every layer, and a small one takes the
GPU less time than the host, so each call first asks in one expression whether
its arguments are all as they should be; only if not does it go through them one
by one to say what is wrong.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from ._lib import _BITS64, TreeAttnError, load

_BF16 = torch.bfloat16
_I32 = torch.int32
_U8 = torch.uint8
_F32 = torch.float32
_CODES = (torch.uint8, torch.float8_e4m3fn)
# What a question about something that is no such tensor raises.
_NOT_SO = (AttributeError, TypeError, ValueError)


def _tensor(t, name: str, dtypes, ndim: int, dev: int, dense: bool = True):
    """Checks one argument; dev: the index of the device the others are on."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev
            and t.dim() == ndim and (not dense or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the other tensors on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.get_device()


def _status(status, dev: int):
    if status is None:
        return None
    _tensor(status, "status", (_I32,), status.dim() if isinstance(status, torch.Tensor) else 1, dev)
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    return status.data_ptr()


class _Place:
    """The device and stream of one call, and what is allocated there."""

    __slots__ = ("dev", "current", "stream", "handle")

    def __init__(self, dev: int, stream):
        self.dev = dev
        self.current = self.stream = None
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(dev)
            return
        if stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
        self.handle = stream.cuda_stream
        current = torch.cuda.current_stream(dev)
        if stream != current:
            self.current, self.stream = current, stream

    def empty(self, shape, dtype) -> torch.Tensor:
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=_DEVICES[self.dev])
        # Taken from the pool of the stream that writes it, so that it cannot
        # be memory that work queued on the current stream still reads; the
        # caller goes on to use it on the current stream.
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=_DEVICES[self.dev])
        t.record_stream(self.current)
        return t

    def call(self, name: str, *args) -> int:
        fn = getattr(load(), name)
        if self.dev == torch.cuda.current_device():
            return fn(*args)
        with torch.cuda.device(self.dev):
            return fn(*args)

    def run(self, name: str, *args) -> None:
        fn = getattr(load(), name)
        if self.dev == torch.cuda.current_device():
            rc = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.dev):
                rc = fn(*args, self.handle)
        if rc != 0:
            raise TreeAttnError(name, rc)


class _Devices(dict):
    def __missing__(self, index: int) -> torch.device:
        self[index] = torch.device("cuda", index)
        return self[index]


_DEVICES = _Devices()
_WORKSPACE: dict = {}  # bytes, by sizes and device


def _workspace_bytes(at: _Place, B: int, Hq: int, Hkv: int, d: int, T: int, P: int) -> int:
    sizes = (B, Hq, Hkv, d, T, P, at.dev)
    need = _WORKSPACE.get(sizes)
    if need is None:
        need = at.call("tree_attn_workspace_size", B, Hq, Hkv, d, T, 0, P)
        if need > 0:  # 0: the library could not say, this time (the call itself says why)
            _WORKSPACE[sizes] = need
    return need


def _pools(k_pages, v_pages, k_scales, v_scales, block_table):
    """Checks the cache's tensors; returns (device index, num_pages, Hkv, P, d)."""
    try:
        dev = k_pages.get_device()
        n, h, P, d = shape = k_pages.shape
        if (dev >= 0 and k_pages.dtype in _CODES and v_pages.dtype in _CODES
                and k_scales.dtype is _U8 and v_scales.dtype is _U8 and block_table.dtype is _I32
                and v_pages.shape == shape and k_scales.shape == (n, h, P)
                and v_scales.shape == (n, h, P) and block_table.dim() == 2
                and v_pages.get_device() == dev and k_scales.get_device() == dev
                and v_scales.get_device() == dev and block_table.get_device() == dev
                and k_pages.is_contiguous() and v_pages.is_contiguous()
                and k_scales.is_contiguous() and v_scales.is_contiguous()
                and block_table.is_contiguous()):
            return dev, n, h, P, d
    except _NOT_SO:
        pass
    dev = _device_of(k_pages, "k_pages")
    _tensor(k_pages, "k_pages", _CODES, 4, dev)
    _tensor(v_pages, "v_pages", _CODES, 4, dev)
    _tensor(k_scales, "k_scales", (_U8,), 3, dev)
    _tensor(v_scales, "v_scales", (_U8,), 3, dev)
    _tensor(block_table, "block_table", (_I32,), 2, dev)
    raise ValueError("k_pages, v_pages, k_scales and v_scales disagree on their sizes")


def _rows(t, name: str, dev, heads: Optional[int], d: Optional[int]):
    """Checks packed rows [N][H][d] with d contiguous; returns (token, head)
    strides, 0 where there is one row of that kind."""
    try:
        n, h, e = t.shape
        if (t.dtype is _BF16 and t.get_device() == dev and (heads is None or h == heads)
                and (d is None or e == d)):
            ts, hs, es = t.stride()
            if es == 1:
                return (ts if n > 1 else 0), (hs if h > 1 else 0)
    except _NOT_SO:
        pass
    _tensor(t, name, (_BF16,), 3, dev, dense=False)
    n, h, e = t.shape
    if (heads is not None and h != heads) or (d is not None and e != d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [N, {heads}, {d}]")
    ts, hs, es = t.stride()
    if es != 1 and e > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return (ts if n > 1 else 0), (hs if h > 1 else 0)


def _vector(t, name: str, n: int, dev):
    try:
        if (t.dtype is _I32 and t.shape == (n,) and t.get_device() == dev
                and t.is_contiguous()):
            return
    except _NOT_SO:
        pass
    _tensor(t, name, (_I32,), 1, dev)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")


def kv_append_fp8(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_seqlens, k, v, *,
                  seq_lens_out=None, status=None, stream=None) -> torch.Tensor:
    """Quantise new tokens' K/V into the 8-bit paged cache.

    k_pages / v_pages uint8 or float8_e4m3fn [num_pages][Hkv][P][d], k_scales /
    v_scales uint8 [num_pages][Hkv][P]; k, v bf16 [N][Hkv][d] packed by
    cu_seqlens int32 [B + 1] (token and head strides free, e.g. slices of a
    fused projection); token j of sequence b goes to position seq_lens[b] + j.
    Returns seq_lens_out (seq_lens plus the new tokens).
    """
    dev, num_pages, Hkv, P, d = _pools(k_pages, v_pages, k_scales, v_scales, block_table)
    B = block_table.shape[0]
    _vector(seq_lens, "seq_lens", B, dev)
    _vector(cu_seqlens, "cu_seqlens", B + 1, dev)
    k_ts, k_hs = _rows(k, "k", dev, Hkv, d)
    v_ts, v_hs = _rows(v, "v", dev, Hkv, d)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v disagree on the number of rows")
    at = _Place(dev, stream)
    if seq_lens_out is None:
        seq_lens_out = at.empty(B, _I32)
    else:
        _vector(seq_lens_out, "seq_lens_out", B, dev)
    at.run("tree_kv_append_fp8", k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
           v_scales.data_ptr(), block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
           cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), k_ts, k_hs, v_ts, v_hs,
           seq_lens_out.data_ptr(), B, k.shape[0], Hkv, d, P, num_pages, _status(status, dev))
    return seq_lens_out


def kv_commit_fp8(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, accept_path,
                  accept_len, tree_k, tree_v, *, seq_lens_out=None, status=None,
                  stream=None) -> torch.Tensor:
    """Quantise each sequence's accepted path (``greedy_accept``) into the 8-bit
    cache at positions seq_lens[b] + k.  tree_k / tree_v bf16 [B][T][Hkv][d].
    Returns seq_lens_out (seq_lens + accept_len)."""
    dev, num_pages, Hkv, P, d = _pools(k_pages, v_pages, k_scales, v_scales, block_table)
    B = block_table.shape[0]
    _vector(seq_lens, "seq_lens", B, dev)
    _vector(accept_len, "accept_len", B, dev)
    _tensor(accept_path, "accept_path", (_I32,), 2, dev)
    _tensor(tree_k, "tree_k", (_BF16,), 4, dev)
    _tensor(tree_v, "tree_v", (_BF16,), 4, dev)
    T = accept_path.shape[1]
    if (accept_path.shape[0] != B or tuple(tree_k.shape) != (B, T, Hkv, d)
            or tree_v.shape != tree_k.shape):
        raise ValueError("accept_path, tree_k, tree_v and the cache disagree on their sizes")
    at = _Place(dev, stream)
    if seq_lens_out is None:
        seq_lens_out = at.empty(B, _I32)
    else:
        _vector(seq_lens_out, "seq_lens_out", B, dev)
    at.run("tree_kv_commit_fp8", k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
           v_scales.data_ptr(), block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
           accept_path.data_ptr(), accept_len.data_ptr(), tree_k.data_ptr(), tree_v.data_ptr(),
           seq_lens_out.data_ptr(), B, Hkv, d, T, P, num_pages, _status(status, dev))
    return seq_lens_out


def kv_read_fp8(k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens, n_tokens: int, *,
                starts=None, k_out=None, v_out=None, status=None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read cached rows back as bf16 (exactly the values they stand for): output
    row cu_seqlens[b] + j is position starts[b] + j (starts None: 0) of
    sequence b.  Returns (k, v), bf16 [n_tokens][Hkv][d]; rows outside every
    sequence's range keep what k_out / v_out held (are uninitialised when the
    call makes them)."""
    dev, num_pages, Hkv, P, d = _pools(k_pages, v_pages, k_scales, v_scales, block_table)
    B, n = block_table.shape[0], int(n_tokens)
    if n < 0:
        raise ValueError("n_tokens must not be negative")
    _vector(cu_seqlens, "cu_seqlens", B + 1, dev)
    if starts is not None:
        _vector(starts, "starts", B, dev)
    at = _Place(dev, stream)
    outs = []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = at.empty((n, Hkv, d), _BF16)
        else:
            _tensor(t, name, (_BF16,), 3, dev)
            if tuple(t.shape) != (n, Hkv, d):
                raise ValueError(f"{name} must have shape {(n, Hkv, d)}")
        outs.append(t)
    at.run("tree_kv_read_fp8", k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
           v_scales.data_ptr(), block_table.data_ptr(), block_table.shape[1],
           None if starts is None else starts.data_ptr(), cu_seqlens.data_ptr(),
           outs[0].data_ptr(), outs[1].data_ptr(), B, n, Hkv, d, P, num_pages,
           _status(status, dev))
    return outs[0], outs[1]


def _check_verify(q, tree_k, tree_v, seq_lens, block_table, mask, parents, mask_out, dev, Hkv, d):
    """verify_fp8's arguments one by one."""
    for t, name in ((q, "q"), (tree_k, "tree_k"), (tree_v, "tree_v")):
        _tensor(t, name, (_BF16,), 4, dev)
    B, T = q.shape[:2]
    _vector(seq_lens, "seq_lens", B, dev)
    if (q.shape[3] != d or tuple(tree_k.shape) != (B, T, Hkv, d) or tree_v.shape != tree_k.shape
            or block_table.shape[0] != B):
        raise ValueError("inconsistent tensor shapes")
    if (mask is None) == (parents is None):
        raise ValueError("give exactly one of mask and parents")
    tree, dtypes, name = (mask, _BITS64, "mask") if parents is None else (parents, (_I32,), "parents")
    _tensor(tree, name, dtypes, tree.dim() if isinstance(tree, torch.Tensor) else 1, dev)
    if tuple(tree.shape) not in ((T,), (B, T)):
        raise ValueError(f"{name} must have shape [T] or [B][T]")
    if mask_out is not None:
        if parents is None:
            raise ValueError("mask_out goes with parents")
        _tensor(mask_out, "mask_out", _BITS64, tree.dim(), dev)
        if mask_out.shape != tree.shape:
            raise ValueError("mask_out must have the shape of parents")


def verify_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, tree_k, tree_v, *,
               mask=None, parents=None, mask_out=None, out=None, lse=None, workspace=None,
               status=None, softmax_scale: Optional[float] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Split tree attention over the 8-bit paged cache (T = 1: plain decoding).

    As ``verify`` / ``verify_tree`` with the committed rows in 8 bits and the
    tree tokens in bf16; give the tree either as ``mask`` (int64 / uint64 bits,
    [T] or [B][T]) or as ``parents`` (int32, [T] or [B][T]).  Returns (out, lse).
    """
    dev, num_pages, Hkv, P, d = _pools(k_pages, v_pages, k_scales, v_scales, block_table)
    tree = mask if parents is None else parents
    try:
        B, T, Hq, _ = q.shape
        sound = (q.dtype is _BF16 and tree_k.dtype is _BF16 and tree_v.dtype is _BF16
                 and seq_lens.dtype is _I32 and q.shape[3] == d
                 and tree_k.shape == (B, T, Hkv, d) and tree_v.shape == (B, T, Hkv, d)
                 and seq_lens.shape == (B,) and block_table.shape[0] == B
                 and (parents is None or mask is None) and tree.shape in ((T,), (B, T))
                 and (tree.dtype is _I32 if mask is None else tree.dtype in _BITS64)
                 and q.get_device() == dev and tree_k.get_device() == dev
                 and tree_v.get_device() == dev and seq_lens.get_device() == dev
                 and tree.get_device() == dev and q.is_contiguous() and tree_k.is_contiguous()
                 and tree_v.is_contiguous() and seq_lens.is_contiguous()
                 and tree.is_contiguous() and mask_out is None)
    except _NOT_SO:
        sound = False
    if not sound:
        _check_verify(q, tree_k, tree_v, seq_lens, block_table, mask, parents, mask_out, dev, Hkv,
                      d)
    stride = T if tree.dim() == 2 else 0
    at = _Place(dev, stream)
    if out is None:
        out = at.empty(q.shape, _BF16)
    else:
        _tensor(out, "out", (_BF16,), 4, dev)
    if lse is None:
        lse = at.empty((B, T, Hq), torch.float32)
    else:
        _tensor(lse, "lse", (torch.float32,), 3, dev)
    if out.shape != q.shape or tuple(lse.shape) != (B, T, Hq):
        raise ValueError("out and lse must have shapes [B][T][Hq][d] and [B][T][Hq]")
    if workspace is None:
        workspace = at.empty(max(_workspace_bytes(at, B, Hq, Hkv, d, T, P), 256), torch.uint8)
    else:
        _tensor(workspace, "workspace", (torch.uint8,), 1, dev)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    at.run("tree_attn_verify_fp8", q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
           k_scales.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(), block_table.shape[1],
           seq_lens.data_ptr(), tree_k.data_ptr(), tree_v.data_ptr(),
           None if mask is None else mask.data_ptr(), stride if parents is None else 0,
           None if parents is None else parents.data_ptr(), 0 if parents is None else stride,
           None if mask_out is None else mask_out.data_ptr(), out.data_ptr(), lse.data_ptr(), B,
           Hq, Hkv, d, T, P, num_pages, float(softmax_scale), workspace.data_ptr(),
           workspace.numel(), _status(status, dev))
    return out, lse


def prefill(q, k, v, cu_seqlens, *, out=None, lse=None, status=None,
            softmax_scale: Optional[float] = None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention over packed prompts of different lengths.

    q bf16 [N][Hq][d], k and v bf16 [N][Hkv][d] (token and head strides free),
    cu_seqlens int32 [B + 1]: sequence b is rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1.  Returns (out [N][Hq][d] bf16, lse [N][Hq] fp32);
    rows outside every sequence keep what out / lse held (are uninitialised
    when the call makes them).
    """
    dev = _device_of(q, "q")
    q_ts, q_hs = _rows(q, "q", dev, None, None)
    N, Hq, d = q.shape
    k_ts, k_hs = _rows(k, "k", dev, None, d)
    Hkv = k.shape[1]
    v_ts, v_hs = _rows(v, "v", dev, Hkv, d)
    if k.shape[0] != N or v.shape[0] != N:
        raise ValueError("q, k and v disagree on the number of rows")
    _tensor(cu_seqlens, "cu_seqlens", (_I32,), 1, dev)
    if cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    at = _Place(dev, stream)
    if out is None:
        out = at.empty((N, Hq, d), _BF16)
    else:
        _tensor(out, "out", (_BF16,), 3, dev)
    if lse is None:
        lse = at.empty((N, Hq), torch.float32)
    else:
        _tensor(lse, "lse", (torch.float32,), 2, dev)
    if tuple(out.shape) != (N, Hq, d) or tuple(lse.shape) != (N, Hq):
        raise ValueError("out and lse must have shapes [N][Hq][d] and [N][Hq]")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    at.run("tree_attn_prefill", q.data_ptr(), k.data_ptr(), v.data_ptr(), q_ts, q_hs, k_ts, k_hs,
           v_ts, v_hs, cu_seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(),
           cu_seqlens.shape[0] - 1, N, Hq, Hkv, d, float(softmax_scale), _status(status, dev))
    return out, lse
