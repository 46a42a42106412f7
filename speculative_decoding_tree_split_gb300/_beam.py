"""Python call for beam search's selection (see ``_serving`` for the conventions)."""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._pages import _workspace
from ._serving import _DEVICES, _F32, _I32, _NOT_SO, _Place, _device_of, _int32, _tensor

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_FLAGS = (torch.bool, torch.uint8)


def _check(logits, scores, finished, dev: int):
    """beam_select's inputs one by one."""
    _tensor(logits, "logits", tuple(_DTYPES), 3, dev, dense=False)
    B, W, V = logits.shape
    if V > 1 and logits.stride(2) != 1:
        raise ValueError("logits' last dimension must be contiguous")
    _tensor(scores, "scores", (_F32,), 2, dev)
    if tuple(scores.shape) != (B, W):
        raise ValueError(f"scores must have shape {(B, W)}")
    if finished is not None:
        _tensor(finished, "finished", _FLAGS, 2, dev)
        if tuple(finished.shape) != (B, W):
            raise ValueError(f"finished must have shape {(B, W)}")


def _out(t, name: str, dtype, shape, at: _Place) -> torch.Tensor:
    if t is None:
        return at.empty(shape, dtype)
    _tensor(t, name, (dtype,), 2, at.dev)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}")
    return t


def beam_select(logits, scores, n_select: int, *, finished=None, eos: Optional[int] = None,
                scores_out=None, rows_out=None, tokens_out=None, workspace=None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The n_select best continuations over a sequence's beams and the vocabulary.

    logits bf16, fp16 or fp32 [B][W][V] (batch and beam strides free, e.g. a slice of
    a padded vocabulary), scores fp32 [B][W]; continuation (w, v) scores scores[w] +
    ln softmax(logits[w])[v].  A beam marked in ``finished`` (bool [B][W], with
    ``eos``) stands for itself alone, as (w, eos) with its score unchanged.
    Returns (scores fp32, rows int32, tokens int32), each [B][n_select], best first,
    ties to the lowest (w, v); rows are b * W + w, the ``src`` of ``kv_fork``.  NaN and
    -inf logits are never taken; where nothing is left: -inf, -1, -1.  Beams with the same
    logits and scores tie wherever they lie in memory; scores of other beams are told apart
    to fp32's rounding of the sums (about 2^-21).
    """
    k = int(n_select)
    try:
        dev = logits.get_device()
        B, W, V = logits.shape
        bs, ws, vs = logits.stride()
        sound = (dev >= 0 and logits.dtype in _DTYPES and vs == 1 and scores.dtype is _F32
                 and scores.shape == (B, W) and scores.get_device() == dev
                 and scores.is_contiguous()
                 and (finished is None or (finished.dtype in _FLAGS and finished.shape == (B, W)
                                           and finished.get_device() == dev
                                           and finished.is_contiguous())))
    except _NOT_SO:
        sound = False
    if not sound:
        dev = _device_of(logits, "logits")
        _check(logits, scores, finished, dev)
        B, W, V = logits.shape
        bs, ws, _ = logits.stride()
    if finished is None:
        eos = -1
    elif eos is None:
        raise ValueError("finished beams need eos")
    _int32(k, eos)
    at = _Place(dev, stream)
    if scores_out is None and rows_out is None and tokens_out is None and at.stream is None and k > 0:
        d = _DEVICES[dev]
        scores_out = torch.empty((B, k), dtype=_F32, device=d)
        rows_out = torch.empty((B, k), dtype=_I32, device=d)
        tokens_out = torch.empty((B, k), dtype=_I32, device=d)
    else:
        scores_out = _out(scores_out, "scores_out", _F32, (B, max(k, 0)), at)
        rows_out = _out(rows_out, "rows_out", _I32, (B, max(k, 0)), at)
        tokens_out = _out(tokens_out, "tokens_out", _I32, (B, max(k, 0)), at)
    workspace = _workspace(workspace, at, "tree_beam_workspace_size", B, W, V, k)
    at.run("tree_beam_select", logits.data_ptr(), _DTYPES[logits.dtype], bs if B > 1 else 0,
           ws if W > 1 else 0, scores.data_ptr(),
           None if finished is None else finished.data_ptr(), int(eos),
           scores_out.data_ptr(), rows_out.data_ptr(), tokens_out.data_ptr(), B, W, V, k,
           None if workspace is None else workspace.data_ptr(),
           0 if workspace is None else workspace.numel())
    return scores_out, rows_out, tokens_out
