"""Drafted tokens: which of them the target's probabilities let stand.

A narrow child of the nested weights drafts a few tokens for each sequence, a wider one takes
them all in one step (``kv_reserve``, ``kv_append`` and ``kv_attend_shared`` with several tokens of
a row), and from both their probabilities

    accepted, next = verify_drafts(target, ids, u, draft=draft, cu=cu)

says how many drafts stand and which token follows.  As everywhere in this package the call
only marshals arguments and queues the work on the current stream of the tensors' GPU.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _lib, _raw_stream, _workspace
from .kv import _BF16, _F32, _INT32, _current_device, _i32, _i64, _is, _vp


class VerifyArgs(ctypes.Structure):
    _fields_ = [("target", _vp), ("draft", _vp), ("target_ld", _i64), ("draft_ld", _i64), ("tokens", _i64),
                ("vocab", _i64), ("rows", _i64), ("dtype", _i32), ("cu", _vp), ("ids", _vp), ("u", _vp),
                ("accepted", _vp), ("next", _vp), ("workspace", _vp), ("workspace_bytes", _i64)]


PROB_DTYPES = {_F32: 0, _BF16: 1}


def declare(lib) -> None:
    """The C signatures of the entry points."""
    lib.nbw_verify_drafts.argtypes = [ctypes.POINTER(VerifyArgs), _vp]
    lib.nbw_verify_drafts.restype = ctypes.c_int
    lib.nbw_verify_drafts_workspace_bytes.argtypes = [_i64, _i64]
    lib.nbw_verify_drafts_workspace_bytes.restype = _i64


def verify_workspace_bytes(rows: int, vocab: int) -> int:
    """Bytes of scratch verify_drafts needs."""
    nbytes = _lib().nbw_verify_drafts_workspace_bytes(rows, vocab)
    if nbytes < 0:
        raise ValueError(f"{rows} rows of {vocab} probabilities are outside what the library takes")
    return nbytes


def _lines(t, name: str, dtype, shape, index: int):
    """Address of a [tokens][vocab] tensor with unit column stride and its stride from line to line."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return t.data_ptr(), shape[1]
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on GPU {index}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    tokens, vocab = shape
    if (vocab > 1 and t.stride(1) != 1) or (tokens > 1 and t.stride(0) < vocab):
        raise ValueError(f"{name} must have unit column stride and lines that do not overlap")
    return t.data_ptr(), t.stride(0) if tokens > 1 else vocab


def verify_drafts(target, ids, u, *, draft=None, cu=None, accepted=None, next=None, workspace="auto"):
    """Which drafts stand, and the token after them: (accepted, next), int32 [rows].

    ``target`` [tokens][vocab] (fp32 or bf16): the target's probabilities after each token.
    ``cu`` (int32 [rows + 1]): row r has tokens cu[r]..cu[r+1]-1, the last one that is certain, then
    its drafts; without it each token is a row of its own, with nothing drafted.  ``ids`` (int32
    [tokens], None without cu): the tokens.  ``draft`` (as target): what the drafts were sampled
    from, a line in the place before each draft; without it a draft stands for itself, as one found
    by looking it up does.  ``u`` (fp32 [tokens]): random numbers within [0, 1), for each draft the
    one in the place before its own, and the row's last one for the next token.

    A draft x stands if those before it do and u * draft[x] < target[x]; the next token is sampled
    from max(target - draft, 0) of the line that refused, or from target's last line if none did.
    ``workspace``: as for :func:`kv_attend`, ``verify_workspace_bytes(rows, vocab)`` bytes."""
    if not isinstance(target, torch.Tensor):
        raise TypeError("target must be a torch.Tensor")
    if target.device.type != "cuda":
        raise ValueError("target must be on a GPU")
    index = target.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return verify_drafts(target, ids, u, draft=draft, cu=cu, accepted=accepted, next=next, workspace=workspace)
    kind = PROB_DTYPES.get(target.dtype)
    if kind is None:
        raise TypeError(f"target must be torch.float32 or torch.bfloat16, got {target.dtype}")
    shape = target.shape
    if len(shape) != 2 or not shape[1]:
        raise ValueError("target must be [tokens][vocab]")
    tokens, vocab = shape
    tp, t_ld = _lines(target, "target", target.dtype, shape, index)
    dp, d_ld = (None, 0) if draft is None else _lines(draft, "draft", target.dtype, shape, index)
    cu_p = ids_p = None
    rows = tokens
    if cu is not None:
        if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or not cu.numel():
            raise ValueError("cu must be an int32 [rows + 1] tensor")
        rows = cu.size(0) - 1
        cu_p = _is(cu, "cu", _INT32, (rows + 1,), index)
        ids_p = _is(ids, "ids", _INT32, (tokens,), index)
    elif draft is not None:
        raise ValueError("without cu nothing is drafted")
    device = target.device
    accepted = torch.empty(rows, dtype=_INT32, device=device) if accepted is None else accepted
    next = torch.empty(rows, dtype=_INT32, device=device) if next is None else next
    lib, stream = _lib(), _raw_stream(index)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', a tensor or None")
        workspace = _workspace(index, stream, verify_workspace_bytes(rows, vocab))
    elif workspace is not None and (workspace.get_device() != index or workspace.dtype != torch.uint8 or
                                    not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on the target's GPU")
    args = VerifyArgs(tp, dp, t_ld, d_ld, tokens, vocab, rows, kind, cu_p, ids_p, _is(u, "u", _F32, (tokens,), index),
                      _is(accepted, "accepted", _INT32, (rows,), index), _is(next, "next", _INT32, (rows,), index),
                      None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    st = lib.nbw_verify_drafts(ctypes.byref(args), stream)
    if st:
        _check(st, "nbw_verify_drafts")
    return accepted, next
