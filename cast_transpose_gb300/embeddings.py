"""The embedding: rows of a table by token id, and the gradient of the table.

An id outside the table, -1 say, is padding: its row is 0, and it adds to no
gradient.
"""
from __future__ import annotations

import torch

from . import _check, _here, _need, _scalar, _space, lib
from .moe import _DTYPES, _INDEX, _rows_of


def _ids(idx, device):
    """The number of ids, their address and their bytes."""
    if not isinstance(idx, torch.Tensor) or idx.dim() != 1:
        raise ValueError("idx must be a 1-D tensor")
    dtype, shape = idx.dtype, idx.shape
    return (shape[0], _need(idx, "idx", dtype if dtype in _INDEX else _INDEX, shape, device),
            4 if dtype is torch.int32 else 8)


def embedding(idx, table, out, scale=1.0, noop_flag=None, stream=None) -> None:
    """idx [T] (int32 or int64), table [V, hidden] -> out [T, hidden] of the
    table's type: scale * table[idx]."""
    device, handle = _here(stream)
    tokens, pi, size = _ids(idx, device)
    hidden, dtype = _rows_of(table, "table")
    shape = table.shape
    _check(lib().embedding(pi, size, tokens, _need(table, "table", dtype, shape, device), shape[0],
                           hidden, _DTYPES[dtype], scale,
                           _need(out, "out", dtype, (tokens, hidden), device),
                           _scalar(noop_flag, "noop_flag", device), handle))


def embedding_backward_workspace_size(tokens: int, vocab: int, hidden: int) -> int:
    return int(lib().embedding_backward_workspace_size(tokens, vocab, hidden))


def embedding_backward(idx, dout, dtable, workspace=None, scale=1.0, accumulate=False, noop_flag=None,
                       stream=None) -> None:
    """dout [T, hidden] -> dtable [V, hidden] of its type or fp32: scale * the
    sum of the rows of each id; accumulate: added to what dtable holds.
    workspace: uint8, of at least embedding_backward_workspace_size(T, V,
    hidden) bytes."""
    device, handle = _here(stream)
    tokens, pi, size = _ids(idx, device)
    hidden, dtype = _rows_of(dout, "dout")
    columns, grad = _rows_of(dtable, "dtable")
    if columns != hidden:
        raise ValueError(f"dtable has {columns} columns, dout {hidden}")
    if grad is not dtype and grad is not torch.float32:
        raise TypeError(f"dtable has dtype {grad}, expected {dtype} or float32")
    shape = dtable.shape
    _check(lib().embedding_backward(
        pi, size, tokens, _need(dout, "dout", dtype, (tokens, hidden), device), shape[0], hidden,
        _DTYPES[dtype], scale, _need(dtable, "dtable", grad, shape, device), _DTYPES[grad],
        1 if accumulate else 0, *_space(workspace, device),
        _scalar(noop_flag, "noop_flag", device), handle))
