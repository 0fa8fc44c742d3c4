"""Tokens sorted by expert and back: argument checks and calls.

T tokens choose K experts each, out of E.  ``MoePlan`` holds the buffers that
``moe_sort`` fills from the router's choices and the other calls read, the
backward calls too: until a layer's backward pass has run, its plan must not be
sorted again.  In training every layer, and every microbatch in flight, has a
plan of its own, reused from step to step; layers that only run forward can
share one, each sorting before it moves.  A plan's buffers, its workspace among
them, are used by one stream at a time.

  moe_router             the choices, their weights and counts, the balance loss
  moe_router_backward    the gradient of the router's logits
  moe_sort               the plan: which sorted row every (token, k) slot gets
  moe_dispatch           out[row] = x[token], padding rows zero
  moe_dispatch_backward  dx[token] = sum over k of dout[row]
  fp8_moe_dispatch       the same rows, weighted if asked, as FP8 + transpose
  moe_combine            out[token] = sum over k of weight * ys[row]
  moe_combine_backward   dys[row] = weight * dout[token], dweights

Like the other calls of the package they only pass device pointers to the C
entry points of the same names: outputs are the caller's, nothing is
synchronised, everything can be captured in a CUDA graph.
"""
from __future__ import annotations

import struct
from operator import attrgetter

import torch

from . import (E4M3, _at, _check, _dev, _here, _need, _opt, _ptr, _scalar, _space, _stream, _U8,
               lib)

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32, _F32 = torch.int32, torch.float32
_INDEX = (torch.int32, torch.int64)


def moe_sorted_rows(tokens: int, topk: int, experts: int, align: int = 1) -> int:
    """Rows that hold every slot whatever the routing, each expert's padded
    to a multiple of ``align``."""
    return int(lib().moe_sorted_rows(tokens, topk, experts, align))


def _kept(name):
    return property(attrgetter("_" + name))


class MoePlan:
    """The buffers of one sorting: ``row_of`` int32 [T, K], ``src`` int32
    [rows], ``offsets`` int32 [E + 1], ``counts`` int32 [E].  Buffers given
    here are used, the others allocated.  ``rows`` defaults to what holds
    every slot (or to ``src``'s length); with fewer, the slots that come last
    in expert order are dropped.

    Sizes and buffers were checked together and stay as they are: the
    attributes cannot be assigned.  What a buffer holds can be changed, by
    moe_sort or in place."""

    tokens, topk, experts, align, rows, slots = map(
        _kept, ("tokens", "topk", "experts", "align", "rows", "slots"))
    row_of, src, offsets, counts, workspace = map(
        _kept, ("row_of", "src", "offsets", "counts", "workspace"))

    def __init__(self, tokens, topk, experts, align=1, rows=None, device="cuda", row_of=None,
                 src=None, offsets=None, counts=None):
        need = moe_sorted_rows(tokens, topk, experts, align)
        if need == 0 and tokens * topk != 0 or min(topk, experts, align) < 1 or tokens < 0:
            raise ValueError(f"a plan for {tokens} tokens, {topk} of {experts} experts, "
                             f"align {align} is outside the limits")
        if rows is None:
            rows = need if src is None else src.numel()
        self._tokens, self._topk, self._experts, self._align, self._rows = (tokens, topk, experts,
                                                                            align, rows)

        def buffer(t, shape):
            return torch.empty(shape, dtype=_I32, device=device) if t is None else t

        self._slots = (tokens, topk)
        self._row_of = buffer(row_of, self._slots)
        self._src = buffer(src, (rows,))
        self._offsets = buffer(offsets, (experts + 1,))
        self._counts = buffer(counts, (experts,))
        self._workspace_size = int(lib().moe_sort_workspace_size(tokens, topk, experts))
        self._workspace = torch.empty(self._workspace_size, dtype=torch.uint8,
                                      device=self._row_of.device)
        # checked once, here; each call asks for their addresses
        _ptr(self._row_of, "row_of", _I32, self._slots)
        _ptr(self._src, "src", _I32, (rows,))
        _ptr(self._offsets, "offsets", _I32, (experts + 1,))
        _ptr(self._counts, "counts", _I32, (experts,))
        self._row_of_at, self._src_at = self._row_of.data_ptr, self._src.data_ptr
        self._offsets_at, self._counts_at = self._offsets.data_ptr, self._counts.data_ptr
        self._workspace_at = self._workspace.data_ptr


def _rows_of(t, name):
    """The columns of a matrix of a floating type, and the type."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D matrix")
    dtype = t.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"{name} has dtype {dtype}, expected bfloat16, float16 or float32")
    return t.shape[1], dtype


def moe_sort(expert_idx, plan: MoePlan, noop_flag=None, stream=None) -> None:
    """Fill the plan from expert_idx [T, K] (int32 or int64).  The sort is
    stable; an index outside [0, E), -1 say, drops the slot."""
    dtype = getattr(expert_idx, "dtype", None)
    # one dtype is the short way through _ptr
    idx = _ptr(expert_idx, "expert_idx", dtype if dtype in _INDEX else _INDEX, plan._slots)
    size = plan._workspace_size
    _check(lib().moe_sort(idx, 4 if dtype is _I32 else 8, plan._tokens, plan._topk,
                          plan._experts, plan._align, plan._rows, plan._row_of_at(),
                          plan._src_at(), plan._offsets_at(), plan._counts_at(),
                          plan._workspace_at() if size else None, size,
                          _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_dispatch(x, plan: MoePlan, out, noop_flag=None, stream=None) -> None:
    """x [T, hidden] -> out [rows, hidden] of the same type."""
    hidden, dtype = _rows_of(x, "x")
    px = _ptr(x, "x", dtype, (plan._tokens, hidden))
    po = _ptr(out, "out", dtype, (plan._rows, hidden))
    _check(lib().moe_dispatch(px, plan._tokens, plan._topk, hidden, _DTYPES[dtype],
                              plan._row_of_at(), plan._src_at(), plan._rows, po,
                              _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_dispatch_backward(dout, plan: MoePlan, dx, noop_flag=None, stream=None) -> None:
    """dout [rows, hidden] -> dx [T, hidden] of the same type."""
    hidden, dtype = _rows_of(dout, "dout")
    pd = _ptr(dout, "dout", dtype, (plan._rows, hidden))
    px = _ptr(dx, "dx", dtype, (plan._tokens, hidden))
    _check(lib().moe_dispatch_backward(pd, plan._tokens, plan._topk, hidden, _DTYPES[dtype],
                                       plan._row_of_at(), plan._rows, px,
                                       _opt(noop_flag, "noop_flag"), _stream(stream)))


def fp8_moe_dispatch(x, plan: MoePlan, scale, amax, scale_inv, out, out_t=None, fmt=E4M3,
                     weights=None, noop_flag=None, stream=None) -> None:
    """bf16 x [T, hidden] -> FP8 out [rows, hidden] and, unless None, out_t
    [hidden, rows].  weights: fp32 [T, K], multiplied in before the amax and
    the cast; with dy for x, FP8 gradients for the experts' outputs."""
    hidden, _ = _rows_of(x, "x")
    px = _ptr(x, "x", torch.bfloat16, (plan._tokens, hidden))
    po = _ptr(out, "out", _U8, (plan._rows, hidden))
    pt = None if out_t is None else _ptr(out_t, "out_t", _U8, (hidden, plan._rows))
    pw = None if weights is None else _ptr(weights, "weights", _F32, plan._slots)
    _check(lib().fp8_moe_dispatch(px, plan._tokens, plan._topk, hidden, plan._src_at(),
                                  plan._rows, pw, _dev(scale, "scale", _F32, 1), _dev(amax, "amax", _F32, 1),
                                  _dev(scale_inv, "scale_inv", _F32, 1), po, pt, fmt,
                                  _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_combine(ys, plan: MoePlan, weights, out, noop_flag=None, stream=None) -> None:
    """ys [rows, hidden], weights fp32 [T, K] -> out [T, hidden] of ys' type."""
    hidden, dtype = _rows_of(ys, "ys")
    py = _ptr(ys, "ys", dtype, (plan._rows, hidden))
    po = _ptr(out, "out", dtype, (plan._tokens, hidden))
    _check(lib().moe_combine(py, plan._tokens, plan._topk, hidden, _DTYPES[dtype],
                             plan._row_of_at(), _ptr(weights, "weights", _F32, plan._slots),
                             plan._rows, po, _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_combine_backward(dout, ys, plan: MoePlan, weights, dys=None, dweights=None,
                         noop_flag=None, stream=None) -> None:
    """dout [T, hidden] -> dys [rows, hidden] and dweights fp32 [T, K]; either
    may be None (ys is read for dweights only)."""
    hidden, dtype = _rows_of(dout, "dout")
    pd = _ptr(dout, "dout", dtype, (plan._tokens, hidden))
    py = None if ys is None else _ptr(ys, "ys", dtype, (plan._rows, hidden))
    ps = None if dys is None else _ptr(dys, "dys", dtype, (plan._rows, hidden))
    pw = None if dweights is None else _ptr(dweights, "dweights", _F32, plan._slots)
    _check(lib().moe_combine_backward(pd, py, plan._tokens, plan._topk, hidden, _DTYPES[dtype],
                                      plan._row_of_at(), plan._src_at(),
                                      _ptr(weights, "weights", _F32, plan._slots), plan._rows, ps,
                                      pw, _opt(noop_flag, "noop_flag"), _stream(stream)))


# ct_router_config: tokens, experts, topk, dtype, flags, balance, z
_router_config = struct.Struct("@q4i2f").pack


def moe_router_workspace_size(tokens: int, topk: int, experts: int) -> int:
    return int(lib().moe_router_workspace_size(tokens, topk, experts))


def _router(logits, expert_idx, normalize, balance, z):
    """The call's config, the number of experts and the shape of what is per slot."""
    experts, dtype = _rows_of(logits, "logits")
    if not isinstance(expert_idx, torch.Tensor) or expert_idx.dim() != 2:
        raise ValueError("expert_idx must be a 2-D matrix")
    slots = logits.shape[0], expert_idx.shape[1]
    return _router_config(slots[0], experts, slots[1], _DTYPES[dtype], 1 if normalize else 0,
                          balance, z), experts, slots


_MASK = (torch.bool, torch.uint8)


def _mask(mask, shape, device):
    if mask is None:
        return None
    dtype = getattr(mask, "dtype", None)
    return _at(mask, "mask", dtype if dtype in _MASK else _MASK, shape, device)


def moe_router(logits, expert_idx, weights, counts, loss=None, mask=None, normalize=True,
               balance=0.0, z=0.0, workspace=None, noop_flag=None, stream=None) -> None:
    """logits [T, E] -> expert_idx int32 [T, K], the experts with the largest
    logits, best first (as moe_sort takes it), weights fp32 [T, K] (as
    moe_combine takes them), counts int32 [E + 1] (slots per expert; last, the
    tokens that are not padding) and loss fp32 [1]: balance times the balance
    loss plus z times the mean squared logsumexp.  weights are probabilities,
    with normalize divided by their sum.  mask bool or uint8 [T]: 0 for padding
    tokens, which choose expert -1.  workspace: uint8, of at least
    moe_router_workspace_size(T, K, E) bytes."""
    device, handle = _here(stream)
    cfg, experts, slots = _router(logits, expert_idx, normalize, balance, z)
    _check(lib().moe_router(
        cfg, _need(logits, "logits", logits.dtype, logits.shape, device),
        _mask(mask, slots[:1], device), _need(expert_idx, "expert_idx", _I32, slots, device),
        _need(weights, "weights", _F32, slots, device),
        _need(counts, "counts", _I32, (experts + 1,), device), _scalar(loss, "loss", device),
        *_space(workspace, device), _scalar(noop_flag, "noop_flag", device), handle))


def moe_router_backward(dweights, dloss, logits, expert_idx, counts, dlogits, mask=None,
                        normalize=True, balance=0.0, z=0.0, noop_flag=None, stream=None) -> None:
    """From dweights fp32 [T, K] and dloss fp32 [1] (either may be None: zero)
    and the forward pass's logits, mask, expert_idx and counts: dlogits [T, E]
    of the logits' type."""
    device, handle = _here(stream)
    cfg, experts, slots = _router(logits, expert_idx, normalize, balance, z)
    dtype, shape = logits.dtype, logits.shape
    _check(lib().moe_router_backward(
        cfg, _need(logits, "logits", dtype, shape, device), _mask(mask, slots[:1], device),
        _need(expert_idx, "expert_idx", _I32, slots, device),
        _need(counts, "counts", _I32, (experts + 1,), device),
        _at(dweights, "dweights", _F32, slots, device), _scalar(dloss, "dloss", device),
        _need(dlogits, "dlogits", dtype, shape, device),
        _scalar(noop_flag, "noop_flag", device), handle))
