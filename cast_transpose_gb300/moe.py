"""Tokens sorted by expert and back: argument checks and calls.

T tokens choose K experts each, out of E.  ``MoePlan`` holds the buffers that
``moe_sort`` fills from the router's choices and the other calls read; one plan
serves every layer and step of a batch shape.

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

import torch

from . import E4M3, _check, _dev, _opt, _stream, _U8, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32 = torch.int32


def moe_sorted_rows(tokens: int, topk: int, experts: int, align: int = 1) -> int:
    """Rows that hold every slot whatever the routing, each expert's padded
    to a multiple of ``align``."""
    return int(lib().moe_sorted_rows(tokens, topk, experts, align))


class MoePlan:
    """The buffers of one sorting: ``row_of`` int32 [T, K], ``src`` int32
    [rows], ``offsets`` int32 [E + 1], ``counts`` int32 [E].  Buffers given
    here are used, the others allocated.  ``rows`` defaults to what holds
    every slot (or to ``src``'s length); with fewer, the slots that come last
    in expert order are dropped."""

    def __init__(self, tokens, topk, experts, align=1, rows=None, device="cuda", row_of=None,
                 src=None, offsets=None, counts=None):
        need = moe_sorted_rows(tokens, topk, experts, align)
        if need == 0 and tokens * topk != 0 or min(topk, experts, align) < 1 or tokens < 0:
            raise ValueError(f"a plan for {tokens} tokens, {topk} of {experts} experts, "
                             f"align {align} is outside the limits")
        if rows is None:
            rows = need if src is None else src.numel()
        self.tokens, self.topk, self.experts, self.align, self.rows = (tokens, topk, experts,
                                                                       align, rows)

        def buffer(t, name, *shape):
            if t is None:
                return torch.empty(*shape, dtype=_I32, device=device)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
            return t

        self.row_of = buffer(row_of, "row_of", tokens, topk)
        self.src = buffer(src, "src", rows)
        self.offsets = buffer(offsets, "offsets", experts + 1)
        self.counts = buffer(counts, "counts", experts)
        size = int(lib().moe_sort_workspace_size(tokens, topk, experts))
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.row_of.device)
        # these buffers stay the plan's: checked once, here
        self._row_of = _dev(self.row_of, "row_of", _I32)
        self._src = _dev(self.src, "src", _I32)
        self._offsets = _dev(self.offsets, "offsets", _I32)
        self._counts = _dev(self.counts, "counts", _I32)
        self._workspace = self.workspace.data_ptr()


def _matrix(t, name, rows, dtypes=_DTYPES, hidden=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D matrix")
    if t.shape[0] != rows or hidden not in (None, t.shape[1]):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"({rows}, {'hidden' if hidden is None else hidden})")
    return _dev(t, name, tuple(dtypes))


def _weights(t, name, plan):
    if tuple(t.shape) != (plan.tokens, plan.topk):
        raise ValueError(f"{name} must be [tokens, topk]")
    return _dev(t, name, torch.float32)


def moe_sort(expert_idx, plan: MoePlan, noop_flag=None, stream=None) -> None:
    """Fill the plan from expert_idx [T, K] (int32 or int64).  The sort is
    stable; an index outside [0, E), -1 say, drops the slot."""
    if tuple(expert_idx.shape) != (plan.tokens, plan.topk):
        raise ValueError("expert_idx must be [tokens, topk]")
    idx = _dev(expert_idx, "expert_idx", (torch.int32, torch.int64))
    _check(lib().moe_sort(idx, expert_idx.element_size(), plan.tokens, plan.topk, plan.experts,
                          plan.align, plan.rows, plan._row_of, plan._src, plan._offsets,
                          plan._counts, plan._workspace, plan.workspace.numel(),
                          _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_dispatch(x, plan: MoePlan, out, noop_flag=None, stream=None) -> None:
    """x [T, hidden] -> out [rows, hidden] of the same type."""
    px = _matrix(x, "x", plan.tokens)
    hidden = x.shape[1]
    po = _matrix(out, "out", plan.rows, (x.dtype,), hidden)
    _check(lib().moe_dispatch(px, plan.tokens, plan.topk, hidden, _DTYPES[x.dtype], plan._row_of,
                              plan._src, plan.rows, po, _opt(noop_flag, "noop_flag"),
                              _stream(stream)))


def moe_dispatch_backward(dout, plan: MoePlan, dx, noop_flag=None, stream=None) -> None:
    """dout [rows, hidden] -> dx [T, hidden] of the same type."""
    pd = _matrix(dout, "dout", plan.rows)
    hidden = dout.shape[1]
    px = _matrix(dx, "dx", plan.tokens, (dout.dtype,), hidden)
    _check(lib().moe_dispatch_backward(pd, plan.tokens, plan.topk, hidden, _DTYPES[dout.dtype],
                                       plan._row_of, plan.rows, px, _opt(noop_flag, "noop_flag"),
                                       _stream(stream)))


def fp8_moe_dispatch(x, plan: MoePlan, scale, amax, scale_inv, out, out_t=None, fmt=E4M3,
                     weights=None, noop_flag=None, stream=None) -> None:
    """bf16 x [T, hidden] -> FP8 out [rows, hidden] and, unless None, out_t
    [hidden, rows].  weights: fp32 [T, K], multiplied in before the amax and
    the cast; with dy for x, FP8 gradients for the experts' outputs."""
    px = _matrix(x, "x", plan.tokens, (torch.bfloat16,))
    hidden = x.shape[1]
    po = _matrix(out, "out", plan.rows, _U8, hidden)
    pt = None if out_t is None else _matrix(out_t, "out_t", hidden, _U8, plan.rows)
    pw = None if weights is None else _weights(weights, "weights", plan)
    _check(lib().fp8_moe_dispatch(px, plan.tokens, plan.topk, hidden, plan._src, plan.rows, pw,
                                  _dev(scale, "scale", torch.float32, 1),
                                  _dev(amax, "amax", torch.float32, 1),
                                  _dev(scale_inv, "scale_inv", torch.float32, 1), po, pt, fmt,
                                  _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_combine(ys, plan: MoePlan, weights, out, noop_flag=None, stream=None) -> None:
    """ys [rows, hidden], weights fp32 [T, K] -> out [T, hidden] of ys' type."""
    py = _matrix(ys, "ys", plan.rows)
    hidden = ys.shape[1]
    po = _matrix(out, "out", plan.tokens, (ys.dtype,), hidden)
    _check(lib().moe_combine(py, plan.tokens, plan.topk, hidden, _DTYPES[ys.dtype], plan._row_of,
                             _weights(weights, "weights", plan), plan.rows, po,
                             _opt(noop_flag, "noop_flag"), _stream(stream)))


def moe_combine_backward(dout, ys, plan: MoePlan, weights, dys=None, dweights=None,
                         noop_flag=None, stream=None) -> None:
    """dout [T, hidden] -> dys [rows, hidden] and dweights fp32 [T, K]; either
    may be None (ys is read for dweights only)."""
    pd = _matrix(dout, "dout", plan.tokens)
    hidden, dtype = dout.shape[1], (dout.dtype,)
    py = None if ys is None else _matrix(ys, "ys", plan.rows, dtype, hidden)
    ps = None if dys is None else _matrix(dys, "dys", plan.rows, dtype, hidden)
    pw = None if dweights is None else _weights(dweights, "dweights", plan)
    _check(lib().moe_combine_backward(pd, py, plan.tokens, plan.topk, hidden, _DTYPES[dout.dtype],
                                      plan._row_of, plan._src,
                                      _weights(weights, "weights", plan), plan.rows, ps, pw,
                                      _opt(noop_flag, "noop_flag"), _stream(stream)))
