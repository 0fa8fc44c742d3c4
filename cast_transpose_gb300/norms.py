"""The junction between two blocks: the norm after a block, its gate, the
residual sum and the norm before the next block, forward and backward.

    z       = u * rstd_post * (weight_offset + w_post)
    res_out = residual_scale * res + branch_scale * gate * z
    y       = res_out * rstd_pre * (weight_offset + w_pre)

with rstd = 1 / sqrt(mean(square) + eps) of u's and of res_out's rows.  Either
norm can be left out (post_norm, pre_norm), and so can the weights (1) and the
gate (1).  Without u (before the first block) only y is made, of res.
"""
from __future__ import annotations

import ctypes

import torch

from . import E4M3, _check, _dev, _opt, _stream, _U8, lib
from .moe import _DTYPES

_F32 = torch.float32


class _Config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("rows_per_gate", ctypes.c_int64), ("w_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int), ("param_dtype", ctypes.c_int),
                ("flags", ctypes.c_int)]


def _typed(t, name, shape, dtypes):
    if t is None:
        return None
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    return _dev(t, name, dtypes)


def _config(res, dtype, w_post, w_pre, gate, rows_per_gate, eps, branch_scale, residual_scale,
            weight_offset, post_norm, pre_norm):
    """The call's config, the types of its parameters and its gate's shape."""
    rows, hidden = res.shape
    params = [t for t in (w_post, w_pre, gate) if t is not None]
    ptype = params[0].dtype if params else dtype
    if rows_per_gate is None:
        rows_per_gate = max(rows, 1)
    groups = (-(-rows // rows_per_gate) if rows_per_gate > 0 else 0, hidden)
    for t, name in ((dtype, "u and y"), (res.dtype, "res"), (ptype, "the parameters")):
        if t not in _DTYPES:
            raise TypeError(f"{name}: dtype {t} is not bfloat16, float16 or float32")
    cfg = _Config(rows, hidden, rows_per_gate, _typed(w_post, "w_post", (hidden,), ptype),
                  _typed(w_pre, "w_pre", (hidden,), ptype), _typed(gate, "gate", groups, ptype),
                  eps, branch_scale, residual_scale, weight_offset, _DTYPES[dtype],
                  _DTYPES[res.dtype], _DTYPES[ptype], (1 if post_norm else 0) |
                  (2 if pre_norm else 0))
    return cfg, ptype, groups


def block_norm(u, res, res_out=None, y=None, w_post=None, w_pre=None, gate=None,
               rows_per_gate=None, eps=1e-6, branch_scale=1.0, residual_scale=1.0,
               weight_offset=0.0, post_norm=True, pre_norm=True, rstd_post=None, rstd_pre=None,
               scale=None, amax=None, scale_inv=None, fmt=E4M3, noop_flag=None,
               stream=None) -> None:
    """u [rows, hidden] (or None), res -> res_out (res itself for an update in
    place) and y.  res is of u's type or fp32; the parameters are all of u's
    type or all fp32.  gate [groups, hidden]: row i uses gate row
    i // rows_per_gate (default: one gate row for all).  rstd_post, rstd_pre
    fp32 [rows]: kept for the backward pass.  With scale, amax and scale_inv
    (fp32 scalars) y is FP8 of format fmt, cast as fp8_cast does."""
    if res.dim() != 2:
        raise ValueError("res must be a 2-D matrix")
    shape = rows, hidden = tuple(res.shape)
    if u is not None:
        dtype = u.dtype
    else:
        dtype = y.dtype if y is not None and scale is None else res.dtype
    cfg, _, _ = _config(res, dtype, w_post, w_pre, gate, rows_per_gate, eps, branch_scale,
                        residual_scale, weight_offset, post_norm, pre_norm)
    _check(lib().block_norm(
        ctypes.byref(cfg), _typed(u, "u", shape, dtype), _typed(res, "res", shape, res.dtype),
        _typed(res_out, "res_out", shape, res.dtype),
        _typed(y, "y", shape, dtype if scale is None else _U8),
        _typed(rstd_post, "rstd_post", (rows,), _F32), _typed(rstd_pre, "rstd_pre", (rows,), _F32),
        _opt(scale, "scale"), _opt(amax, "amax"), _opt(scale_inv, "scale_inv"), fmt,
        _opt(noop_flag, "noop_flag"), _stream(stream)))


def block_norm_backward_workspace_size(rows: int, hidden: int) -> int:
    return int(lib().block_norm_backward_workspace_size(rows, hidden))


def block_norm_backward(dy, dres_out, u, res_out, rstd_post, rstd_pre, du=None, dres=None,
                        dw_post=None, dw_pre=None, dgate=None, workspace=None, w_post=None,
                        w_pre=None, gate=None, rows_per_gate=None, branch_scale=1.0,
                        residual_scale=1.0, weight_offset=0.0, post_norm=True, pre_norm=True,
                        noop_flag=None, stream=None) -> None:
    """From dy (of y) and dres_out (of res_out; None: zero), and the forward
    pass's u, res_out (res where there was no u), rstd_post and rstd_pre: du,
    dres, and those of dw_post, dw_pre, dgate that are given, in the
    parameters' type.  workspace: uint8, of at least
    block_norm_backward_workspace_size(rows, hidden) bytes."""
    if dres.dim() != 2:
        raise ValueError("dres must be a 2-D matrix")
    shape = rows, hidden = tuple(dres.shape)
    dtype = u.dtype if u is not None else dy.dtype
    cfg, ptype, groups = _config(dres, dtype, w_post, w_pre, gate, rows_per_gate, 0.0,
                                 branch_scale, residual_scale, weight_offset, post_norm, pre_norm)
    grads = [t for t in (dw_post, dw_pre, dgate) if t is not None]
    if w_post is None and w_pre is None and gate is None and grads:
        raise ValueError("a gradient of a weight that is not given")
    _check(lib().block_norm_backward(
        ctypes.byref(cfg), _typed(dy, "dy", shape, dtype),
        _typed(dres_out, "dres_out", shape, dres.dtype), _typed(u, "u", shape, dtype),
        _typed(res_out, "res_out", shape, dres.dtype),
        _typed(rstd_post, "rstd_post", (rows,), _F32), _typed(rstd_pre, "rstd_pre", (rows,), _F32),
        _typed(du, "du", shape, dtype), _typed(dres, "dres", shape, dres.dtype),
        _typed(dw_post, "dw_post", (hidden,), ptype), _typed(dw_pre, "dw_pre", (hidden,), ptype),
        _typed(dgate, "dgate", groups, ptype),
        None if workspace is None else _dev(workspace, "workspace", torch.uint8),
        0 if workspace is None else workspace.numel(), _opt(noop_flag, "noop_flag"),
        _stream(stream)))
