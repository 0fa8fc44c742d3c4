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

from . import E4M3, _check, _dev, _opt, _ptr, _stream, _U8, lib
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


def _given(t, name, dtype, shape):
    """_ptr of an optional tensor."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, name, dtype, shape)


def _dtype_of(t, name):
    try:
        return t.dtype
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None


def _matrix(t, name):
    """The shape and type of a matrix that no call can do without."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D matrix")
    return tuple(t.shape), t.dtype


def _config(shape, res_dtype, dtype, w_post, w_pre, gate, rows_per_gate, eps, branch_scale,
            residual_scale, weight_offset, post_norm, pre_norm):
    """The call's config, the type of its parameters and its gate's shape."""
    rows, hidden = shape
    first = w_post if w_post is not None else w_pre if w_pre is not None else gate
    try:
        ptype = dtype if first is None else first.dtype
    except AttributeError:
        name = "w_post" if first is w_post else "w_pre" if first is w_pre else "gate"
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if rows_per_gate is None:
        rows_per_gate = max(rows, 1)
    groups = (-(-rows // rows_per_gate) if rows_per_gate > 0 else 0, hidden)
    try:
        types = _DTYPES[dtype], _DTYPES[res_dtype], _DTYPES[ptype]
    except KeyError as e:
        raise TypeError(f"dtype {e} is not bfloat16, float16 or float32") from None
    cfg = _Config(rows, hidden, rows_per_gate, _given(w_post, "w_post", ptype, (hidden,)),
                  _given(w_pre, "w_pre", ptype, (hidden,)), _given(gate, "gate", ptype, groups),
                  eps, branch_scale, residual_scale, weight_offset, *types,
                  (1 if post_norm else 0) | (2 if pre_norm else 0))
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
    shape, rtype = _matrix(res, "res")
    rows = shape[:1]
    if u is not None:
        dtype = _dtype_of(u, "u")
    else:
        dtype = _dtype_of(y, "y") if y is not None and scale is None else rtype
    cfg, _, _ = _config(shape, rtype, dtype, w_post, w_pre, gate, rows_per_gate, eps, branch_scale,
                        residual_scale, weight_offset, post_norm, pre_norm)
    _check(lib().block_norm(
        ctypes.byref(cfg), _given(u, "u", dtype, shape), _ptr(res, "res", rtype, shape),
        _given(res_out, "res_out", rtype, shape),
        _given(y, "y", dtype if scale is None else _U8, shape),
        _given(rstd_post, "rstd_post", _F32, rows), _given(rstd_pre, "rstd_pre", _F32, rows),
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
    pass's u, res_out (res where there was no u), rstd_post and rstd_pre: du
    (with u), dres (always), and those of dw_post, dw_pre, dgate that are given, in the
    parameters' type.  workspace: uint8, of at least
    block_norm_backward_workspace_size(rows, hidden) bytes."""
    shape, rtype = _matrix(dres, "dres")
    rows, columns = shape[:1], shape[1:]
    dtype = _dtype_of(u, "u") if u is not None else _dtype_of(dy, "dy")
    cfg, ptype, groups = _config(shape, rtype, dtype, w_post, w_pre, gate, rows_per_gate, 0.0,
                                 branch_scale, residual_scale, weight_offset, post_norm, pre_norm)
    if w_post is None and w_pre is None and gate is None and not (
            dw_post is None and dw_pre is None and dgate is None):
        raise ValueError("a gradient of a weight that is not given")
    _check(lib().block_norm_backward(
        ctypes.byref(cfg), _given(dy, "dy", dtype, shape), _given(dres_out, "dres_out", rtype, shape),
        _given(u, "u", dtype, shape), _given(res_out, "res_out", rtype, shape),
        _given(rstd_post, "rstd_post", _F32, rows), _given(rstd_pre, "rstd_pre", _F32, rows),
        _given(du, "du", dtype, shape), _ptr(dres, "dres", rtype, shape),
        _given(dw_post, "dw_post", ptype, columns), _given(dw_pre, "dw_pre", ptype, columns),
        _given(dgate, "dgate", ptype, groups),
        None if workspace is None else _dev(workspace, "workspace", torch.uint8),
        0 if workspace is None else workspace.numel(), _opt(noop_flag, "noop_flag"),
        _stream(stream)))
