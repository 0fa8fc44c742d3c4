"""Dropout by a counter-based generator: nothing is stored, the gradient makes
the same choice again.

``rng`` is an int64 tensor [2] on the device, a seed and a step, which the
kernels read when they run: a program that adds 1 to the step in place, in a
captured graph or out of it, gets other choices in every step.  ``site``, one
number for each dropout of the model, tells those of a step apart.  ``p`` counts
to the nearest 1/65536.
"""
from __future__ import annotations

from . import _check, _here, _need, _random, _scalar, lib
from .moe import _DTYPES, _rows_of


def dropout(x, out, p, rng, site=0, noop_flag=None, stream=None) -> None:
    """x [rows, cols] -> out of the same type, or x itself: 0 with probability
    p, else x / (1 - p).  With the gradient of out for x, its gradient."""
    device, handle = _here(stream)
    cols, dtype = _rows_of(x, "x")
    shape = x.shape
    _check(lib().dropout(_need(x, "x", dtype, shape, device), shape[0], cols, _DTYPES[dtype], p,
                         _random(rng, p, site, device), site,
                         _need(out, "out", dtype, shape, device),
                         _scalar(noop_flag, "noop_flag", device), handle))
