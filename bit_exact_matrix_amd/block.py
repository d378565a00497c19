"""Torch layer of the gated block's operators in libmmaemu.so.

As in ops.py: argument marshalling only, the operators run in the HIP kernels
(include/mmaops.h states their formulas, types and memory), results take no
part in autograd, and gradients come from the backward functions, which the
program calls itself.
"""
from __future__ import annotations

from operator import index

from . import ops
from .ops import _Call, _done, _load, _matrix


def _known(dt, what):
    if dt not in ops._dt:
        raise TypeError(f"{what}: expected float16, bfloat16 or float32, got {dt}")
    return ops._dt[dt]


def _seeds(p, seed, offset, dev):
    """(p, seed, offset, pointer of a state on the device or None)."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"a probability is in [0, 1], got {p}")
    torch = ops._torch
    if isinstance(seed, torch.Tensor):
        if not seed.is_cuda:
            raise TypeError("seed must be an int or a device tensor")
        if seed.device != dev:
            raise ValueError(f"seed is on {seed.device}, the call runs on {dev}")
        if seed.dtype != torch.int64 or tuple(seed.shape) != (2,) or not seed.is_contiguous():
            raise TypeError("a seed on the device is a contiguous int64 tensor (seed, offset)")
        if offset != 0:
            raise ValueError("a seed on the device has the offset beside it")
        return p, 0, 0, seed.data_ptr()
    for v, what in ((seed, "seed"), (offset, "offset")):
        if not hasattr(v, "__index__"):
            raise TypeError(f"{what} must be an int, got {type(v).__name__}")
        if not 0 <= index(v) < 1 << 64:
            raise ValueError(f"{what} must be in [0, 2^64), got {v}")
    return p, index(seed), index(offset), None


def dropout(x, p, seed=0, offset=0, residual=None, stream=None):
    """y = mask x / (1 - p) + residual on the current stream (mma_dropout).

    x: rows x cols, float16, bfloat16 or float32; residual: the same, or None;
    p: the probability of an element's being dropped, in [0, 1] (met to within
    2^-17; the factor is that of the probability that is met).  The mask is a
    function of an element's row and column, seed and offset (both in [0,
    2^64)) and is not stored: the same numbers give it again, others another
    one.  seed may be an int64 device tensor (seed, offset), read when the call
    runs, so that a captured graph can be given new ones.  Outside autograd: y
    never requires grad.
    """
    call = _Call(x, "x", stream)
    px, ldx = _matrix(x, "x")
    dt, dev = x.dtype, call.dev
    t = _known(dt, "x")
    rows, cols = x.shape
    pr, ldr = (None, 0) if residual is None else _matrix(residual, "residual", dt, (rows, cols),
                                                         dev)
    p, seed, offset, state = _seeds(p, seed, offset, dev)
    with call:
        y = call.empty((rows, cols), dt)
        rc = _load()["mma_dropout"](t, px, ldx, pr, ldr, y.data_ptr(), cols, rows, cols, p, seed,
                                    offset, state, call.raw)
    _done(rc, "mma_dropout")
    return y


def dropout_backward(dy, p, seed=0, offset=0, stream=None):
    """The gradient of dropout's x: mask dy / (1 - p), with the mask of the
    forward pass's p, seed and offset.  The residual's gradient is dy."""
    return dropout(dy, p, seed, offset, None, stream)
