"""Torch layer of the gated block's operators in libmmaemu.so.

As in ops.py: argument marshalling only, the operators run in the HIP kernels
(include/mmaops.h states their formulas, types and memory), results take no
part in autograd, and gradients come from the backward functions, which the
program calls itself.
"""
from __future__ import annotations

import struct
from operator import index
from typing import NamedTuple

from . import ops
from .ops import Checkpoint, _activation, _Call, _done, _load, _matrix, _saved, _vector, _weight

NORMS = {None: 0, "layer": 1, "rms": 2}

# mma_gated_linear_args and mma_gated_linear_backward_args
_GATED = struct.Struct("6i3q18Q")
_GATED_BACKWARD = struct.Struct("6i3q26Q")

# mma_residual_norm_args and mma_residual_norm_backward_args
_JOIN = struct.Struct("4i2fd3Q2q17Q")
_JOIN_BACKWARD = struct.Struct("4ifid3Q2q25Q")


def _several(call, wanted, n, dtype):
    """Vectors of n elements, one for each true value of wanted and None for the
    others, in one allocation (an allocation takes 1.9 us, a part of one 0.8).  As
    data, for a view of a tensor shares its version and may not be added to in place
    under autograd."""
    count = sum(map(bool, wanted))
    if count < 2:
        return [call.empty((n,), dtype) if w else None for w in wanted]
    rows = iter(call.empty((count, n), dtype).unbind(0))
    return [next(rows).data if w else None for w in wanted]


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
        y = ops._torch.empty_like(x)  # rows of cols elements, whatever x's stride
        rc = _load()["mma_dropout"](t, px, ldx, pr, ldr, y.data_ptr(), cols, rows, cols, p, seed,
                                    offset, state, call.raw)
    _done(rc, "mma_dropout")
    return y


def dropout_backward(dy, p, seed=0, offset=0, stream=None):
    """The gradient of dropout's x: mask dy / (1 - p), with the mask of the
    forward pass's p, seed and offset.  The residual's gradient is dy."""
    return dropout(dy, p, seed, offset, None, stream)


class ResidualParams(NamedTuple):
    """The vectors of residual_norm, cols values each or None, all of the
    matrices' type or all float32; the backward pass returns their gradients
    in the same places."""
    gate: object = None
    post_weight: object = None
    post_bias: object = None
    pre_weight: object = None
    pre_bias: object = None


class ResidualStats(NamedTuple):
    """What residual_norm_backward needs of the forward pass's norms: float32
    vectors, None where there is no such norm, the means of an rms norm too."""
    post_mean: object
    post_rstd: object
    mean: object
    rstd: object


def _norm_kind(name, what):
    if name not in NORMS:
        raise ValueError(f"{what}: unknown norm {name!r}: None, 'layer' or 'rms'")
    return NORMS[name]


def _params(params, post, pre, dt, cols, dev):
    """(the five pointers, the vectors' type)."""
    if not isinstance(params, ResidualParams):
        raise TypeError("params is a ResidualParams")
    pointers, kind = [0] * 5, None
    for i, t in enumerate(params):
        if t is None:
            continue
        name = ResidualParams._fields[i]
        if i and not (post if i < 3 else pre):
            raise ValueError(f"{name} without that norm")
        pointers[i] = _vector(t, name, cols, dev, (dt, ops._torch.float32))[0] or 0
        if kind is not None and t.dtype != kind:
            raise TypeError("the vectors must be of one type")
        kind = t.dtype
    return pointers, dt if kind is None else kind


def residual_norm(x, branch, params=ResidualParams(), post=None, pre=None, scale=1.0, eps=1e-5,
                  dropout=0.0, seed=0, offset=0, stream=None):
    """A block's output into the residual stream, and the norm before the next
    block, on the current stream (mma_residual_norm):

        r = scale x + gate drop(post(branch)),  h = pre(r)

    x, branch: rows x cols, float16, bfloat16 or float32; post, pre: "layer",
    "rms" or None; params: a ResidualParams; dropout, seed, offset: as in
    ``dropout``, whose mask it is.  h is made from r before its rounding.
    Returns (r, h, ResidualStats); h is None without a pre norm.  Outside
    autograd: the results never require grad.
    """
    call = _Call(x, "x", stream)
    px, ldx = _matrix(x, "x")
    dt, dev = x.dtype, call.dev
    t = _known(dt, "x")
    rows, cols = x.shape
    pb, ldb = _matrix(branch, "branch", dt, (rows, cols), dev)
    kp, kr = _norm_kind(post, "post"), _norm_kind(pre, "pre")
    vectors, vt = _params(params, kp, kr, dt, cols, dev)
    p, seed, offset, state = _seeds(dropout, seed, offset, dev)
    f32 = ops._torch.float32
    with call:
        r = ops._torch.empty_like(x)  # rows of cols elements, whatever x's stride
        h = ops._torch.empty_like(x) if kr else None
        stats = ResidualStats(*_several(call, (kp == 1, kp, kr == 1, kr), rows, f32))
        args = _JOIN.pack(t, ops._dt[vt], kp, kr, scale, eps, p, seed, offset, state or 0, rows,
                          cols, px, ldx, pb, ldb, *vectors, r.data_ptr(), cols,
                          h.data_ptr() if kr else 0, cols,
                          *(0 if s is None else s.data_ptr() for s in stats))
        rc = _load()["mma_residual_norm"](args, call.raw)
    _done(rc, "mma_residual_norm")
    return r, h, stats


def residual_norm_backward(dr, dh, r, branch, params, stats, post=None, pre=None, scale=1.0,
                           dropout=0.0, seed=0, offset=0, need_dx=True, need_dbranch=True,
                           need_dparams=True, stream=None):
    """Gradients of residual_norm on the current stream.

    dr, dh: the gradients of r and h; dr may be None (0) where there is a pre
    norm, dh is None without one.  r, stats: what the forward pass returned (r
    may be None without a pre norm); branch, params, post, pre, scale, dropout,
    seed, offset: what it was called with (branch may be None without a post norm
    and a gate).  Returns (dx, dbranch, ResidualParams of the vectors'
    gradients); what is not needed, or belongs to no vector, is None.
    """
    kp, kr = _norm_kind(post, "post"), _norm_kind(pre, "pre")
    lead = dh if kr else dr
    call = _Call(lead, "dh" if kr else "dr", stream)
    _matrix(lead, "dh" if kr else "dr")
    dt, dev = lead.dtype, call.dev
    t = _known(dt, "dh" if kr else "dr")
    rows, cols = shape = tuple(lead.shape)
    if not kr and dh is not None:
        raise ValueError("dh without a pre norm")
    if not isinstance(stats, ResidualStats):
        raise TypeError("stats is a ResidualStats")
    f32 = ops._torch.float32

    def matrix(m, what):
        return (0, 0) if m is None else _matrix(m, what, dt, shape, dev)

    matrices = (*matrix(dr, "dr"), *matrix(dh, "dh"), *matrix(r if kr else None, "r"),
                *matrix(branch, "branch"))
    vectors, vt = _params(params, kp, kr, dt, cols, dev)
    pointers = [_vector(s, n, rows, dev, (f32,))[0] or 0
                for n, s in zip(ResidualStats._fields, stats)]
    p, seed, offset, state = _seeds(dropout, seed, offset, dev)
    fns = _load()
    with call:
        # rows of cols elements, whatever the stride of the gradient given
        dx = ops._torch.empty_like(lead) if need_dx else None
        db = ops._torch.empty_like(lead) if need_dbranch else None
        grads = ResidualParams(*_several(
            call, [need_dparams and v is not None for v in params], cols, vt))
        args = _JOIN_BACKWARD.pack(
            t, ops._dt[vt], kp, kr, scale, 0, p, seed, offset, state or 0, rows, cols, *matrices,
            *vectors[:4], *pointers, dx.data_ptr() if need_dx else 0, cols,
            db.data_ptr() if need_dbranch else 0, cols,
            *(0 if g is None else g.data_ptr() for g in grads))
        size = fns["mma_residual_norm_backward_workspace"](args)
        ws = call.workspace(size)
        rc = fns["mma_residual_norm_backward"](args, ws.data_ptr() if size else None, size,
                                               call.raw)
    _done(rc, "mma_residual_norm_backward")
    return dx, db, grads


def _weights(w_gate, w_up, dt, dev):
    """(pointer and ld of both, transposed)."""
    pg, ldg, tg = _weight(w_gate, "w_gate", dt, dev)
    if (isinstance(w_up, ops._torch.Tensor) and w_up.dtype == dt and w_up.device == dev
            and w_up.shape == w_gate.shape and w_up.stride() == w_gate.stride()):
        return pg, ldg, w_up.data_ptr(), ldg, tg
    pu, ldu, tu = _weight(w_up, "w_up", dt, dev)
    if w_up.shape != w_gate.shape:
        raise ValueError(f"w_up must have shape {tuple(w_gate.shape)}, got {tuple(w_up.shape)}")
    if tg != tu:
        if 1 not in w_up.shape:
            raise ValueError("w_gate and w_up must be stored alike")
        # a matrix of one column is row-major however far apart its elements are,
        # one of one row the view of such a column
        tg = 0 if w_up.shape[1] == 1 else 1
        (pg, ldg), (pu, ldu) = (_matrix(w.t() if tg else w, what, dt, None, dev)
                                for w, what in ((w_gate, "w_gate"), (w_up, "w_up")))
    return pg, ldg, pu, ldu, tg


def gated_linear(x, w_gate, w_up, bias_gate=None, bias_up=None, activation="silu", keep=None,
                 out_dtype=None, stream=None):
    """y = act(x w_gate + bias_gate) * (x w_up + bias_up) on the current stream
    (mma_gated_linear).

    x: M x K, float16 or bfloat16; w_gate, w_up: K x N of the same type, both
    row-major or both the transposed view of a row-major N x K matrix; biases: N
    values of x's type or float32 (both the same), or None; activation: one of
    ops.ACTIVATIONS; out_dtype: x's type (the default) or float32.
    keep="checkpoint" also saves both products (with their biases) in 8 bits,
    keep="full" returns them in x's type: what gated_linear_backward needs.
    Returns (y, kept): kept is the pair of the gate's product and the other, or
    None.  Outside autograd: y never requires grad.
    """
    call = _Call(x, "x", stream)
    torch, dt, dev = ops._torch, x.dtype, call.dev
    if dt != torch.bfloat16 and dt != torch.float16:
        raise TypeError(f"x: expected float16 or bfloat16, got {dt}")
    px, ldx = _matrix(x, "x")
    pg, ldg, pu, ldu, wt = _weights(w_gate, w_up, dt, dev)
    m, k = x.shape
    k2, n = w_gate.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    act = _activation(activation)
    od = dt if out_dtype is None else out_dtype
    if od != dt and od != torch.float32:
        raise TypeError(f"out_dtype: expected {dt} or float32, got {od}")
    if keep not in (None, "full", "checkpoint"):
        raise ValueError("keep is None, 'full' or 'checkpoint'")
    bg, gt = _vector(bias_gate, "bias_gate", n, dev, (dt, torch.float32))
    bu, ut = _vector(bias_up, "bias_up", n, dev, (dt, torch.float32))
    if gt is not None and ut is not None and gt != ut:
        raise TypeError("bias_gate and bias_up must be of one type")
    t = ops._dt[dt]
    bt = gt if gt is not None else ut if ut is not None else t
    fns = _load()
    with call:
        y = call.empty((m, n), od)
        kept, whole, saved = None, (0, n, 0, n), (0, 0, 0, 0)
        if keep == "full":
            kept = call.empty((m, n), dt), call.empty((m, n), dt)
            whole = kept[0].data_ptr(), n, kept[1].data_ptr(), n
        elif keep == "checkpoint":
            kept = call.checkpoint((m, n), dt), call.checkpoint((m, n), dt)
            saved = tuple(p.data_ptr() for c in kept for p in (c.codes, c.scales))
        args = _GATED.pack(t, ops._dt[od], bt, act, wt, 0, m, n, k, px, ldx, pg, ldg, pu, ldu,
                           bg or 0, bu or 0, y.data_ptr(), n, *whole, *saved)
        size = fns["mma_gated_linear_workspace"](args)
        ws = call.workspace(size)
        rc = fns["mma_gated_linear"](args, ws.data_ptr() if size else None, size, call.raw)
    _done(rc, "mma_gated_linear")
    return y, kept


def gated_linear_backward(dy, x, w_gate, w_up, kept, activation="silu", need_dx=True,
                          need_dw=True, need_dbias=True, dw_dtype=None, bias_dtype=None,
                          stream=None):
    """Gradients of gated_linear on the current stream
    (mma_gated_linear_backward).

    dy: M x N; x: M x K or its Checkpoint; w_gate, w_up as in gated_linear; kept:
    the pair that it returned (two matrices or two Checkpoints).  Returns (dx,
    dw_gate, dw_up, dbias_gate, dbias_up), None for those not needed: dx of dy's
    type, the weights' laid out as they are, of dw_dtype (their type or
    float32), the biases' of bias_dtype (the same choice).  The gradients of the
    two products enter the others rounded to dy's type, which the matrix cores
    take (the biases' sum them before): the error of dx and the weights'
    gradients in that type is about 1.4 times that of rounding them alone.
    """
    call = _Call(dy, "dy", stream)
    torch, dt, dev = ops._torch, dy.dtype, call.dev
    if dt != torch.bfloat16 and dt != torch.float16:
        raise TypeError(f"dy: expected float16 or bfloat16, got {dt}")
    pd, ldd = _matrix(dy, "dy")
    pg, ldg, pu, ldu, wt = _weights(w_gate, w_up, dt, dev)
    m, n = dy.shape
    k, n2 = w_gate.shape
    if n != n2:
        raise ValueError("dy and the weights differ in their columns")
    act = _activation(activation)
    wd, bd = dw_dtype or dt, bias_dtype or dt
    for d, what in ((wd, "dw_dtype"), (bd, "bias_dtype")):
        if d != dt and d != torch.float32:
            raise TypeError(f"{what}: expected {dt} or float32, got {d}")
    px = ldx = xc = xs = 0
    if isinstance(x, Checkpoint):
        xc, xs = _saved(x, "x", (m, k), dt, dev)
    else:
        px, ldx = _matrix(x, "x", dt, (m, k), dev)
    if not isinstance(kept, (tuple, list)) or isinstance(kept, Checkpoint) or len(kept) != 2:
        raise TypeError("kept is the pair that gated_linear returned")
    whole, saved = (0, 0, 0, 0), (0, 0, 0, 0)
    if isinstance(kept[0], Checkpoint) != isinstance(kept[1], Checkpoint):
        raise TypeError("kept: two matrices or two Checkpoints")
    if isinstance(kept[0], Checkpoint):
        saved = (*_saved(kept[0], "kept[0]", (m, n), dt, dev),
                 *_saved(kept[1], "kept[1]", (m, n), dt, dev))
    else:
        whole = (*_matrix(kept[0], "kept[0]", dt, (m, n), dev),
                 *_matrix(kept[1], "kept[1]", dt, (m, n), dev))
    t = ops._dt[dt]
    fns = _load()
    with call:
        dx = call.empty((m, k), dt) if need_dx else None
        dw = [None, None]
        if need_dw:
            dw = [call.empty((n, k), wd).t() if wt else call.empty((k, n), wd) for _ in range(2)]
        db = _several(call, (need_dbias, need_dbias), n, bd)
        ldw = k if wt else n
        args = _GATED_BACKWARD.pack(
            t, ops._dt[wd], ops._dt[bd], act, wt, 0, m, n, k, pd, ldd, px, ldx, xc, xs, pg, ldg,
            pu, ldu, *whole, *saved, dx.data_ptr() if need_dx else 0, k,
            *((dw[0].data_ptr(), ldw, dw[1].data_ptr(), ldw) if need_dw else (0, 0, 0, 0)),
            *((db[0].data_ptr(), db[1].data_ptr()) if need_dbias else (0, 0)))
        size = fns["mma_gated_linear_backward_workspace"](args)
        ws = call.workspace(size)
        rc = fns["mma_gated_linear_backward"](args, ws.data_ptr() if size else None, size,
                                              call.raw)
    _done(rc, "mma_gated_linear_backward")
    return dx, *dw, *db
