"""Python binding of the native training operators in libmmaemu.so.

Argument marshalling only, as in the package's binding of the emulator: the
operators run in the HIP kernels of libmmaemu.so (include/mmaops.h states
their formulas, types and memory), PyTorch supplies device memory and the
current stream, and there is no CPU fallback.

``layer_norm``, ``layer_norm_backward``, ``linear``, ``linear_backward``,
``checkpoint`` and ``restore`` take torch tensors (matrices; a row stride
larger than the row is taken as it is).  They take no part in autograd:
results never require grad, whatever the arguments do, and gradients come from
the two backward functions, which the program calls itself.  The raw C entry
points (``EXPORTED``) take integers exactly as the C functions do.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

FP16, BF16, FP32 = 0, 1, 3
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
BLOCK = 32  # elements of a checkpoint block
EXPORTED = ("mma_layer_norm", "mma_layer_norm_backward", "mma_layer_norm_backward_workspace",
            "mma_checkpoint", "mma_restore", "mma_linear", "mma_linear_workspace",
            "mma_linear_backward", "mma_linear_backward_workspace", "mma_gated_linear",
            "mma_gated_linear_workspace", "mma_gated_linear_backward",
            "mma_gated_linear_backward_workspace", "mma_dropout", "mma_residual_norm",
            "mma_residual_norm_backward",
            "mma_residual_norm_backward_workspace", "mma_ops_strerror")

# mma_linear_args and mma_linear_backward_args
_LINEAR = struct.Struct("6i3q13Q")
_BACKWARD = struct.Struct("6i3q17Q")


class MmaOpsError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {mma_ops_strerror(code)} (code {code})")


class Checkpoint(NamedTuple):
    """A matrix in 8 bits (mma_checkpoint).

    codes: rows x cols float8_e4m3fn (or uint8 of the same bytes); scales:
    rows x ceil(cols / 32) uint8, exponent + 127 of each block's power of
    two; dtype: the element type that was saved, which it restores to.
    """
    codes: object
    scales: object
    dtype: object

    @property
    def shape(self):
        return self.codes.shape


_fns = None


def _load():
    """The C functions by name, with their argument types set."""
    global _fns
    if _fns is None:
        from . import load_library
        lib = load_library()
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        f64, u64 = ctypes.c_double, ctypes.c_uint64
        types = {
            "mma_layer_norm": [i32, i32, vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, i64, i64,
                               f32, vp],
            "mma_layer_norm_backward": [i32, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, i64,
                                        vp, vp, i64, i64, vp, i64, vp],
            "mma_layer_norm_backward_workspace": [i64, i64],
            "mma_checkpoint": [i32, vp, i64, vp, vp, i64, i64, vp],
            "mma_restore": [i32, vp, vp, vp, i64, i64, i64, vp],
            "mma_linear": [vp, vp, i64, vp],
            "mma_linear_workspace": [vp],
            "mma_linear_backward": [vp, vp, i64, vp],
            "mma_linear_backward_workspace": [vp],
            "mma_gated_linear": [vp, vp, i64, vp],
            "mma_gated_linear_workspace": [vp],
            "mma_gated_linear_backward": [vp, vp, i64, vp],
            "mma_gated_linear_backward_workspace": [vp],
            "mma_dropout": [i32, vp, i64, vp, i64, vp, i64, i64, i64, f64, u64, u64, vp, vp],
            "mma_residual_norm": [vp, vp],
            "mma_residual_norm_backward": [vp, vp, i64, vp],
            "mma_residual_norm_backward_workspace": [vp],
            "mma_ops_strerror": [i32],
        }
        fns = {}
        for name, args in types.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = (ctypes.c_char_p if name == "mma_ops_strerror"
                         else i64 if name.endswith("_workspace") else i32)
            fns[name] = f
        _fns = fns
    return _fns


# ------------------------------------------------------- raw C entry points
def mma_layer_norm(*args):
    return _load()["mma_layer_norm"](*args)


def mma_layer_norm_backward(*args):
    return _load()["mma_layer_norm_backward"](*args)


def mma_layer_norm_backward_workspace(rows, cols):
    return _load()["mma_layer_norm_backward_workspace"](rows, cols)


def mma_checkpoint(*args):
    return _load()["mma_checkpoint"](*args)


def mma_restore(*args):
    return _load()["mma_restore"](*args)


def mma_linear(args, workspace, workspace_bytes, hip_stream):
    """args: the bytes of an mma_linear_args."""
    return _load()["mma_linear"](args, workspace, workspace_bytes, hip_stream)


def mma_linear_workspace(args):
    return _load()["mma_linear_workspace"](args)


def mma_linear_backward(args, workspace, workspace_bytes, hip_stream):
    """args: the bytes of an mma_linear_backward_args."""
    return _load()["mma_linear_backward"](args, workspace, workspace_bytes, hip_stream)


def mma_linear_backward_workspace(args):
    return _load()["mma_linear_backward_workspace"](args)


def mma_gated_linear(args, workspace, workspace_bytes, hip_stream):
    """args: the bytes of an mma_gated_linear_args."""
    return _load()["mma_gated_linear"](args, workspace, workspace_bytes, hip_stream)


def mma_gated_linear_workspace(args):
    return _load()["mma_gated_linear_workspace"](args)


def mma_gated_linear_backward(args, workspace, workspace_bytes, hip_stream):
    """args: the bytes of an mma_gated_linear_backward_args."""
    return _load()["mma_gated_linear_backward"](args, workspace, workspace_bytes, hip_stream)


def mma_gated_linear_backward_workspace(args):
    return _load()["mma_gated_linear_backward_workspace"](args)


def mma_dropout(*args):
    return _load()["mma_dropout"](*args)


def mma_residual_norm(args, hip_stream):
    """args: the bytes of an mma_residual_norm_args."""
    return _load()["mma_residual_norm"](args, hip_stream)


def mma_residual_norm_backward(args, workspace, workspace_bytes, hip_stream):
    """args: the bytes of an mma_residual_norm_backward_args."""
    return _load()["mma_residual_norm_backward"](args, workspace, workspace_bytes, hip_stream)


def mma_residual_norm_backward_workspace(args):
    return _load()["mma_residual_norm_backward_workspace"](args)


def mma_ops_strerror(code) -> str:
    return _load()["mma_ops_strerror"](int(code)).decode()


# ------------------------------------------------------------ torch layer
def _types():
    """{torch type: type number} and torch itself, built once."""
    import torch
    return torch, {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32}


_torch = _dt = _raw_stream = None


def _start():
    """torch and what is taken from it, on the first call."""
    global _torch, _dt, _raw_stream
    torch, types = _types()
    # the handle of a device's current stream: torch's own short way to it,
    # where this torch has it (making a Stream object takes 2.7 us)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda i: torch.cuda.current_stream(i).cuda_stream)
    _dt = types
    _torch = torch  # last: what another thread's call looks at


def _matrix(t, what, dtype=None, shape=None, dev=None):
    """(pointer, row stride) of a matrix with unit stride along its rows."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    if dev is not None and t.device != dev:
        raise ValueError(f"{what} is on {t.device}, the call runs on {dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    r, c = t.shape
    ld, one = t.stride()
    if c > 1 and one != 1:
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    if r <= 1 or c == 0:
        ld = c
    elif ld < c:
        raise ValueError(f"{what}: rows overlap")
    return t.data_ptr(), ld


def _vector(t, what, n, dev, dtypes):
    """(pointer, type number) of a contiguous vector, or of none."""
    if t is None:
        return None, None
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device tensor")
    if t.device != dev:
        raise ValueError(f"{what} is on {t.device}, the call runs on {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if tuple(t.shape) != (n,):
        raise ValueError(f"{what} must have shape {(n,)}, got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr(), _dt[t.dtype]


def _saved(ck, what, shape, dtype, dev):
    """(codes, scales) pointers of a checkpoint of the given shape."""
    for t, s, sizes in ((ck.codes, shape, (1,)),
                        (ck.scales, (shape[0], -(-shape[1] // BLOCK)), (1,))):
        if not isinstance(t, _torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what}: a checkpoint is of device tensors")
        if t.device != dev:
            raise ValueError(f"{what} is on {t.device}, the call runs on {dev}")
        if tuple(t.shape) != s:
            raise ValueError(f"{what} must have shape {s}, got {tuple(t.shape)}")
        if t.element_size() not in sizes:
            raise TypeError(f"{what}: expected 1-byte elements, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
    if ck.dtype != dtype:
        raise TypeError(f"{what}: a checkpoint of {ck.dtype}, where {dtype} is used")
    return ck.codes.data_ptr(), ck.scales.data_ptr()


class _Call:
    """The device and stream of a call.  Both become current for the time of
    the call where they are not, so that torch's allocator ties outputs and
    workspace to the stream that writes them."""
    __slots__ = ("dev", "raw", "_guards")

    def __init__(self, t, what, stream):
        if _torch is None:
            _start()
        if not isinstance(t, _torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be a device tensor")
        self.dev = t.device
        self._guards = None
        cuda = _torch.cuda
        if stream is None and cuda.current_device() == self.dev.index:
            self.raw = _raw_stream(self.dev.index)
            return
        if stream is not None and stream.device != self.dev:
            raise ValueError(f"the stream is on {stream.device}, the operands on {self.dev}")
        s = stream if stream is not None else cuda.current_stream(self.dev)
        self.raw = s.cuda_stream
        self._guards = (cuda.device(self.dev), cuda.stream(s))

    def __enter__(self):
        if self._guards:
            for g in self._guards:
                g.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guards:
            for g in reversed(self._guards):
                g.__exit__(*exc)

    def empty(self, shape, dtype):
        return _torch.empty(shape, dtype=dtype, device=self.dev)

    def checkpoint(self, shape, dtype):
        r, c = shape
        return Checkpoint(self.empty((r, c), _torch.float8_e4m3fn),
                          self.empty((r, -(-c // BLOCK)), _torch.uint8), dtype)

    def workspace(self, n):
        return self.empty((n,), _torch.uint8) if n else None


def _done(rc, where):
    if rc != 0:
        raise MmaOpsError(rc, where)


def _activation(name):
    code = ACTIVATIONS.get("none" if name is None else name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return code


def layer_norm(x, weight=None, bias=None, eps=1e-5, checkpoint=False, stream=None):
    """Layer norm of the rows of x on the current stream (mma_layer_norm).

    x: rows x cols, float16, bfloat16 or float32; weight, bias: cols values
    of x's type or float32 (both the same), or None.  checkpoint=True also
    saves x in 8 bits, in the same pass.
    Returns (y, mean, rstd, saved): mean and rstd are float32 vectors that
    layer_norm_backward takes, saved a Checkpoint of x or None.  Outside
    autograd: y never requires grad.
    """
    call = _Call(x, "x", stream)
    px, ldx = _matrix(x, "x")
    dt, dev = x.dtype, call.dev
    if dt not in _dt:
        raise TypeError(f"x: expected float16, bfloat16 or float32, got {dt}")
    rows, cols = x.shape
    pw, wt = _vector(weight, "weight", cols, dev, (dt, _torch.float32))
    pb, bt = _vector(bias, "bias", cols, dev, (dt, _torch.float32))
    if wt is not None and bt is not None and wt != bt:
        raise TypeError("weight and bias must be of one type")
    pt = wt if wt is not None else bt if bt is not None else _dt[dt]
    with call:
        y = _torch.empty_like(x)  # rows of cols elements, whatever x's stride
        mean, rstd = call.empty((rows,), _torch.float32), call.empty((rows,), _torch.float32)
        ck = call.checkpoint((rows, cols), dt) if checkpoint else None
        rc = _load()["mma_layer_norm"](
            _dt[dt], pt, px, ldx, pw, pb, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(),
            ck.codes.data_ptr() if ck else None, ck.scales.data_ptr() if ck else None, rows,
            cols, eps, call.raw)
    _done(rc, "mma_layer_norm")
    return y, mean, rstd, ck


def layer_norm_backward(dy, x, weight, mean, rstd, need_dx=True, need_dparams=True, stream=None):
    """Gradients of layer_norm on the current stream.

    dy: rows x cols; x: the forward pass's input, or its Checkpoint; weight,
    mean, rstd as there.  Returns (dx, dweight, dbias); dx is None without
    need_dx, the other two (of weight's type, or dy's where weight is None)
    without need_dparams.
    """
    call = _Call(dy, "dy", stream)
    pd, ldd = _matrix(dy, "dy")
    dt, dev = dy.dtype, call.dev
    if dt not in _dt:
        raise TypeError(f"dy: expected float16, bfloat16 or float32, got {dt}")
    rows, cols = dy.shape
    px = ldx = codes = scales = None
    if isinstance(x, Checkpoint):
        codes, scales = _saved(x, "x", (rows, cols), dt, dev)
    else:
        px, ldx = _matrix(x, "x", dt, (rows, cols), dev)
    f32 = _torch.float32
    pw, wt = _vector(weight, "weight", cols, dev, (dt, f32))
    pm, _ = _vector(mean, "mean", rows, dev, (f32,))
    pr, _ = _vector(rstd, "rstd", rows, dev, (f32,))
    ptype = dt if weight is None else weight.dtype
    with call:
        dx = call.empty((rows, cols), dt) if need_dx else None
        dw = db = ws = None
        n = 0
        if need_dparams:
            dw, db = call.empty((cols,), ptype), call.empty((cols,), ptype)
            n = _load()["mma_layer_norm_backward_workspace"](rows, cols)
            ws = call.workspace(n)
        rc = _load()["mma_layer_norm_backward"](
            _dt[dt], _dt[ptype], pd, ldd, px, ldx or 0, codes, scales, pw, pm, pr,
            dx.data_ptr() if need_dx else None, cols, dw.data_ptr() if need_dparams else None,
            db.data_ptr() if need_dparams else None, rows, cols,
            ws.data_ptr() if ws is not None else None, n, call.raw)
    _done(rc, "mma_layer_norm_backward")
    return dx, dw, db


def checkpoint(x, stream=None):
    """x (rows x cols, float16, bfloat16 or float32) in 8 bits: a Checkpoint."""
    call = _Call(x, "x", stream)
    px, ldx = _matrix(x, "x")
    if x.dtype not in _dt:
        raise TypeError(f"x: expected float16, bfloat16 or float32, got {x.dtype}")
    rows, cols = x.shape
    with call:
        ck = call.checkpoint((rows, cols), x.dtype)
        rc = _load()["mma_checkpoint"](_dt[x.dtype], px, ldx, ck.codes.data_ptr(),
                                       ck.scales.data_ptr(), rows, cols, call.raw)
    _done(rc, "mma_checkpoint")
    return ck


def restore(ck, dtype=None, stream=None):
    """The matrix of a Checkpoint, in the type that was saved or in dtype."""
    if not isinstance(ck, Checkpoint):
        raise TypeError("restore takes a Checkpoint")
    call = _Call(ck.codes, "codes", stream)
    dt = ck.dtype if dtype is None else dtype
    if dt not in _dt:
        raise TypeError(f"expected float16, bfloat16 or float32, got {dt}")
    if ck.codes.dim() != 2:
        raise ValueError("codes must be a matrix")
    rows, cols = ck.codes.shape
    pc, ps = _saved(ck, "checkpoint", (rows, cols), ck.dtype, call.dev)
    with call:
        y = call.empty((rows, cols), dt)
        rc = _load()["mma_restore"](_dt[dt], pc, ps, y.data_ptr(), cols, rows, cols, call.raw)
    _done(rc, "mma_restore")
    return y


def _weight(w, what, dtype, dev):
    """(pointer, ld, transposed) of a K x N weight: its rows adjacent, or
    its columns (a transposed view of an N x K matrix)."""
    if not isinstance(w, _torch.Tensor) or not w.is_cuda:
        raise TypeError(f"{what} must be a device tensor")
    if w.dim() == 2 and w.stride(1) != 1 and w.stride(0) == 1:
        p, ld = _matrix(w.t(), what, dtype, None, dev)
        return p, ld, 1
    p, ld = _matrix(w, what, dtype, None, dev)
    return p, ld, 0


def linear(x, w, bias=None, activation=None, residual=None, keep=None, out_dtype=None,
           stream=None):
    """y = act(x w + bias) + residual on the current stream (mma_linear).

    x: M x K, float16 or bfloat16; w: K x N of the same type, row-major or
    the transposed view of a row-major N x K matrix (``weight.t()``); bias:
    N values of x's type or float32; residual: M x N of the output's type;
    activation: one of ACTIVATIONS; out_dtype: x's type (the default) or
    float32.  keep="checkpoint" also saves z = x w + bias in 8 bits,
    keep="full" returns it in x's type: what linear_backward needs of it.
    Returns (y, kept), kept None without keep.  Outside autograd: y never
    requires grad.
    """
    call = _Call(x, "x", stream)
    dt, dev = x.dtype, call.dev
    if dt != _torch.bfloat16 and dt != _torch.float16:
        raise TypeError(f"x: expected float16 or bfloat16, got {dt}")
    px, ldx = _matrix(x, "x")
    pw, ldw, wt = _weight(w, "w", dt, dev)
    m, k = x.shape
    k2, n = w.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    act = _activation(activation)
    od = dt if out_dtype is None else out_dtype
    if od != dt and od != _torch.float32:
        raise TypeError(f"out_dtype: expected {dt} or float32, got {od}")
    if keep not in (None, "full", "checkpoint"):
        raise ValueError("keep is None, 'full' or 'checkpoint'")
    pb, bt = _vector(bias, "bias", n, dev, (dt, _torch.float32))
    pr, ldr = (None, 0) if residual is None else _matrix(residual, "residual", od, (m, n), dev)
    t = _dt[dt]
    fns = _load()
    with call:
        y = call.empty((m, n), od)
        kept, pz, pc, ps = None, 0, 0, 0
        if keep == "full":
            kept = call.empty((m, n), dt)
            pz = kept.data_ptr()
        elif keep == "checkpoint":
            kept = call.checkpoint((m, n), dt)
            pc, ps = kept.codes.data_ptr(), kept.scales.data_ptr()
        args = _LINEAR.pack(t, _dt[od], t if bt is None else bt, act, wt, 0, m, n, k, px, ldx,
                            pw, ldw, pb or 0, pr or 0, ldr, y.data_ptr(), n, pz, n, pc, ps)
        size = fns["mma_linear_workspace"](args)
        ws = call.workspace(size)
        rc = fns["mma_linear"](args, ws.data_ptr() if size else None, size, call.raw)
    _done(rc, "mma_linear")
    return y, kept


def linear_backward(dy, x, w, z=None, activation=None, need_dx=True, need_dw=True,
                    need_dbias=True, dw_dtype=None, bias_dtype=None, stream=None):
    """Gradients of linear on the current stream (mma_linear_backward).

    dy: M x N; x: M x K or its Checkpoint; w as in linear; z: what linear
    kept (a matrix or a Checkpoint), needed with an activation.  Returns
    (dx, dw, dbias), None for those not needed: dx of dy's type, dw laid out
    as w is, of dw_dtype (w's type or float32), dbias of bias_dtype (the
    same choice).  The residual's gradient is dy.  The gradient of the
    pre-activation enters both products rounded to dy's type, which the matrix
    cores take (dbias sums it before): the error of dx and dw in that type is
    about 1.4 times that of rounding them alone.
    """
    call = _Call(dy, "dy", stream)
    dt, dev = dy.dtype, call.dev
    if dt != _torch.bfloat16 and dt != _torch.float16:
        raise TypeError(f"dy: expected float16 or bfloat16, got {dt}")
    pd, ldd = _matrix(dy, "dy")
    pw, ldw, wt = _weight(w, "w", dt, dev)
    m, n = dy.shape
    k, n2 = w.shape
    if n != n2:
        raise ValueError("dy and w differ in their columns")
    act = _activation(activation)
    wd, bd = dw_dtype or dt, bias_dtype or dt
    for d, what in ((wd, "dw_dtype"), (bd, "bias_dtype")):
        if d != dt and d != _torch.float32:
            raise TypeError(f"{what}: expected {dt} or float32, got {d}")
    px = ldx = xc = xs = pz = ldz = zc = zs = 0
    if isinstance(x, Checkpoint):
        xc, xs = _saved(x, "x", (m, k), dt, dev)
    else:
        px, ldx = _matrix(x, "x", dt, (m, k), dev)
    if act:
        if z is None:
            raise ValueError("the backward pass of an activation needs z")
        if isinstance(z, Checkpoint):
            zc, zs = _saved(z, "z", (m, n), dt, dev)
        else:
            pz, ldz = _matrix(z, "z", dt, (m, n), dev)
    t = _dt[dt]
    fns = _load()
    with call:
        dx = call.empty((m, k), dt) if need_dx else None
        dw = None
        if need_dw:
            dw = call.empty((n, k), wd).t() if wt else call.empty((k, n), wd)
        db = call.empty((n,), bd) if need_dbias else None
        args = _BACKWARD.pack(t, _dt[wd], _dt[bd], act, wt, 0, m, n, k, pd, ldd, px, ldx, xc,
                              xs, pw, ldw, pz, ldz, zc, zs, dx.data_ptr() if need_dx else 0, k,
                              dw.data_ptr() if need_dw else 0, k if wt else n,
                              db.data_ptr() if need_dbias else 0)
        size = fns["mma_linear_backward_workspace"](args)
        ws = call.workspace(size)
        rc = fns["mma_linear_backward"](args, ws.data_ptr() if size else None, size, call.raw)
    _done(rc, "mma_linear_backward")
    return dx, dw, db
