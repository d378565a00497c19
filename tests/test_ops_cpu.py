"""Host-side checks of the native operators that need no GPU: every entry
point of include/mmaops.h is exported and bound, and bad arguments are
answered before anything is enqueued (fake device addresses throughout)."""
import os
import re
import struct
import subprocess

import pytest

import bit_exact_matrix_amd as mm
from bit_exact_matrix_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, DTYPE, UNSUPPORTED, SHAPE, NULL, ALIAS, ALIGN, SCRATCH = 0, -2, -3, -4, -5, -6, -8, -9
X, W, B, Y, R, S, C, P, Z = (i << 36 for i in range(1, 10))  # far apart


def test_every_declared_entry_point_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "mmaops.h")).read()
    names = set(re.findall(r"^(?:int|int64_t|const char \*)\s*(mma_\w+)\s*\(", text, re.M))
    assert names == set(ops.EXPORTED)
    lib = mm.load_library()
    for name in names:
        assert hasattr(lib, name) and callable(getattr(ops, name))


def test_strerror():
    texts = {ops.mma_ops_strerror(c) for c in (0, -2, -3, -4, -5, -6, -7, -8, -9)}
    assert len(texts) == 9 and "unknown error" in ops.mma_ops_strerror(42)


# dtype, param dtype, X, ldx, weight, bias, Y, ldy, mean, rstd, codes, scales, rows, cols, eps
NORM = [1, 1, X, 64, W, B, Y, 64, R, S, C, P, 8, 64, 1e-5, None]


@pytest.mark.parametrize("at,value,code", [
    (0, 2, DTYPE), (0, 7, DTYPE), (1, 0, DTYPE), (1, 2, DTYPE),
    (13, 0, SHAPE), (13, -1, SHAPE), (12, -1, SHAPE), (3, 63, SHAPE), (7, 63, SHAPE),
    (13, 1 << 31, SHAPE), (13, (1 << 27) + 1, SHAPE), (12, 1 << 41, SHAPE),
    (2, 0, NULL), (6, 0, NULL), (8, 0, NULL), (9, 0, NULL), (10, 0, NULL), (11, 0, NULL),
    (2, X + 1, ALIGN), (4, W + 1, ALIGN), (5, B + 1, ALIGN), (6, Y + 1, ALIGN), (8, R + 2, ALIGN),
    (6, X, ALIAS), (6, X + 64, ALIAS), (6, W, ALIAS), (10, Y + 5, ALIAS), (9, R + 4, ALIAS),
    (12, 0, OK),
])
def test_layer_norm_argument_errors(at, value, code):
    args = list(NORM)
    args[at] = value
    assert ops.mma_layer_norm(*args) == code


# dtype, pdt, dY, lddy, X, ldx, codes, scales, weight, mean, rstd, dX, lddx, dw, db, rows, cols
NORM_B = [1, 1, Y, 64, X, 64, 0, 0, W, R, S, Z, 64, B, C, 8, 64, P, 1 << 20, None]


@pytest.mark.parametrize("at,value,code", [
    (0, 2, DTYPE), (1, 0, DTYPE), (16, 0, SHAPE), (15, -1, SHAPE), (3, 10, SHAPE), (5, 10, SHAPE),
    (12, 10, SHAPE), (2, 0, NULL), (4, 0, NULL), (9, 0, NULL), (10, 0, NULL), (6, C, NULL),
    (7, C, NULL), (2, Y + 1, ALIGN), (13, B + 1, ALIGN), (17, P + 128, ALIGN), (17, 0, SCRATCH),
    (18, 100, SCRATCH), (11, X, ALIAS), (11, Y + 2, ALIAS), (14, B + 2, ALIAS), (13, P, ALIAS),
])
def test_layer_norm_backward_argument_errors(at, value, code):
    args = list(NORM_B)
    args[at] = value
    assert ops.mma_layer_norm_backward(*args) == code


def test_layer_norm_backward_with_nothing_to_do():
    args = list(NORM_B)
    args[11] = args[13] = args[14] = 0
    assert ops.mma_layer_norm_backward(*args) == OK


@pytest.mark.parametrize("args,code", [
    ((2, X, 64, C, P, 8, 64, None), DTYPE), ((1, X, 10, C, P, 8, 64, None), SHAPE),
    ((1, X, 64, C, P, -8, 64, None), SHAPE), ((1, 0, 64, C, P, 8, 64, None), NULL),
    ((1, X, 64, 0, P, 8, 64, None), NULL), ((1, X, 64, C, 0, 8, 64, None), NULL),
    ((1, X + 1, 64, C, P, 8, 64, None), ALIGN), ((3, X + 2, 64, C, P, 8, 64, None), ALIGN),
    ((1, X, 64, X + 64, P, 8, 64, None), ALIAS), ((1, X, 64, C, C + 3, 8, 64, None), ALIAS),
    ((1, X, 64, C, P, 0, 64, None), OK), ((1, X, 64, C, P, 8, 0, None), OK),
])
def test_checkpoint_argument_errors(args, code):
    assert ops.mma_checkpoint(*args) == code


@pytest.mark.parametrize("args,code", [
    ((2, C, P, Y, 64, 8, 64, None), DTYPE), ((1, C, P, Y, 60, 8, 64, None), SHAPE),
    ((1, 0, P, Y, 64, 8, 64, None), NULL), ((1, C, 0, Y, 64, 8, 64, None), NULL),
    ((1, C, P, 0, 64, 8, 64, None), NULL), ((1, C, P, Y + 1, 64, 8, 64, None), ALIGN),
    ((1, C, P, C, 64, 8, 64, None), ALIAS), ((1, C, P, Y, 64, 8, 0, None), OK),
])
def test_restore_argument_errors(args, code):
    assert ops.mma_restore(*args) == code


LINEAR = ("dtype out_dtype bias_dtype activation w_transposed reserved M N K X ldx W ldw bias "
          "residual ldr Y ldy Z ldz codes scales").split()
LINEAR_OK = dict(dtype=1, out_dtype=1, bias_dtype=1, activation=2, w_transposed=0, reserved=0,
                 M=100, N=96, K=64, X=X, ldx=64, W=W, ldw=96, bias=B, residual=R, ldr=96, Y=Y,
                 ldy=96, Z=Z, ldz=96, codes=C, scales=P)


def _linear(change, ws=S, ws_bytes=1 << 30):
    v = dict(LINEAR_OK, **change)
    return ops.mma_linear(struct.pack("6i3q13Q", *(v[k] for k in LINEAR)), ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), DTYPE), (dict(dtype=2), DTYPE), (dict(out_dtype=0), DTYPE),
    (dict(bias_dtype=0), DTYPE), (dict(activation=5), UNSUPPORTED),
    (dict(activation=-1), UNSUPPORTED), (dict(w_transposed=2), UNSUPPORTED),
    (dict(reserved=1), UNSUPPORTED), (dict(M=-1), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(M=1 << 29, N=1 << 29), SHAPE), (dict(ldx=63), SHAPE), (dict(ldw=95), SHAPE),
    (dict(w_transposed=1, ldw=63), SHAPE), (dict(ldy=95), SHAPE), (dict(ldr=95), SHAPE),
    (dict(ldz=95), SHAPE), (dict(X=0), NULL), (dict(W=0), NULL), (dict(Y=0), NULL),
    (dict(codes=0), NULL), (dict(scales=0), NULL), (dict(X=X + 1), ALIGN), (dict(Y=Y + 1), ALIGN),
    (dict(bias=B + 1), ALIGN), (dict(out_dtype=3, residual=R + 2), ALIGN), (dict(Y=X), ALIAS),
    (dict(Y=R), ALIAS), (dict(Z=Y + 2), ALIAS), (dict(codes=Y + 7), ALIAS),
    (dict(M=0), OK), (dict(N=0, ldw=0, ldy=0, ldr=0, ldz=0), OK),
])
def test_linear_argument_errors(change, code):
    assert _linear(change) == code


def test_linear_workspace_is_asked_for_and_checked():
    few = dict(M=4, N=4096, K=16384, ldx=16384, ldw=4096, ldy=4096, ldr=4096, ldz=4096)
    v = dict(LINEAR_OK, **few)
    need = ops.mma_linear_workspace(struct.pack("6i3q13Q", *(v[k] for k in LINEAR)))
    assert need > 0 and need % 256 == 0
    assert _linear(few, None, 0) == SCRATCH
    assert _linear(few, S, need - 1) == SCRATCH
    assert _linear(few, S + 16, need) == ALIGN
    assert _linear(few, Y, need) == ALIAS


def test_columns_of_one_buffer_do_not_overlap():
    """Y and the residual side by side in rows of 192 elements pass the
    alias check (this one stops at the missing workspace of a call that
    needs one, before any launch); one column more on either side does not."""
    few = dict(M=4, N=4096, K=16384, ldx=16384, ldw=4096, ldz=4096, ldy=8192, ldr=8192)
    v = dict(few, Y=Y, residual=Y + 4096 * 2)
    need = ops.mma_linear_workspace(struct.pack(
        "6i3q13Q", *(dict(LINEAR_OK, **v)[k] for k in LINEAR)))
    assert _linear(dict(v, residual=Y + 4095 * 2), S, need) == ALIAS
    assert _linear(dict(v, residual=Y + 4097 * 2), S, need) == ALIAS
    assert _linear(dict(v, Z=X), S, need) == ALIAS


BACK = ("dtype dw_dtype bias_dtype activation w_transposed reserved M N K dY lddy X ldx x_codes "
        "x_scales W ldw Z ldz z_codes z_scales dX lddx dW lddw dbias").split()
BACK_OK = dict(dtype=1, dw_dtype=1, bias_dtype=1, activation=2, w_transposed=0, reserved=0, M=100,
               N=96, K=64, dY=Y, lddy=96, X=X, ldx=64, x_codes=0, x_scales=0, W=W, ldw=96, Z=Z,
               ldz=96, z_codes=0, z_scales=0, dX=R, lddx=64, dW=C, lddw=96, dbias=B)


def _back(change, ws=S, ws_bytes=1 << 30):
    v = dict(BACK_OK, **change)
    return ops.mma_linear_backward(struct.pack("6i3q17Q", *(v[k] for k in BACK)), ws, ws_bytes,
                                   None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), DTYPE), (dict(dw_dtype=0), DTYPE), (dict(bias_dtype=2), DTYPE),
    (dict(activation=9), UNSUPPORTED), (dict(K=-1), SHAPE), (dict(lddy=95), SHAPE),
    (dict(ldx=63), SHAPE), (dict(lddx=63), SHAPE), (dict(lddw=95), SHAPE), (dict(ldz=95), SHAPE),
    (dict(dY=0), NULL), (dict(W=0), NULL), (dict(X=0), NULL), (dict(Z=0), NULL),
    (dict(x_codes=P, x_scales=P + (1 << 20)), NULL), (dict(X=0, x_codes=P), NULL),
    (dict(z_codes=P, z_scales=P + (1 << 20)), NULL), (dict(dY=Y + 1), ALIGN),
    (dict(dX=R + 1), ALIGN), (dict(dw_dtype=3, dW=C + 2), ALIGN), (dict(dX=Y), ALIAS),
    (dict(dW=W), ALIAS), (dict(dbias=C), ALIAS), (dict(dX=0, dW=0, dbias=0), OK),
])
def test_linear_backward_argument_errors(change, code):
    assert _back(change) == code


def test_linear_backward_workspace_is_checked():
    need = ops.mma_linear_backward_workspace(struct.pack("6i3q17Q", *(BACK_OK[k] for k in BACK)))
    assert need >= 100 * 96 * 2
    assert _back({}, None, 0) == SCRATCH and _back({}, S, need - 1) == SCRATCH
    assert _back({}, S + 8, need) == ALIGN and _back({}, W, need) == ALIAS


def test_null_arguments():
    assert ops.mma_linear(None, None, 0, None) == NULL
    assert ops.mma_linear_backward(None, None, 0, None) == NULL
    assert ops.mma_linear_workspace(None) == 0 and ops.mma_linear_backward_workspace(None) == 0


def test_torch_layer_refuses_host_tensors():
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    v = torch.zeros(4)
    for call in (lambda: mm.layer_norm(x), lambda: mm.layer_norm_backward(x, x, None, v, v),
                 lambda: mm.linear(x, x.t()), lambda: mm.linear_backward(x, x, x),
                 lambda: mm.checkpoint(x),
                 lambda: mm.restore(mm.Checkpoint(x, x, torch.bfloat16))):
        with pytest.raises(TypeError, match="device tensor"):
            call()
    with pytest.raises(TypeError, match="Checkpoint"):
        mm.restore(x)


def test_header_compiles_as_c99(tmp_path):
    src = tmp_path / "ops.c"
    src.write_text('#include "mmaops.h"\n'
                   "int main(void) { return mma_linear(0, 0, 0, 0) == MMAEMU_ERR_NULL ? 0 : 1; }\n")
    exe = str(tmp_path / "ops")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", exe, "-L",
                    os.path.dirname(mm.LIB_PATH), "-lmmaemu",
                    "-Wl,-rpath," + os.path.dirname(mm.LIB_PATH)], check=True)
    assert subprocess.run([exe], timeout=120).returncode == 0
    # the structures are what the binding packs
    src.write_text('#include <stdio.h>\n#include "mmaops.h"\nint main(void) { printf("%zu %zu\\n", '
                   "sizeof(mma_linear_args), sizeof(mma_linear_backward_args)); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert out == [str(ops._LINEAR.size), str(ops._BACKWARD.size)]
