"""Host-side checks of the gated block's operators that need no GPU: bad
arguments are answered before anything is enqueued (fake device addresses
throughout), and the reference's own parts."""
import math
import os
import subprocess

import numpy as np
import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
from bit_exact_matrix_amd import block, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, DTYPE, UNSUPPORTED, SHAPE, NULL, ALIAS, ALIGN, SCRATCH = 0, -2, -3, -4, -5, -6, -8, -9
X, W, B, Y, R, S, C, P, Z = (i << 36 for i in range(1, 10))  # far apart


# ---------------------------------------------------------------- dropout
def test_reference_generator_against_its_published_vectors():
    """Known answers that the generator's authors publish with it."""
    for counter, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((2 ** 32 - 1,) * 4, (2 ** 32 - 1,) * 2,
             (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]:
        got = ref.philox([np.array([c]) for c in counter], key)
        assert tuple(int(w[0]) for w in got) == want


# dtype, X, ldx, residual, ldr, Y, ldy, rows, cols, p, seed, offset, state
DROP = [1, X, 64, R, 64, Y, 64, 8, 64, 0.1, 1, 2, S, None]


@pytest.mark.parametrize("at,value,code", [
    (0, 2, DTYPE), (0, -1, DTYPE), (9, -0.1, UNSUPPORTED), (9, 1.5, UNSUPPORTED),
    (9, math.nan, UNSUPPORTED), (2, 63, SHAPE), (4, 63, SHAPE), (6, 63, SHAPE), (7, -1, SHAPE),
    (8, -1, SHAPE), (8, (1 << 27) + 1, SHAPE), (7, 1 << 41, SHAPE), (1, 0, NULL), (5, 0, NULL),
    (1, X + 1, ALIGN), (3, R + 1, ALIGN), (5, Y + 1, ALIGN), (12, S + 4, ALIGN), (5, X, ALIAS),
    (5, X + 128, ALIAS), (5, R, ALIAS), (5, S - 64, ALIAS), (7, 0, OK), (8, 0, OK),
])
def test_dropout_argument_errors(at, value, code):
    args = list(DROP)
    args[at] = value
    assert ops.mma_dropout(*args) == code


def test_torch_layer_refuses_host_tensors():
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: mm.dropout(x, 0.1), lambda: mm.dropout_backward(x, 0.1)):
        with pytest.raises(TypeError, match="device tensor"):
            call()


# ------------------------------------------------- sum into the residual
JOIN = ("dtype param_dtype post pre scale eps p seed offset state rows cols X ldx branch ldb gate "
        "post_weight post_bias pre_weight pre_bias R ldr H ldh post_mean post_rstd mean rstd").split()
STATS = (10 << 36, 11 << 36, 12 << 36, 13 << 36)
VECTORS = (14 << 36, 15 << 36, 16 << 36, 17 << 36, 18 << 36)
JOIN_OK = dict(zip(JOIN, (1, 1, 1, 2, 1.0, 1e-5, 0.1, 1, 2, S, 8, 64, X, 64, B, 64, *VECTORS, R, 64,
                          Y, 64, *STATS)))


def _join(change):
    v = dict(JOIN_OK, **change)
    return ops.mma_residual_norm(block._JOIN.pack(*(v[k] for k in JOIN)), None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), DTYPE), (dict(param_dtype=0), DTYPE), (dict(post=3), UNSUPPORTED),
    (dict(pre=-1), UNSUPPORTED), (dict(p=1.01), UNSUPPORTED), (dict(p=math.nan), UNSUPPORTED),
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(ldx=63), SHAPE), (dict(ldb=63), SHAPE),
    (dict(ldr=63), SHAPE), (dict(ldh=63), SHAPE), (dict(cols=(1 << 27) + 1), SHAPE),
    (dict(X=0), NULL), (dict(branch=0), NULL), (dict(R=0), NULL), (dict(H=0), NULL),
    (dict(X=X + 1), ALIGN), (dict(gate=VECTORS[0] + 1), ALIGN), (dict(mean=STATS[2] + 2), ALIGN),
    (dict(state=S + 4), ALIGN), (dict(R=X), ALIAS), (dict(H=B), ALIAS), (dict(H=R + 64), ALIAS),
    (dict(rstd=STATS[2] + 4), ALIAS), (dict(R=VECTORS[3]), ALIAS), (dict(R=S - 8), ALIAS),
    (dict(rows=0), OK),
])
def test_residual_norm_argument_errors(change, code):
    assert _join(change) == code


JOIN_B = ("dtype param_dtype post pre scale reserved p seed offset state rows cols dR lddr dH lddh R "
          "ldr branch ldb gate post_weight post_bias pre_weight post_mean post_rstd mean rstd dX "
          "lddx dbranch lddb dgate dpost_weight dpost_bias dpre_weight dpre_bias").split()
GRADS = tuple(i << 36 for i in range(19, 24))
JOIN_B_OK = dict(zip(JOIN_B, (1, 1, 1, 1, 1.0, 0, 0.1, 1, 2, S, 8, 64, X, 64, W, 64, R, 64, B, 64,
                              *VECTORS[:4], *STATS, Y, 64, Z, 64, *GRADS)))


def _join_b(change, ws=C, ws_bytes=1 << 30):
    v = dict(JOIN_B_OK, **change)
    return ops.mma_residual_norm_backward(block._JOIN_BACKWARD.pack(*(v[k] for k in JOIN_B)), ws,
                                          ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), DTYPE), (dict(param_dtype=0), DTYPE), (dict(post=9), UNSUPPORTED),
    (dict(reserved=1), UNSUPPORTED), (dict(p=-1), UNSUPPORTED),
    (dict(post=0), UNSUPPORTED), (dict(pre=0), UNSUPPORTED),   # gradients of a norm's vectors
    (dict(cols=0), SHAPE), (dict(lddr=63), SHAPE), (dict(lddh=63), SHAPE), (dict(ldr=63), SHAPE),
    (dict(ldb=63), SHAPE), (dict(lddx=63), SHAPE), (dict(lddb=63), SHAPE), (dict(rows=-5), SHAPE),
    (dict(dH=0), NULL), (dict(R=0), NULL), (dict(rstd=0), NULL), (dict(mean=0), NULL),
    (dict(post_rstd=0), NULL), (dict(post_mean=0), NULL), (dict(branch=0), NULL),
    (dict(pre=0, dpre_weight=0, dpre_bias=0, dR=0), NULL),
    (dict(dR=X + 1), ALIGN), (dict(dgate=GRADS[0] + 1), ALIGN), (dict(state=S + 2), ALIGN),
    (dict(pre_weight=VECTORS[3] + 1), ALIGN), (dict(rstd=STATS[3] + 1), ALIGN),
    (dict(dX=X), ALIAS), (dict(dbranch=Y), ALIAS), (dict(dgate=GRADS[1] + 2), ALIAS),
    (dict(dpre_bias=R), ALIAS), (dict(rows=0, dpost_bias=GRADS[0]), ALIAS),
    (dict(dX=0, dbranch=0, dgate=0, dpost_weight=0, dpost_bias=0, dpre_weight=0, dpre_bias=0), OK),
])
def test_residual_norm_backward_argument_errors(change, code):
    assert _join_b(change) == code


def test_residual_norm_backward_workspace_is_checked():
    args = block._JOIN_BACKWARD.pack(*(JOIN_B_OK[k] for k in JOIN_B))
    need = ops.mma_residual_norm_backward_workspace(args)
    assert need > 0 and need % 256 == 0
    assert _join_b({}, None, 0) == SCRATCH and _join_b({}, C, need - 1) == SCRATCH
    assert _join_b({}, C + 8, need) == ALIGN and _join_b({}, R, need) == ALIAS
    assert ops.mma_residual_norm(None, None) == NULL
    assert ops.mma_residual_norm_backward(None, None, 0, None) == NULL
    assert ops.mma_residual_norm_backward_workspace(None) == 0


def test_structures_are_what_the_binding_packs(tmp_path):
    src, exe = tmp_path / "sizes.c", str(tmp_path / "sizes")
    names = ("mma_residual_norm_args", "mma_residual_norm_backward_args")
    src.write_text('#include <stdio.h>\n#include "mmaops.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu\\n", sizeof({n}));\n' for n in names) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert out == [str(s.size) for s in (block._JOIN, block._JOIN_BACKWARD)]
