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


# ------------------------------------------------------------ gated layer
GATED = ("dtype out_dtype bias_dtype activation w_transposed reserved M N K X ldx Wg ldwg Wu ldwu "
         "bias_g bias_u Y ldy G ldg U ldu g_codes g_scales u_codes u_scales").split()
MORE = tuple(i << 36 for i in range(24, 32))
GATED_OK = dict(zip(GATED, (1, 1, 1, 4, 0, 0, 100, 96, 64, X, 64, W, 96, B, 96, R, S, Y, 96, C, 96,
                            P, 96, *MORE[:4])))


def _gated(change, ws=MORE[4], ws_bytes=1 << 30):
    v = dict(GATED_OK, **change)
    return ops.mma_gated_linear(block._GATED.pack(*(v[k] for k in GATED)), ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), DTYPE), (dict(out_dtype=0), DTYPE), (dict(bias_dtype=0), DTYPE),
    (dict(activation=5), UNSUPPORTED), (dict(w_transposed=2), UNSUPPORTED),
    (dict(reserved=1), UNSUPPORTED), (dict(M=-1), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(M=1 << 27, N=1 << 27), SHAPE), (dict(ldx=63), SHAPE), (dict(ldwg=95), SHAPE),
    (dict(ldwu=95), SHAPE), (dict(w_transposed=1, ldwu=63), SHAPE), (dict(ldy=95), SHAPE),
    (dict(ldg=95), SHAPE), (dict(ldu=95), SHAPE), (dict(X=0), NULL), (dict(Wg=0), NULL),
    (dict(Wu=0), NULL), (dict(Y=0), NULL), (dict(U=0), NULL), (dict(g_codes=0), NULL),
    (dict(u_scales=0), NULL), (dict(X=X + 1), ALIGN), (dict(Wu=B + 1), ALIGN),
    (dict(bias_u=S + 1), ALIGN), (dict(G=C + 1), ALIGN), (dict(Y=X), ALIAS), (dict(G=B), ALIAS),
    (dict(U=C + 2), ALIAS), (dict(u_codes=MORE[0] + 7), ALIAS), (dict(M=0), OK),
    (dict(N=0, ldwg=0, ldwu=0, ldy=0, ldg=0, ldu=0), OK),
])
def test_gated_linear_argument_errors(change, code):
    assert _gated(change) == code


def test_gated_linear_workspace_is_checked():
    few = dict(M=4, N=4096, K=16384, ldx=16384, ldwg=4096, ldwu=4096, ldy=4096, ldg=4096, ldu=4096)
    v = dict(GATED_OK, **few)
    need = ops.mma_gated_linear_workspace(block._GATED.pack(*(v[k] for k in GATED)))
    assert need > 0 and need % 256 == 0
    assert _gated(few, None, 0) == SCRATCH and _gated(few, MORE[4], need - 1) == SCRATCH
    assert _gated(few, MORE[4] + 16, need) == ALIGN and _gated(few, Y, need) == ALIAS
    assert ops.mma_gated_linear(None, None, 0, None) == NULL
    assert ops.mma_gated_linear_workspace(None) == 0


GATED_B = ("dtype dw_dtype bias_dtype activation w_transposed reserved M N K dY lddy X ldx x_codes "
           "x_scales Wg ldwg Wu ldwu G ldg U ldu g_codes g_scales u_codes u_scales dX lddx dWg "
           "lddwg dWu lddwu dbias_g dbias_u").split()
GATED_B_OK = dict(zip(GATED_B, (1, 1, 1, 4, 0, 0, 100, 96, 64, Y, 96, X, 64, 0, 0, W, 96, B, 96, C,
                                96, P, 96, 0, 0, 0, 0, R, 64, S, 96, Z, 96, *MORE[:2])))


def _gated_b(change, ws=MORE[4], ws_bytes=1 << 30):
    v = dict(GATED_B_OK, **change)
    return ops.mma_gated_linear_backward(block._GATED_BACKWARD.pack(*(v[k] for k in GATED_B)), ws,
                                         ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), DTYPE), (dict(dw_dtype=0), DTYPE), (dict(bias_dtype=2), DTYPE),
    (dict(activation=-1), UNSUPPORTED), (dict(reserved=3), UNSUPPORTED), (dict(K=-1), SHAPE),
    (dict(lddy=95), SHAPE), (dict(ldx=63), SHAPE), (dict(ldwu=95), SHAPE), (dict(ldu=95), SHAPE),
    (dict(lddx=63), SHAPE), (dict(lddwg=95), SHAPE), (dict(lddwu=95), SHAPE), (dict(dY=0), NULL),
    (dict(X=0), NULL), (dict(Wg=0), NULL), (dict(Wu=0), NULL), (dict(G=0), NULL), (dict(U=0), NULL),
    (dict(dWu=0), NULL), (dict(G=0, U=0), NULL), (dict(g_codes=MORE[5]), NULL),
    (dict(x_codes=MORE[5], x_scales=MORE[6]), NULL),
    (dict(G=0, U=0, g_codes=MORE[5], g_scales=MORE[6], u_codes=MORE[7]), NULL),
    (dict(dY=Y + 1), ALIGN), (dict(dw_dtype=3, dWu=Z + 2), ALIGN), (dict(dbias_u=MORE[1] + 1), ALIGN),
    (dict(dX=Y), ALIAS), (dict(dWg=B), ALIAS), (dict(dWu=S + 64), ALIAS),
    (dict(dbias_u=MORE[0] + 2), ALIAS), (dict(dbias_g=P), ALIAS),
    (dict(dX=0, dWg=0, dWu=0, dbias_g=0, dbias_u=0), OK),
])
def test_gated_linear_backward_argument_errors(change, code):
    assert _gated_b(change) == code


def test_gated_linear_backward_workspace_is_checked():
    args = block._GATED_BACKWARD.pack(*(GATED_B_OK[k] for k in GATED_B))
    need = ops.mma_gated_linear_backward_workspace(args)
    assert need >= 2 * 100 * 96 * 2
    assert _gated_b({}, None, 0) == SCRATCH and _gated_b({}, MORE[4], need - 1) == SCRATCH
    assert _gated_b({}, MORE[4] + 8, need) == ALIGN and _gated_b({}, W, need) == ALIAS
    assert ops.mma_gated_linear_backward(None, None, 0, None) == NULL
    assert ops.mma_gated_linear_backward_workspace(None) == 0


def test_gated_structures_are_what_the_binding_packs(tmp_path):
    src, exe = tmp_path / "sizes.c", str(tmp_path / "sizes")
    src.write_text('#include <stdio.h>\n#include "mmaops.h"\nint main(void) {\n'
                   '  printf("%zu %zu\\n", sizeof(mma_gated_linear_args),\n'
                   "         sizeof(mma_gated_linear_backward_args));\n  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert out == [str(s.size) for s in (block._GATED, block._GATED_BACKWARD)]


@pytest.mark.parametrize("wanted", [(True, True, False, True), (False, True), (False, False)])
@pytest.mark.parametrize("grad", [True, False])
def test_vectors_of_one_allocation_are_tensors_like_any_other(wanted, grad):
    """Each may be added to in place, under autograd too, and has a version of its own."""
    torch = pytest.importorskip("torch")

    class Call:
        @staticmethod
        def empty(shape, dtype):
            return torch.empty(shape, dtype=dtype)

    with torch.set_grad_enabled(grad):
        got = block._several(Call, wanted, 3, torch.float32)
    assert [v is not None for v in got] == list(wanted)
    got = [v for v in got if v is not None]
    for i, v in enumerate(got):
        assert tuple(v.shape) == (3,) and v.is_contiguous() and not v.requires_grad
        v.fill_(i)
    versions = [v._version for v in got]
    for v in got[:1]:
        v.add_(torch.ones(3, requires_grad=True))
        assert v.requires_grad
    assert [v._version for v in got[1:]] == versions[1:]
    assert [v.tolist() for v in got[1:]] == [[i] * 3 for i in range(1, len(got))]


@pytest.mark.parametrize("change", [
    dict(post=0, post_weight=VECTORS[1] + 1), dict(post=0, post_bias=VECTORS[2] + 1),
    dict(post=0, post_mean=STATS[0] + 1), dict(post=0, post_rstd=STATS[1] + 1),
    dict(pre=0, pre_weight=VECTORS[3] + 1), dict(pre=0, pre_bias=VECTORS[4] + 1),
    dict(pre=0, mean=STATS[2] + 1), dict(pre=0, rstd=STATS[3] + 1), dict(pre=0, H=Y + 1, ldh=1),
])
def test_residual_norm_does_not_look_at_an_absent_norm(change):
    """Pointers of a norm that is not there may be anything: the call is refused for
    what comes after its checks of alignment."""
    assert _join(dict(change, R=X)) == ALIAS


NO_POST, NO_PRE = dict(post=0, dpost_weight=0, dpost_bias=0), dict(pre=0, dpre_weight=0, dpre_bias=0)


@pytest.mark.parametrize("change", [
    dict(NO_POST, post_weight=VECTORS[1] + 1), dict(NO_POST, post_bias=VECTORS[2] + 1),
    dict(NO_POST, post_mean=STATS[0] + 1), dict(NO_POST, post_rstd=STATS[1] + 1),
    dict(NO_POST, dgate=0, branch=B + 1, ldb=1), dict(NO_PRE, pre_weight=VECTORS[3] + 1),
    dict(NO_PRE, dH=W + 1, lddh=1), dict(NO_PRE, R=R + 1, ldr=1), dict(NO_PRE, mean=STATS[2] + 1),
    dict(NO_PRE, rstd=STATS[3] + 1), dict(post=2, post_mean=STATS[0] + 1),
    dict(pre=2, mean=STATS[2] + 1),
])
def test_residual_norm_backward_does_not_look_at_an_absent_norm(change):
    assert _join_b(dict(change, dX=X)) == ALIAS
