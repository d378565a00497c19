"""Host-side checks of the gated block's operators that need no GPU: bad
arguments are answered before anything is enqueued (fake device addresses
throughout), and the reference's own parts."""
import math

import numpy as np
import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
from bit_exact_matrix_amd import ops

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
