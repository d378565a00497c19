"""Edges of the native operators: blocks of a checkpoint that end inside the
matrix and hold values that are not finite."""
import math

import pytest

import bit_exact_matrix_amd as mm
import ops_reference as ref
from test_gpu_ops_linear import TILES
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- ragged blocks
RAGGED = [(2, 75, 131), (2, 300, 256), (16, 72, 256), (16, 75, 256), (40, 141, 200),
          (300, 77, 200), (260, 270, 136)]


@pytest.mark.parametrize("tile", [None, *TILES])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_checkpoint_of_a_ragged_block_with_special_values(torch_dev, monkeypatch, tile, layout, dt):
    """The scale goes by the block's finite elements, not by what stands
    beside the weight or by repeated columns without their bias.  Small whole
    numbers: z is exact, so codes and scales are the format's own."""
    torch, dev = torch_dev
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    if tile:
        monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES[tile])
    g = torch.Generator(device=dev).manual_seed(11)
    for m, n, k in RAGGED:
        x = torch.randint(0, 3, (m, k), generator=g, device=dev).to(dtype)
        # rows that start on 16 bytes, large numbers in the columns past n
        wide = torch.full((k, n + 16 - n % 8), 64.0, dtype=dtype, device=dev)
        wide[:, :n] = torch.randint(-1, 2, (k, n), generator=g, device=dev).to(dtype)
        wide[:, n - 1] = 2
        bias = torch.zeros(n, device=dev)
        bias[n - 1] = -2.0 * k
        w = wide[:, :n] if layout == "kn" else wide.t().contiguous().t()[:, :n]
        for special in (math.nan, math.inf, 1e30):
            bias[n - 3] = special
            z = x.double() @ w.double() + bias.double()
            if special == 1e30 and dtype != torch.float16:
                continue  # a number like others there
            say("ragged checkpoint", tile, layout, dt, m, n, k, special)
            y, ck = mm.linear(x, w, bias, keep="checkpoint")
            codes, scales, _ = ref.checkpoint(z, dtype)
            assert torch.equal(ck.scales, scales), (m, n, k, special)
            got = ck.codes.double()
            assert torch.equal(torch.isnan(got), torch.isnan(codes))
            assert torch.equal(got.nan_to_num(0), codes.nan_to_num(0)), (m, n, k, special)
