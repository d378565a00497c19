"""How the replayed step compares two runs, on host tensors."""
import math

import pytest
import torch

from bit_exact_matrix_amd import ops, replay


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_same_bits(dtype):
    t = torch.tensor([[0.0, 1.0, math.nan]], dtype=dtype)
    assert replay.same_bits(t, t.clone())
    other = t.clone()
    other[0, 0] = -0.0
    assert torch.equal(t[:, :2], other[:, :2]) and not replay.same_bits(t, other)
    assert not replay.same_bits(t, t.float() if dtype != torch.float32 else t.half())
    codes = torch.arange(256, dtype=torch.uint8)
    e4m3 = codes.view(torch.float8_e4m3fn)
    assert replay.same_bits(e4m3, e4m3.clone())
    assert not replay.same_bits(e4m3, codes.flip(0).view(torch.float8_e4m3fn))
    # rows of another layout
    assert replay.same_bits(t.t().contiguous().t(), t)


def test_a_step_is_compared_in_everything_it_leaves():
    """y, dx, six gradients, mean, rstd, and three checkpoints' codes and
    scales."""
    def tensor():
        return torch.zeros(1)

    def checkpoint():
        return ops.Checkpoint(tensor(), tensor(), torch.bfloat16)

    y, dx, grads = tensor(), tensor(), replay.Block(*(tensor() for _ in range(6)))
    saved = replay.Saved(checkpoint(), tensor(), tensor(), checkpoint(), checkpoint())
    got = {id(t) for t in replay.outputs(y, saved, dx, grads)}
    want = [y, dx, *grads, saved.mean, saved.rstd]
    for ck in (saved.x, saved.z, saved.a):
        want += [ck.codes, ck.scales]
    assert got == {id(t) for t in want}
