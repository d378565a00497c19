"""The replayed training step: the operators together, against float64
autograd of the same block, and its own two findings."""
import pytest

from bit_exact_matrix_amd import replay
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,sizes", [("bf16", (300, 96, 260)), ("fp16", (64, 256, 512)),
                                         ("bf16", (1, 64, 128))])
def test_step_against_autograd(torch_dev, dtype, sizes):
    """E4M3 keeps values to within 2^-4; uniform errors of that size are off
    by 2^-4 / sqrt(3) in the mean (0.036), in each of up to three places
    that a gradient passes (the checkpoints of x, z and a; h is made from
    the first): 0.11 with all of one sign.  y sees 16-bit roundings only:
    of h, a and y, 2^-8 each."""
    torch, dev = torch_dev
    p, x, dy = replay.make(*sizes, torch.bfloat16 if dtype == "bf16" else torch.float16, 3, dev)
    say("replayed step", dtype, sizes)
    y, saved = replay.forward(x, p)
    dx, grads = replay.backward(dy, saved, p)
    leaf = [t.double().requires_grad_() for t in (x, *p)]
    lx, nw, nb, w1, b1, w2, b2 = leaf
    h = torch.nn.functional.layer_norm(lx, (sizes[1],), nw, nb, 1e-5)
    want = torch.nn.functional.gelu(h @ w1 + b1) @ w2 + b2 + lx
    want.backward(dy.double())
    want = want.detach()
    assert float((y.double() - want).norm() / want.norm()) < 3 * 2.0 ** -8
    for got, t in zip((dx, *grads), leaf):
        assert got.shape == t.grad.shape
        assert float((got.double() - t.grad).norm() / t.grad.norm()) < 0.11


def test_replay_findings(torch_dev):
    """The step repeats bit for bit.  The emulated product truncates each of
    K/16 steps at 2^-24 of the largest term and the native one rounds its
    sums: with K = 512 and terms of one size both are within 512 2^-23 of
    the exact sum of |terms|, which here is below 32 times the result."""
    for model in ("hopper", "ampere"):
        say("replay", model)
        r = replay.replay(257, 512, 384, "bf16", model, seed=5)
        assert r["repeats"]
        assert 0 < r["emulated_relative_difference"] < 32 * 512 * 2.0 ** -23
        assert r["saved_bytes"] * 1.9 < r["whole_bytes"]
