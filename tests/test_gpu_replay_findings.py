"""What the replayed step finds, with a mistake planted in what it looks at
(in the binding, beside the kernels)."""
import pytest

from bit_exact_matrix_amd import replay
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_emulated_rows_are_of_the_steps_product(torch_dev, monkeypatch):
    """A product that is wrong at the step's own number of rows only."""
    linear, rows = replay.ops.linear, 257

    def wrong(x, *args, **kw):
        y, kept = linear(x, *args, **kw)
        return (y + 1 if x.shape[0] == rows else y), kept

    say("replay, planted product")
    fine = replay.replay(rows, 512, 384, "bf16", "hopper", seed=5)
    monkeypatch.setattr(replay.ops, "linear", wrong)
    found = replay.replay(rows, 512, 384, "bf16", "hopper", seed=5)
    assert fine["emulated_relative_difference"] < 1e-4
    assert found["emulated_relative_difference"] > 0.1
