"""Dropout on the GPU: the mask element by element against the generator's
definition, values against float64, and how a program uses it."""
import math

import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
import ops_reference
from test_gpu_ops_linear import matrix
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
DT = ["fp16", "bf16", "fp32"]


def types(torch):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 8), (2, 4099), (70, 33), (130, 200),
                                   (300, 64), (17, 2048)], ids=str)
def test_dropout(torch_dev, dt, pad, shape):
    """y is rounded once from x * up + residual: two float32 roundings (of
    the factor and of the product, each U of the product, and one of the sum)
    before it."""
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    p, seed, offset = 0.3, 0x9E3779B97F4A7C15, (7 << 32) + sum(shape)
    x, res = (matrix(torch, dev, *shape, dtype, i + shape[1], pad) for i in (1, 2))
    m = ref.mask(*shape, p, seed, offset, dev)
    say("dropout", dt, shape, pad)
    y = mm.dropout(x, p, seed, offset)
    want = ref.dropped(x.double(), m)
    assert torch.equal(y == 0, (m == 0) | (x == 0))
    ops_reference.close(y, want, 3 * ref.U * want.abs(), "y")
    y = mm.dropout(x, p, seed, offset, residual=res)
    want = want + res.double()
    ops_reference.close(y, want, 3 * ref.U * (x.double() * m).abs() + ref.U * want.abs(),
                        "y with residual")


def test_probabilities(torch_dev):
    """0 keeps everything as it is, 1 nothing; between, the share that is kept
    is the threshold's, within six standard deviations."""
    torch, dev = torch_dev
    x = matrix(torch, dev, 500, 1000, torch.float32, 1) + 3
    say("dropout probabilities")
    assert torch.equal(mm.dropout(x, 0.0, 5), x)
    assert torch.equal(mm.dropout(x, 2.0 ** -18, 5), x)          # a threshold of 0
    assert not mm.dropout(x, 1.0, 5).any()
    res = matrix(torch, dev, 500, 1000, torch.float32, 2)
    assert torch.equal(mm.dropout(x, 1.0, 5, residual=res), res)
    for p in (0.05, 0.5, 0.9, 1 - 2.0 ** -16):
        share = float((mm.dropout(x, p, 11) != 0).double().mean())
        q = 1 - ref.threshold(p) / 65536
        assert abs(share - q) <= 6 * math.sqrt(q * (1 - q) / x.numel()) + 1e-12


@pytest.mark.parametrize("dt", DT)
def test_what_is_dropped_is_zero(torch_dev, dt):
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    m = ref.mask(9, 100, 0.5, 3, 4, dev)
    for v in (math.inf, -math.inf, math.nan):
        x = torch.full((9, 100), v, dtype=dtype, device=dev)
        say("dropout of", v)
        y = mm.dropout(x, 0.5, 3, 4)
        assert not y[m == 0].any() and torch.equal(torch.isfinite(y), m == 0)


def test_backward_is_the_forward_masks(torch_dev):
    """The gradient of sum(dy * y) against differences: y is linear in x, so a
    step of 1 in every kept element moves the sum by its gradient."""
    torch, dev = torch_dev
    dy = matrix(torch, dev, 40, 300, torch.bfloat16, 1)
    ones = torch.ones((40, 300), device=dev)
    say("dropout backward")
    dx = mm.dropout_backward(dy, 0.25, 77, 1)
    step = mm.dropout(ones, 0.25, 77, 1).double()   # y(x + 1) - y(x)
    ops_reference.close(dx, step * dy.double(), 3 * ref.U * dy.double().abs() * 2, "dx")


def test_masks_go_by_place_seed_and_offset(torch_dev):
    """Rows on their own have the same mask, other seeds and offsets another."""
    torch, dev = torch_dev
    x = torch.ones((64, 512), dtype=torch.bfloat16, device=dev)
    say("dropout masks")
    y = mm.dropout(x, 0.5, 9, 1)
    assert torch.equal(mm.dropout(x[:5], 0.5, 9, 1), y[:5])
    assert torch.equal(mm.dropout(x[:, :77], 0.5, 9, 1), y[:, :77])
    assert torch.equal(mm.dropout(x.float(), 0.5, 9, 1).bfloat16(), y)
    for seed, offset in ((10, 1), (9, 2), (9 + (1 << 32), 1), (9, 1 + (1 << 32))):
        other = mm.dropout(x, 0.5, seed, offset)
        agree = float((other == y).double().mean())
        assert abs(agree - 0.5) < 6 * 0.5 / math.sqrt(x.numel())


def test_offsets_past_32_bits(torch_dev):
    """A matrix of 2.2e9 elements, its last rows against the definition."""
    torch, dev = torch_dev
    rows, cols, last = 65600, 32768 + 1024, 2
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device=dev)
    say("dropout past 32 bits")
    y = mm.dropout(x, 0.5, 21, 5)
    m = ref.mask(range(rows - last, rows), cols, 0.5, 21, 5, dev)
    assert torch.equal(y[-last:].double(), m)


def test_seed_on_the_device_in_a_captured_graph(torch_dev):
    """A graph reads the seed when it runs: new numbers, a new mask; streams
    give the same bits."""
    torch, dev = torch_dev
    x = matrix(torch, dev, 60, 700, torch.bfloat16, 1)
    seed = torch.tensor([5, 6], dtype=torch.int64, device=dev)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mm.dropout(x, 0.2, seed)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mm.dropout(x, 0.2, seed)
    for s, o in ((5, 6), (1, 2), (2 ** 63 + 5, 2 ** 64 - 1)):
        seed.copy_(torch.tensor([s - (s >> 63 << 64), o - (o >> 63 << 64)]))
        say("dropout replay", s, o)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, mm.dropout(x, 0.2, s, o))
        assert torch.equal(got, mm.dropout(x, 0.2, seed, stream=side))
        side.synchronize()


def test_empty_and_refusals(torch_dev):
    torch, dev = torch_dev
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    assert mm.dropout(x[:0], 0.5).shape == (0, 64) and mm.dropout(x[:, :0], 0.5).shape == (4, 0)
    with pytest.raises(TypeError, match="float16"):
        mm.dropout(x.double(), 0.5)
    with pytest.raises(ValueError, match="probability"):
        mm.dropout(x, 1.1)
    with pytest.raises(ValueError, match="probability"):
        mm.dropout(x, float("nan"))
    with pytest.raises(ValueError, match="seed must"):
        mm.dropout(x, 0.5, -1)
    with pytest.raises(ValueError, match="offset must"):
        mm.dropout(x, 0.5, 1, 1 << 64)
    with pytest.raises(TypeError, match="seed"):
        mm.dropout(x, 0.5, 1.5)
    with pytest.raises(TypeError, match="int64"):
        mm.dropout(x, 0.5, torch.zeros(2, device=dev))
    with pytest.raises(TypeError, match="device tensor"):
        mm.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="beside"):
        mm.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64, device=dev), 3)
    with pytest.raises(TypeError, match="residual"):
        mm.dropout(x, 0.5, residual=x.float())
    with pytest.raises(ValueError, match="adjacent"):
        mm.dropout(x.t(), 0.5)
