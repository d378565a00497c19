"""Edges of the native operators: blocks of a checkpoint that end inside the
matrix and hold values that are not finite, results beside other outputs,
activations at infinity and to the last bits of float32, rows of equal
values."""
import math

import pytest

import bit_exact_matrix_amd as mm
import ops_reference as ref
from test_gpu_ops_linear import ACTS, TILES, matrix, operands
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    """The words of a tensor, so that signed zeros and NaN compare too."""
    import torch
    size = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t.contiguous().view(size)


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


# --------------------------------------- the same bits beside other outputs
@pytest.mark.parametrize("tile", [None, *TILES])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_outputs_do_not_depend_on_what_is_kept(torch_dev, monkeypatch, tile, layout):
    """y of a forward pass that keeps z is that of one that does not, so
    that a pass and its recomputation compare word for word."""
    torch, dev = torch_dev
    if tile:
        monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES[tile])
    shapes = [(1, 64, 96), (1, 255, 100), (2, 1499, 127), (1, 1499, 1023), (2, 4097, 300),
              (2, 9000, 200), (1, 255, 2047), (16, 264, 512), (7, 96, 1024), (33, 96, 2048),
              (130, 260, 200), (300, 1000, 264)]
    for i, (m, n, k) in enumerate(shapes):
        for pad in (0, 3):
            dtype = torch.bfloat16 if i % 2 else torch.float16
            x, w = operands(torch, dev, m, n, k, dtype, layout, i, pad)
            bias = torch.randn(n, device=dev)
            res = matrix(torch, dev, m, n, dtype, i + 7, pad)
            say("linear beside z", tile, layout, m, n, k, pad)
            for act in ("none", "silu"):
                a = dict(activation=act, residual=res)
                y, _ = mm.linear(x, w, bias, **a)
                whole, z = mm.linear(x, w, bias, keep="full", **a)
                saved, ck = mm.linear(x, w, bias, keep="checkpoint", **a)
                assert torch.equal(bits(y), bits(whole)), (m, n, k, pad, act)
                assert torch.equal(bits(y), bits(saved)), (m, n, k, pad, act)


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_bias_gradient_does_not_depend_on_the_other_gradients(torch_dev, layout):
    torch, dev = torch_dev
    for i, (m, n, k) in enumerate([(17, 24, 40), (299, 260, 640), (1000, 65, 129),
                                   (512, 512, 512), (2100, 520, 264)]):
        x, w = operands(torch, dev, m, n, k, torch.bfloat16, layout, i, 0)
        dy = matrix(torch, dev, m, n, torch.bfloat16, i + 3)
        z = matrix(torch, dev, m, n, torch.bfloat16, i + 4)
        say("bias gradient beside others", layout, m, n, k)
        runs = [mm.linear_backward(dy, x, w, z, activation="silu", need_dx=dx, need_dw=dw,
                                   bias_dtype=torch.float32)[2]
                for dx in (True, False) for dw in (True, False)]
        for other in runs[1:]:
            assert torch.equal(bits(runs[0]), bits(other)), (m, n, k)


# ------------------------------------------------------------ activations
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_slopes_at_infinity(torch_dev, dt):
    """The slopes' limits, 0 and 1: a forward pass in 16 bits keeps a
    pre-activation past its type's range as an infinity."""
    torch, dev = torch_dev
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    z = torch.tensor([[-math.inf, math.inf, math.nan]], device=dev).to(dtype)
    dy, x = torch.ones_like(z), torch.ones((1, 1), dtype=dtype, device=dev)
    for act in ACTS[1:]:
        say("slopes at infinity", dt, act)
        dx, _, db = mm.linear_backward(dy, x, torch.ones_like(z), z, activation=act,
                                       bias_dtype=torch.float32)
        assert db[:2].tolist() == [0.0, 1.0], act
        assert act == "relu" or math.isnan(float(db[2])), act
    big = torch.full((3, 64), 3e4, dtype=torch.float16, device=dev)
    w = torch.ones((64, 40), dtype=torch.float16, device=dev)
    w[:, ::2] = -1
    for act in ACTS[1:]:
        _, z = mm.linear(big, w, activation=act, keep="full")
        assert torch.isinf(z).all()
        _, _, db = mm.linear_backward(torch.ones_like(z), big, w, z, activation=act)
        assert (db[::2] == 0).all() and (db[1::2] == 3).all(), act


def every_half(torch, dev, top):
    """Every float16 number of magnitude up to top, as a row."""
    v = torch.arange(65536, dtype=torch.int32, device=dev).to(torch.int16).view(torch.float16)
    return v[v.abs() <= top].reshape(1, -1)


def test_gelu_to_float32(torch_dev):
    """gelu(z) = max(z, 0) - |z| Q(|z|) with the normal tail Q as 2 to the
    power of its logarithm, which is held in float32 and grows as z^2 / 2: a
    few roundings of it (6 with the power's and the sum's) are a relative
    error of 6 U (1 + z^2 / 2), of the result's magnitude where z < 0 and
    less of it elsewhere.  An approximation to 1.5e-7 of 1 exceeds it."""
    torch, dev = torch_dev
    z = every_half(torch, dev, 6.0).t().contiguous()
    one = torch.ones((1, 1), dtype=torch.float16, device=dev)
    say("gelu to float32")
    y, kept = mm.linear(z, one, activation="gelu", keep="full", out_dtype=torch.float32)
    assert torch.equal(kept, z)
    want = ref.act(z.double(), "gelu")
    ref.close(y, want, 6 * ref.U * (1 + z.double() ** 2 / 2) * want.abs(), "gelu")
    # past 13 nothing is left of the tail
    far = torch.tensor([[13.5], [20.0], [300.0], [6e4]], dtype=torch.float16, device=dev)
    y, _ = mm.linear(far, one, activation="gelu", out_dtype=torch.float32)
    assert torch.equal(y, far.float())
    y, _ = mm.linear(-far, one, activation="gelu", out_dtype=torch.float32)
    assert not y.any()


def test_gelu_slope_to_float32(torch_dev):
    """Phi(z) + z phi(z): each term below 1, in a few roundings (4) of values
    below 1."""
    torch, dev = torch_dev
    z = every_half(torch, dev, 12.0)
    one = torch.ones((1, 1), dtype=torch.float16, device=dev)
    say("gelu's slope to float32")
    _, _, db = mm.linear_backward(torch.ones_like(z), one, torch.ones_like(z), z,
                                  activation="gelu", need_dx=False, need_dw=False,
                                  bias_dtype=torch.float32)
    want = ref.act_slope(z.double(), "gelu")[0]
    ref.close(db, want, torch.full_like(want, 4 * ref.U), "gelu's slope")


# ------------------------------------------------- rows without spread
@pytest.mark.parametrize("cols", [5, 77, 1000, 8200, 20000])
@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
def test_rows_of_equal_values(torch_dev, dt, cols):
    """A row of equal values c has y = b, also where its float32 sum is not
    exact.  Where c is more than four times sqrt(eps) the mean is corrected:
    it is off by no more than its own rounding, U |c|, and a few U of what was
    corrected; elsewhere its few roundings (8 here) are 8 U 4 of y."""
    torch, dev = torch_dev
    dtype = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[dt]
    c = torch.tensor([[12345.678], [-0.1], [1e-3], [3.0], [60000.0], [1.1]], device=dev).to(dtype)
    x = c.expand(len(c), cols).contiguous()
    w = torch.ones(cols, device=dev)
    b = torch.randn(cols, device=dev)
    say("rows of equal values", dt, cols)
    y, mean, rstd, _ = mm.layer_norm(x, w, b, eps=1e-5)
    exact = c[:, 0].double()
    off = (mean.double() - exact).abs()
    assert (off <= torch.where(exact.abs() > 4 * 1e-5 ** 0.5, 2, 8) * ref.U * exact.abs()).all()
    off = (y.double() - b.double()).abs()
    assert (off <= 32 * ref.U + ref.ROUND[dtype] * b.double().abs() * 2).all()


def test_rows_of_small_spread(torch_dev):
    """Rows with an offset of 10^2 to 10^5 times their spread, against
    float64: the mean's own rounding (U |mean|) moves y by U |mean| rstd, and
    so do the elements' differences from it; a row beside them is not
    touched."""
    torch, dev = torch_dev
    g = torch.Generator(device=dev).manual_seed(3)
    for cols in (77, 700, 1000, 3000, 9000, 20000):
        x = torch.randn((9, cols), generator=g, device=dev)
        alone = mm.layer_norm(x[4:5].contiguous())[0]
        offset = torch.tensor([1e2, -1e3, 1e4, 1e5, 0, 3, 5, -1e5, 1e4], device=dev)[:, None]
        x += offset
        say("rows of small spread", cols)
        y, mean, rstd, _ = mm.layer_norm(x)
        assert torch.equal(y[4:5], alone)
        xd = x.double()
        m = xd.mean(1, keepdim=True)
        r = 1 / torch.sqrt((xd - m).square().mean(1, keepdim=True) + 1e-5)
        want = (xd - m) * r
        room = 4 * ref.U * m.abs() * r + 64 * ref.U * (want.abs() + 1)
        ref.close(y, want, room, "y")


# ------------------------------------------------------- beside autograd
def test_results_are_outside_autograd(torch_dev):
    """As documented: arguments that require grad are taken, and give results
    that do not."""
    torch, dev = torch_dev
    x = torch.randn((4, 64), device=dev).bfloat16().requires_grad_()
    w = torch.randn((64, 32), device=dev).bfloat16().requires_grad_()
    v = torch.ones(64, device=dev, requires_grad=True)
    y, _ = mm.linear(x, w)
    h, mean, rstd, _ = mm.layer_norm(x, v, v)
    grads = mm.linear_backward(y, x, w) + mm.layer_norm_backward(h, x, v, mean, rstd)
    assert not any(t.requires_grad for t in (y, h, mean, rstd, *grads))
    for f in (mm.ops, mm.linear, mm.layer_norm):
        assert "autograd" in f.__doc__
