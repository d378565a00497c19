"""The gated layer and its backward pass on the GPU, against float64 formulas
(tests/block_reference.py), on every tile, with split inner sizes, and at the
sizes and strides where they can go wrong."""
import itertools
import math

import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
import ops_reference
from test_gpu_ops_linear import ACTS, SHAPES, TILES, matrix
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")


def operands(torch, dev, m, n, k, dtype, layout, seed, pad):
    x = matrix(torch, dev, m, k, dtype, seed, pad)
    weights = []
    for i in (1, 2):
        r, c = (k, n) if layout == "kn" else (n, k)
        w = matrix(torch, dev, r, c, dtype, seed + 10 * i, pad, max(k, 1) ** -0.5)
        weights.append(w if layout == "kn" else w.t())
    return x, *weights


def codes(ck):
    import torch
    return ck.codes.view(torch.uint8), ck.scales


def check_linear(torch, dev, m, n, k, dtype, layout, act, pad, wide_out=False, seed=0):
    x, wg, wu = operands(torch, dev, m, n, k, dtype, layout, seed, pad)
    od = torch.float32 if wide_out else dtype
    bd = torch.float32 if (m + n) % 2 else dtype
    bg, bu = torch.randn(n, device=dev).to(bd), torch.randn(n, device=dev).to(bd)
    say("gated", m, n, k, dtype, layout, act, pad)
    want, zg, zu, ey, eg, eu = ref.gated_linear(x, wg, wu, bg, bu, act)
    y, (g, u) = mm.gated_linear(x, wg, wu, bg, bu, activation=act, keep="full", out_dtype=od)
    ops_reference.close(y, want, ey, "y")
    ops_reference.close(g, zg, eg, "g")
    ops_reference.close(u, zu, eu, "u")
    y2, kept = mm.gated_linear(x, wg, wu, bg, bu, activation=act, keep="checkpoint",
                               out_dtype=od)
    assert torch.equal(y, y2), "y beside a checkpoint"
    for ck, z, ez in zip(kept, (zg, zu), (eg, eu)):
        # within the product's bound, then to 8 bits: a step of a code at most
        s = torch.exp2(ck.scales.double() - 127).repeat_interleave(32, 1)[:, :n]
        values = ck.codes.double() * s
        step = torch.maximum(z.abs() / 16, s * 2.0 ** -10)
        assert ((values - z).abs() <= step * (1 + 2.0 ** -3) + 2 * ez).all(), "checkpoint"
    y3, none = mm.gated_linear(x, wg, wu, bias_up=bu, activation=act, out_dtype=od)
    want, _, _, ey, _, _ = ref.gated_linear(x, wg, wu, None, bu, act)
    ops_reference.close(y3, want, ey, "y without the gate's bias")
    assert none is None


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_gated_linear(torch_dev, monkeypatch, tile, layout, pad):
    """Every tile on every shape, without and with split inner sizes."""
    torch, dev = torch_dev
    monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES[tile])
    for i, (m, n, k) in enumerate(SHAPES):
        dtype = torch.bfloat16 if (i + pad) % 2 else torch.float16
        if i % 3 == 1:
            monkeypatch.setenv("MMAOPS_LINEAR_SPLITS", str(1 + i % 4))
        else:
            monkeypatch.delenv("MMAOPS_LINEAR_SPLITS", raising=False)
        check_linear(torch, dev, m, n, k, dtype, layout, ACTS[(i + pad) % 5], pad,
                     wide_out=i % 4 == 2, seed=10 * i)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_gated_linear_as_chosen(torch_dev, dt, act):
    """The library's own choice of tile and splits."""
    torch, dev = torch_dev
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    for i, (m, n, k) in enumerate([(1, 1024, 1024), (4, 1000, 4096), (33, 96, 2048),
                                   (520, 1040, 96), (1024, 1024, 256), (1100, 1300, 65),
                                   (16, 4096, 512)]):
        check_linear(torch, dev, m, n, k, dtype, "kn" if i % 2 else "nk", act, 0, seed=i)


def check_backward(torch, dev, m, n, k, dtype, layout, act, pad, saved, wide=False, seed=0):
    x, wg, wu = operands(torch, dev, m, n, k, dtype, layout, seed, pad)
    dy = matrix(torch, dev, m, n, dtype, seed + 3, pad)
    g, u = (matrix(torch, dev, m, n, dtype, seed + i, pad, 1.5) for i in (4, 5))
    xa, kept = x, (g, u)
    xr, gr, ur = x.double(), g.double(), u.double()
    if saved:
        xa, kept = mm.checkpoint(x), (mm.checkpoint(g), mm.checkpoint(u))
        xr, gr, ur = (ops_reference.checkpoint(t, dtype)[2] for t in (xr, gr, ur))
    od = torch.float32 if wide else dtype
    how = dict(activation=act, dw_dtype=od, bias_dtype=od)
    say("gated backward", m, n, k, dtype, layout, act, pad, saved)
    got = mm.gated_linear_backward(dy, xa, wg, wu, kept, **how)
    values, bounds = ref.gated_linear_backward(dy, xr, wg, wu, gr, ur, act, dtype)
    for name, t, v, e in zip(NAMES, got, values, bounds):
        ops_reference.close(t, v, e, name)
    for dw in got[1:3]:
        assert dw.stride() == ((1, k) if layout == "nk" and k > 0 else (n, 1))
    for i, part in enumerate([(0,), (1, 2), (3, 4)]):
        need = [j == i for j in range(3)]
        alone = mm.gated_linear_backward(dy, xa, wg, wu, kept, need_dx=need[0], need_dw=need[1],
                                         need_dbias=need[2], **how)
        for j, t in enumerate(alone):
            assert (t is not None) == (j in part)
            if j in part and i < 2:
                assert torch.equal(t, got[j]), NAMES[j]
            elif j in part:
                ops_reference.close(t, values[j], bounds[j], NAMES[j] + " alone")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("saved", [False, True])
def test_gated_linear_backward(torch_dev, monkeypatch, tile, layout, saved):
    torch, dev = torch_dev
    monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES[tile])
    for i, (m, n, k) in enumerate(SHAPES):
        dtype = torch.bfloat16 if i % 2 else torch.float16
        if i % 3 == 1:
            monkeypatch.setenv("MMAOPS_LINEAR_SPLITS", str(1 + i % 4))
        else:
            monkeypatch.delenv("MMAOPS_LINEAR_SPLITS", raising=False)
        check_backward(torch, dev, m, n, k, dtype, layout, ACTS[i % 5], (0, 3, 8)[i % 3], saved,
                       wide=i % 4 == 2, seed=10 * i)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_gated_linear_backward_as_chosen(torch_dev, dt, act):
    torch, dev = torch_dev
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    for i, (m, n, k) in enumerate([(1, 1024, 1024), (4, 1000, 2048), (299, 260, 640),
                                   (520, 1040, 96), (1100, 1300, 65), (2048, 512, 512)]):
        check_backward(torch, dev, m, n, k, dtype, "kn" if i % 2 else "nk", act, 0, i % 3 == 0,
                       seed=i)


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_weights_with_leading_dimensions_of_their_own(torch_dev, layout):
    """Halves of one buffer, and one weight in wider rows than the other."""
    torch, dev = torch_dev
    for m, n, k in ((3, 136, 192), (130, 264, 200)):
        x, wg, wu = operands(torch, dev, m, n, k, torch.bfloat16, layout, 1, 0)
        dy = matrix(torch, dev, m, n, torch.bfloat16, 7)
        say("gated, strides apart", layout, m, n, k)
        y, kept = mm.gated_linear(x, wg, wu, keep="full")
        grads = mm.gated_linear_backward(dy, x, wg, wu, kept)
        stored = [w if layout == "kn" else w.t() for w in (wg, wu)]
        r, c = stored[0].shape
        both = torch.cat(stored, dim=1)
        halves = both[:, :c], both[:, c:]
        wide = torch.full((r, c + 24), math.nan, dtype=torch.bfloat16, device=dev)
        wide[:, :c] = stored[1]
        for a, b in (halves, (stored[0].contiguous(), wide[:, :c])):
            a, b = (a, b) if layout == "kn" else (a.t(), b.t())
            z, _ = mm.gated_linear(x, a, b)
            want, _, _, ey, _, _ = ref.gated_linear(x, wg, wu, None, None, "silu")
            ops_reference.close(z, want, ey, "y")
            values, bounds = ref.gated_linear_backward(
                dy, x.double(), wg, wu, kept[0].double(), kept[1].double(), "silu",
                torch.bfloat16)
            for name, t, v, e in zip(NAMES, mm.gated_linear_backward(dy, x, a, b, kept), values,
                                     bounds):
                ops_reference.close(t, v, e, name)
        assert all(torch.equal(s, t) for s, t in zip(
            grads, mm.gated_linear_backward(dy, x, wg, wu, kept)))


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(torch_dev, act):
    """The change of sum(c y) along random directions, in float64, against the
    gradients: the kernels' own error is their bound (from the kept products'
    rounding too: half a unit of 16 bits of g and u, through slopes of at most
    1.2 and second derivatives of at most 1.5), that of the differences h^2 / 6
    of third derivatives below 100 (relu's kink apart: c of every element
    within a step of it)."""
    torch, dev = torch_dev
    m, n, k, h = 7, 24, 40, 1e-3
    x, wg, wu = operands(torch, dev, m, n, k, torch.float16, "kn", 1, 0)
    bg, bu = torch.randn(n, device=dev), torch.randn(n, device=dev)
    c = matrix(torch, dev, m, n, torch.float16, 9)
    _, kept = mm.gated_linear(x, wg, wu, bg, bu, activation=act, keep="full")
    say("gated gradients", act)
    got = mm.gated_linear_backward(c, x, wg, wu, kept, activation=act, dw_dtype=torch.float32,
                                   bias_dtype=torch.float32)
    g, u = kept[0].double(), kept[1].double()
    _, bounds = ref.gated_linear_backward(c, x.double(), wg, wu, g, u, act, torch.float16)
    point = [x.double(), wg.double(), wu.double(), bg.double(), bu.double()]
    cd = c.double()
    half = 2.0 ** -11
    moved_g = cd.abs() * (1.2 * u.abs() + 1.5 * u.abs() * g.abs()) * half * 1.01
    moved_u = cd.abs() * (1.2 * g.abs() + 1) * half * 1.01
    moves = [moved_g @ wg.double().abs().t() + moved_u @ wu.double().abs().t(),
             x.double().abs().t() @ moved_g, x.double().abs().t() @ moved_u, moved_g.sum(0),
             moved_u.sum(0)]
    kink = (g.abs() < 10 * h).double() * cd.abs() * u.abs() if act == "relu" else 0 * cd
    kinks = [kink @ wg.double().abs().t(), x.double().abs().t() @ kink, 0 * moves[2],
             kink.sum(0), 0 * moves[4]]

    def loss(at):
        a = ops_reference.act(at[0] @ at[1] + at[3], act)
        return float((cd * a * (at[0] @ at[2] + at[4])).sum())

    for i, grad in enumerate(got):
        gen = torch.Generator(device=dev).manual_seed(i)
        v = torch.randn(grad.shape, generator=gen, device=dev).double()
        up, down = list(point), list(point)
        up[i], down[i] = point[i] + h * v, point[i] - h * v
        diff = (loss(up) - loss(down)) / (2 * h)
        mine = float((grad.double() * v).sum())
        room = float(((bounds[i] + ops_reference.ROUND[grad.dtype] * grad.double().abs()
                       + moves[i] + kinks[i]) * v.abs()).sum())
        room += h * h / 6 * 100 * float(cd.abs().sum()) * 10 + 1e-15 * abs(loss(point)) / h
        assert abs(mine - diff) <= room, (act, NAMES[i], mine, diff, room)


def test_outputs_do_not_depend_on_what_is_kept(torch_dev):
    torch, dev = torch_dev
    for layout, (m, n, k) in itertools.product(
            ("kn", "nk"), [(1, 64, 96), (1, 255, 100), (16, 264, 512), (7, 96, 1024),
                           (33, 96, 2048), (130, 260, 200), (300, 1000, 264), (600, 500, 520)]):
        x, wg, wu = operands(torch, dev, m, n, k, torch.bfloat16, layout, 1, 0)
        say("gated beside what is kept", layout, m, n, k)
        ys = [mm.gated_linear(x, wg, wu, keep=kept)[0] for kept in (None, "full", "checkpoint")]
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_checkpoints_are_those_of_the_products(torch_dev):
    """Small whole numbers: g and u are exact, so codes and scales are the
    format's own, ragged blocks and special values among them."""
    torch, dev = torch_dev
    gen = torch.Generator(device=dev).manual_seed(5)
    for (m, n, k), dtype in itertools.product(
            [(2, 75, 128), (16, 72, 256), (40, 141, 200), (300, 77, 200), (260, 270, 136)],
            (torch.float16, torch.bfloat16)):
        x = torch.randint(0, 3, (m, k), generator=gen, device=dev).to(dtype)
        wg, wu = (torch.randint(-1, 2, (k, n), generator=gen, device=dev).to(dtype)
                  for _ in range(2))
        bias = torch.zeros(n, device=dev)
        bias[n - 3] = math.nan
        say("gated checkpoints", m, n, k, dtype)
        y, kept = mm.gated_linear(x, wg, wu, bias, bias, keep="checkpoint")
        for w, ck in zip((wg, wu), kept):
            z = x.double() @ w.double() + bias.double()
            want, scales, _ = ops_reference.checkpoint(z, dtype)
            assert torch.equal(ck.scales, scales)
            got = ck.codes.double()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


def test_empty_sizes(torch_dev):
    torch, dev = torch_dev
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    b = torch.randn(5, device=dev)
    y, kept = mm.gated_linear(e(3, 0), e(0, 5), e(0, 5), b, b, activation="relu",
                              keep="checkpoint")
    assert torch.equal(y, (torch.relu(b) * b).bfloat16().expand(3, 5)) and len(kept) == 2
    for m, n in ((0, 5), (3, 0)):
        y, kept = mm.gated_linear(e(m, 4), e(4, n), e(4, n), keep="full")
        assert y.shape == (m, n)
        dx, dg, du, bg, bu = mm.gated_linear_backward(y, e(m, 4), e(4, n), e(4, n), kept)
        assert dx.shape == (m, 4) and dg.shape == du.shape == (4, n) and bg.shape == (n,)
        assert not any(t.any() for t in (dx, dg, du, bg, bu))
    dy = torch.ones((3, 5), dtype=torch.bfloat16, device=dev)
    dx, dg, du, bg, bu = mm.gated_linear_backward(dy, e(3, 0), e(0, 5), e(0, 5), (dy, dy),
                                                  activation="none")
    assert dx.shape == (3, 0) and dg.shape == (0, 5) and (bg == 3).all() and (bu == 3).all()


def test_special_values(torch_dev):
    """Rows stay by themselves; a kept infinity stands for a number."""
    torch, dev = torch_dev
    for m, n, k in ((5, 70, 200), (200, 150, 100)):
        x, wg, wu = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 1, 0)
        y0, _ = mm.gated_linear(x, wg, wu)
        x2 = x.clone()
        x2[4, 0] = math.nan
        say("gated special values", m, n, k)
        y, kept = mm.gated_linear(x2, wg, wu, keep="full")
        rest = [i for i in range(m) if i != 4]
        assert torch.equal(y[rest], y0[rest]) and torch.isnan(y[4]).all()
        w2 = wu.clone()
        w2[1, 7] = math.nan
        y, _ = mm.gated_linear(x, wg, w2)
        cols = [j for j in range(n) if j != 7]
        assert torch.equal(y[:, cols], y0[:, cols]) and torch.isnan(y[:, 7]).all()
        dy = torch.ones_like(y)
        dx, _, _, _, _ = mm.gated_linear_backward(dy, x2, wg, wu, kept)
        assert torch.isnan(dx[4]).all() and torch.isfinite(dx[rest]).all()
    # a gate far below zero, past FP16 in what is kept: no part of any gradient
    inf = math.inf
    one = torch.ones((1, 3), dtype=torch.float16, device=dev)
    g = torch.tensor([[-inf, inf, -inf]], dtype=torch.float16, device=dev)
    u = torch.tensor([[inf, 2.0, -inf]], dtype=torch.float16, device=dev)
    for act in ACTS[1:]:
        say("gated, kept infinities", act)
        dx, dg, du, bg, bu = mm.gated_linear_backward(
            one, one[:, :1], one, one, (g, u), activation=act, bias_dtype=torch.float32)
        assert torch.equal(bg, torch.tensor([0.0, 2.0, 0.0], device=dev)), act
        assert not bu[[0, 2]].any() and bu[1] > 1e6 and not dg[0, [0, 2]].any()


def test_offsets_past_32_bits(torch_dev):
    """Outputs past 2^31 elements: the last rows are those of the same rows on
    their own."""
    torch, dev = torch_dev
    m, n, k, last = 530000, 4104, 64, 200
    x = matrix(torch, dev, m, k, torch.bfloat16, 1)
    wg, wu = (matrix(torch, dev, k, n, torch.bfloat16, i, scale=0.1) for i in (2, 3))
    say("gated past 32 bits")
    y, kept = mm.gated_linear(x, wg, wu, keep="checkpoint")
    ty, tk = mm.gated_linear(x[-last:], wg, wu, keep="checkpoint")
    # another number of rows may choose another order of the sums
    values, _, _, ey, _, _ = ref.gated_linear(x[-last:], wg, wu, None, None, "silu")
    ops_reference.close(y[-last:], values, ey, "y")
    ops_reference.close(ty, values, ey, "y of the rows alone")
    y[:-last] = 0
    tail = tuple(mm.Checkpoint(c.codes[-last:].contiguous(), c.scales[-last:].contiguous(),
                               c.dtype) for c in kept)
    got = mm.gated_linear_backward(y, x, wg, wu, kept)
    assert not got[0][:-last].any()
    values, bounds = ref.gated_linear_backward(
        y[-last:], x[-last:].double(), wg, wu, mm.restore(tail[0]).double(),
        mm.restore(tail[1]).double(), "silu", torch.bfloat16)
    for name, t, v, e in zip(NAMES, (got[0][-last:], *got[1:]), values, bounds):
        ops_reference.close(t, v, e, name)


def test_repeats_streams_and_graphs(torch_dev):
    """The same bits on every call and stream, and in every replay of a
    captured pass on new inputs."""
    torch, dev = torch_dev
    side = torch.cuda.Stream(device=dev)
    for m, n, k in ((2, 1024, 2048), (96, 320, 512), (700, 900, 1100), (1024, 2048, 512)):
        x, wg, wu = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 5, 0)
        dy = matrix(torch, dev, m, n, torch.bfloat16, 6)

        def step(stream=None):
            y, kept = mm.gated_linear(x, wg, wu, keep="checkpoint", stream=stream)
            grads = mm.gated_linear_backward(dy, x, wg, wu, kept, stream=stream)
            return [y, *codes(kept[0]), *codes(kept[1]), *grads]

        side.wait_stream(torch.cuda.current_stream())
        say("gated repeats", m, n, k)
        first, other = step(), step(side)
        side.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(first, other))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(3):
            x.copy_(matrix(torch, dev, m, k, torch.bfloat16, 100 + i))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            assert all(torch.equal(s, t) for s, t in zip(got, step()))


def test_refusals(torch_dev):
    torch, dev = torch_dev
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.zeros((64, 32), dtype=torch.bfloat16, device=dev)
    dy = torch.zeros((4, 32), dtype=torch.bfloat16, device=dev)
    v = torch.zeros(32, device=dev)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        mm.gated_linear(x.float(), w.float(), w.float())
    with pytest.raises(TypeError, match="w_up: expected"):
        mm.gated_linear(x, w, w.half())
    with pytest.raises(ValueError, match="w_up must have shape"):
        mm.gated_linear(x, w, w[:, :30])
    with pytest.raises(ValueError, match="stored alike"):
        mm.gated_linear(x, w, w.t().contiguous().t())
    with pytest.raises(ValueError, match="inner dimensions"):
        mm.gated_linear(x, w[:60], w[:60])
    with pytest.raises(ValueError, match="unknown activation 'tanh'"):
        mm.gated_linear(x, w, w, activation="tanh")
    with pytest.raises(ValueError, match="keep is"):
        mm.gated_linear(x, w, w, keep="z")
    with pytest.raises(TypeError, match="one type"):
        mm.gated_linear(x, w, w, v, v.bfloat16())
    with pytest.raises(ValueError, match="bias_up must have shape"):
        mm.gated_linear(x, w, w, None, v[:31])
    with pytest.raises(TypeError, match="out_dtype"):
        mm.gated_linear(x, w, w, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="pair"):
        mm.gated_linear_backward(dy, x, w, w, None)
    with pytest.raises(TypeError, match="pair"):
        mm.gated_linear_backward(dy, x, w, w, mm.checkpoint(dy))
    with pytest.raises(TypeError, match="two matrices or two"):
        mm.gated_linear_backward(dy, x, w, w, (dy, mm.checkpoint(dy)))
    with pytest.raises(ValueError, match="columns"):
        mm.gated_linear_backward(dy[:, :31], x, w, w, (dy, dy))
    with pytest.raises(ValueError, match="shape"):
        mm.gated_linear_backward(dy, x[:3], w, w, (dy, dy))
    with pytest.raises(TypeError, match="dw_dtype"):
        mm.gated_linear_backward(dy, x, w, w, (dy, dy), dw_dtype=torch.float16)
