"""The product with its epilogue and its backward pass on the GPU, against
float64 formulas (tests/ops_reference.py), on every tile size, with split
inner sizes, and at the sizes and strides where they can go wrong."""
import pytest

import bit_exact_matrix_amd as mm
import ops_reference as ref
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
TILES = {"big": "0", "mid": "1", "small": "2", "few": "3", "rows": "4", "vec": "5"}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def matrix(torch, dev, rows, cols, dtype, seed, pad=0, scale=1.0):
    """rows x cols of N(0, scale) inside a wider, taller matrix of NaN."""
    g = torch.Generator(device=dev).manual_seed(seed)
    wide = torch.full((rows + 2, cols + 2 * pad), float("nan"), dtype=dtype, device=dev)
    view = wide[1:rows + 1, pad:pad + cols]
    view.copy_(torch.randn((rows, cols), generator=g, device=dev) * scale)
    return view


def operands(torch, dev, m, n, k, dtype, layout, seed, pad):
    x = matrix(torch, dev, m, k, dtype, seed, pad)
    if layout == "kn":
        w = matrix(torch, dev, k, n, dtype, seed + 1, pad, max(k, 1) ** -0.5)
    else:
        w = matrix(torch, dev, n, k, dtype, seed + 1, pad, max(k, 1) ** -0.5).t()
    return x, w


def check_linear(torch, dev, m, n, k, dtype, layout, act, pad, wide_out=False, seed=0):
    x, w = operands(torch, dev, m, n, k, dtype, layout, seed, pad)
    od = torch.float32 if wide_out else dtype
    bias = torch.randn(n, device=dev).to(torch.float32 if (m + n) % 2 else dtype)
    res = matrix(torch, dev, m, n, od, seed + 2, pad)
    say("linear", m, n, k, dtype, layout, act, pad)
    want, wz, ey, ez = ref.linear(x, w, bias, act, res)
    y, z = mm.linear(x, w, bias, activation=act, residual=res, keep="full", out_dtype=od)
    ref.close(y, want, ey, "y")
    ref.close(z, wz, ez, "z")
    y2, ck = mm.linear(x, w, bias, activation=act, residual=res, keep="checkpoint",
                       out_dtype=od)
    # z within its bound, then to 8 bits: a step of a code at most
    s = torch.exp2(ck.scales.double() - 127).repeat_interleave(32, 1)[:, :n]
    values = ck.codes.double() * s
    step = torch.maximum(wz.abs() / 16, s * 2.0 ** -10)
    assert ((values - wz).abs() <= step * (1 + 2.0 ** -3) + 2 * ez).all(), "checkpoint of z"
    assert torch.equal(mm.restore(ck).double(), values)
    ref.close(y2, want, ey, "y beside a checkpoint")
    y3, none = mm.linear(x, w)
    want, _, ey, _ = ref.linear(x, w, None, "none", None)
    ref.close(y3, want, ey, "plain product")
    assert none is None


SHAPES = [(1, 1, 1), (1, 64, 128), (2, 40, 4200), (2, 8200, 9), (1, 4099, 37), (5, 136, 1088),
          (16, 50, 7), (17, 33, 130), (64, 64, 64), (65, 129, 191), (130, 72, 8), (300, 260, 640),
          (256, 512, 72), (257, 264, 320)]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_linear(torch_dev, monkeypatch, tile, layout, pad):
    """Every tile size on every shape, without and with split inner sizes."""
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
def test_linear_as_chosen(torch_dev, dt, act):
    """The library's own choice of tile and splits."""
    torch, dev = torch_dev
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    for i, (m, n, k) in enumerate([(1, 1024, 1024), (4, 1000, 4096), (33, 96, 2048),
                                   (520, 1040, 96), (1024, 1024, 256), (1100, 1300, 65)]):
        check_linear(torch, dev, m, n, k, dtype, "kn" if i % 2 else "nk", act, 0, seed=i)


def check_backward(torch, dev, m, n, k, dtype, layout, act, pad, saved, wide=False, seed=0):
    x, w = operands(torch, dev, m, n, k, dtype, layout, seed, pad)
    dy = matrix(torch, dev, m, n, dtype, seed + 3, pad)
    z = matrix(torch, dev, m, n, dtype, seed + 4, pad, 1.5)
    xr, zr, xa, za = x.double(), z.double(), x, z
    if saved:
        xa, za = mm.checkpoint(x), mm.checkpoint(z)
        xr, zr = ref.checkpoint(xr, dtype)[2], ref.checkpoint(zr, dtype)[2]
    od = torch.float32 if wide else dtype
    say("linear backward", m, n, k, dtype, layout, act, pad, saved)
    dx, dw, db = mm.linear_backward(dy, xa, w, za if act != "none" else None, activation=act,
                                    dw_dtype=od, bias_dtype=od)
    wx, ww, wb, ex, ew, eb = ref.linear_backward(dy, xr, w, zr, act, dtype)
    ref.close(dx, wx, ex, "dx")
    ref.close(dw, ww, ew, "dw")
    ref.close(db, wb, eb, "dbias")
    assert dw.stride() == ((1, k) if layout == "nk" and k > 0 else (n, 1))
    for i, got in enumerate((dx, dw, db)):
        need = [j == i for j in range(3)]
        part = mm.linear_backward(dy, xa, w, za if act != "none" else None, activation=act,
                                  need_dx=need[0], need_dw=need[1], need_dbias=need[2],
                                  dw_dtype=od, bias_dtype=od)
        assert sum(t is not None for t in part) == 1
        if i < 2:
            assert torch.equal(part[i], got)
        else:
            ref.close(part[i], wb, eb, "dbias alone")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("saved", [False, True])
def test_linear_backward(torch_dev, monkeypatch, tile, layout, saved):
    torch, dev = torch_dev
    monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES[tile])
    for i, (m, n, k) in enumerate(SHAPES):
        dtype = torch.float16 if (i + saved) % 2 else torch.bfloat16
        if i % 3 == 2:
            monkeypatch.setenv("MMAOPS_LINEAR_SPLITS", str(2 + i % 3))
        else:
            monkeypatch.delenv("MMAOPS_LINEAR_SPLITS", raising=False)
        check_backward(torch, dev, m, n, k, dtype, layout, ACTS[i % 5], (0, 3, 8)[i % 3], saved,
                       wide=i % 4 == 1, seed=20 * i)


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_as_chosen(torch_dev, act):
    torch, dev = torch_dev
    for i, (m, n, k) in enumerate([(1, 1024, 1000), (300, 1024, 512), (2100, 520, 264)]):
        check_backward(torch, dev, m, n, k, torch.bfloat16 if i % 2 else torch.float16,
                       "nk" if i % 2 else "kn", act, 0, i != 1, seed=i)


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_backward_products_in_one_launch(torch_dev, monkeypatch, layout):
    """Small tiles, whole: dX, dW and the bias sums share a launch, and the
    products' bits are those of each asked for alone."""
    torch, dev = torch_dev
    monkeypatch.setenv("MMAOPS_LINEAR_TILE", TILES["small"])
    monkeypatch.setenv("MMAOPS_LINEAR_SPLITS", "1")
    for i, (m, n, k) in enumerate([(17, 24, 40), (299, 261, 643), (64, 640, 8), (1000, 65, 129)]):
        for act in ("none", ACTS[1 + i]):
            check_backward(torch, dev, m, n, k, torch.float16 if i % 2 else torch.bfloat16,
                           layout, act, (0, 3)[i % 2], i == 3, wide=i == 0, seed=i)


def test_gradient_against_differences(torch_dev):
    """<gradient, v> against central differences of the float64 formula of
    sum(c y): the difference is off by h^2/6 of a third derivative (below
    1e2 here, v of unit length) and 1e-16 |L| / h, the gradient by the
    roundings of dz and of the outputs: 2^-11 of sum |terms| each."""
    torch, dev = torch_dev
    m, n, k, h = 7, 40, 24, 1e-4
    g = torch.Generator(device=dev).manual_seed(3)

    def r(*shape):
        t = torch.randn(shape, generator=g, device=dev).half()
        return t

    x, w, b, c = r(m, k), r(k, n) * 0.2, r(n), r(m, n)
    for act in ACTS:
        y, z = mm.linear(x, w, b, activation=act, keep="full", out_dtype=torch.float32)
        grads = mm.linear_backward(c, x, w, z, activation=act)
        point = [t.double() for t in (x, w, b)]
        # z is kept in 16 bits: the slope (1.2 at most steep) moves with it
        moved = 1.2 * 2.0 ** -11 * z.double().abs() * c.double().abs()
        for i in range(3):
            v = torch.randn(point[i].shape, generator=g, device=dev).double()
            v = v / v.norm()

            def loss(t):
                p = list(point)
                p[i] = p[i] + t * v
                return float((c.double() * ref.act(p[0] @ p[1] + p[2], act)).sum())

            got = float((grads[i].double() * v).sum())
            terms = float(([moved @ w.double().abs().t(), x.double().abs().t() @ moved,
                            moved.sum(0)][i] * v.abs()).sum())
            dz = c.double().abs() * 1.2
            size = [dz @ w.double().abs().t(), x.double().abs().t() @ dz, dz.sum(0)][i]
            room = (h * h / 6 * 1e2 + 1e-16 * abs(loss(0)) / h + terms
                    + 3 * 2.0 ** -11 * float((size * v.abs()).sum()))
            if act == "relu":
                # a z within a step of the kink: at most its whole slope
                near = (z.double().abs() < 1e-3).double() * c.double().abs()
                room += float(([near @ w.double().abs().t(), x.double().abs().t() @ near,
                                near.sum(0)][i] * v.abs()).sum())
            assert abs(got - (loss(h) - loss(-h)) / (2 * h)) <= room, (act, i)


def test_empty_sizes(torch_dev):
    torch, dev = torch_dev
    bf = torch.bfloat16
    e = lambda *s: torch.empty(s, dtype=bf, device=dev)  # noqa: E731
    bias = torch.randn(5, device=dev)
    y, ck = mm.linear(e(3, 0), e(0, 5), bias, activation="relu", keep="checkpoint")
    assert torch.equal(y, torch.relu(bias).to(bf).expand(3, 5))
    for m, n in ((0, 5), (3, 0)):
        y, _ = mm.linear(e(m, 4), e(4, n))
        assert y.shape == (m, n)
    dx, dw, db = mm.linear_backward(e(0, 5), e(0, 4), e(4, 5))
    assert dx.shape == (0, 4) and not dw.any() and not db.any() and dw.shape == (4, 5)
    dx, dw, db = mm.linear_backward(e(3, 0), e(3, 4), e(4, 0))
    assert not dx.any() and dx.shape == (3, 4) and dw.shape == (4, 0) and db.shape == (0,)
    dy = torch.ones((3, 5), dtype=bf, device=dev)
    dx, dw, db = mm.linear_backward(dy, e(3, 0), e(0, 5))
    assert dx.shape == (3, 0) and dw.shape == (0, 5) and (db == 3).all()


def test_special_values_stay_in_their_rows(torch_dev):
    """A NaN or an infinity in a row of X reaches that row of Y only; one in
    a column of W that column only; large products become infinities of
    the output type; nothing is flushed among the small ones."""
    torch, dev = torch_dev
    for m, n, k in ((5, 70, 200), (200, 150, 100)):
        x, w = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 1, 0)
        y0, _ = mm.linear(x, w, activation="gelu")
        x2 = x.clone()
        x2[2, 3] = float("inf")
        x2[4, 0] = float("nan")
        say("linear special values", m, n, k)
        y, _ = mm.linear(x2, w, activation="gelu")
        rest = [i for i in range(m) if i not in (2, 4)]
        assert torch.equal(y[rest], y0[rest])
        assert torch.isnan(y[4]).all() and not torch.isfinite(y[2].float()).all()
        w2 = w.clone()
        w2[1, 7] = float("nan")
        y, _ = mm.linear(x, w2, activation="gelu")
        cols = [j for j in range(n) if j != 7]
        assert torch.equal(y[:, cols], y0[:, cols]) and torch.isnan(y[:, 7]).all()
    big = torch.full((3, 64), 3e4, dtype=torch.float16, device=dev)
    y, ck = mm.linear(big, torch.ones((64, 40), dtype=torch.float16, device=dev),
                      keep="checkpoint")
    assert torch.isinf(y).all()
    assert torch.equal(mm.restore(ck), torch.full_like(y, 61440.0))


def test_backward_far_from_the_origin(torch_dev):
    """Slopes at pre-activations beyond the functions' bends: 0 or 1."""
    torch, dev = torch_dev
    z = torch.tensor([[-1e30, -300.0, -30.0, 30.0, 300.0, 1e30]], device=dev).bfloat16()
    want = torch.tensor([0.0, 0, 0, 1, 1, 1], device=dev)
    dy, x = torch.ones_like(z), torch.ones((1, 1), dtype=torch.bfloat16, device=dev)
    for act in ACTS[1:]:
        _, _, db = mm.linear_backward(dy, x, torch.ones_like(z), z, activation=act,
                                      bias_dtype=torch.float32)
        assert torch.allclose(db, want, rtol=0, atol=1e-10), act


def test_offsets_past_32_bits(torch_dev):
    """Outputs past 2^31 elements, and an operand past 2^32 bytes: the last
    rows are those of the same rows on their own."""
    torch, dev = torch_dev
    m, n, k, last = 530000, 4104, 64, 200
    x = matrix(torch, dev, m, k, torch.bfloat16, 1)
    w = matrix(torch, dev, k, n, torch.bfloat16, 2, scale=0.1)
    say("linear past 32 bits")
    y, ck = mm.linear(x, w, keep="checkpoint")
    ty, tk = mm.linear(x[-last:], w, keep="checkpoint")
    for a, b in ((y[-last:], ty), (ck.codes[-last:].view(torch.uint8),
                                   tk.codes.view(torch.uint8)), (ck.scales[-last:], tk.scales)):
        assert torch.equal(a, b)
    # y as the operand: M and the inner size of dW past the same bound
    y[:-last] = 0
    dx, dw, db = mm.linear_backward(y, x, w)
    tx, tw, tb = mm.linear_backward(ty, x[-last:], w)
    assert torch.equal(dx[-last:], tx) and not dx[:-last].any()
    ey = ref.linear_backward(ty, x[-last:].double(), w, None, "none", torch.bfloat16)
    ref.close(dw, ey[1], ey[4], "dw")
    ref.close(db, ey[2], ey[5], "dbias")


def test_same_bits_on_every_call_and_stream(torch_dev):
    torch, dev = torch_dev
    side = torch.cuda.Stream(device=dev)
    for m, n, k in ((2, 2048, 4096), (700, 900, 1100), (1024, 2048, 512)):
        x, w = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 5, 0)
        dy = matrix(torch, dev, m, n, torch.bfloat16, 6)
        side.wait_stream(torch.cuda.current_stream())
        say("linear repeats", m, n, k)
        runs = []
        for s in (None, side, None):
            y, ck = mm.linear(x, w, activation="silu", keep="checkpoint", stream=s)
            g = mm.linear_backward(dy, x, w, ck, activation="silu", stream=s)
            (s or torch.cuda.current_stream()).synchronize()
            runs.append([y, ck.codes.view(torch.uint8), ck.scales, *g])
        for other in runs[1:]:
            for a, b in zip(runs[0], other):
                assert torch.equal(a, b)


def test_captured_in_a_graph(torch_dev):
    """A forward and backward pass captured once and replayed on new inputs,
    each replay against the eager calls."""
    torch, dev = torch_dev
    m, n, k = 96, 320, 512
    x, w = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 1, 0)
    dy = matrix(torch, dev, m, n, torch.bfloat16, 2)
    nw = torch.ones(k, dtype=torch.bfloat16, device=dev)

    def step():
        h, mean, rstd, ck = mm.layer_norm(x, nw, checkpoint=True)
        y, z = mm.linear(h, w, activation="gelu", keep="checkpoint")
        dh, dw, db = mm.linear_backward(dy, h, w, z, activation="gelu")
        dx, dnw, dnb = mm.layer_norm_backward(dh, ck, nw, mean, rstd)
        return [y, dw, db, dx, dnw, dnb]

    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(matrix(torch, dev, m, k, torch.bfloat16, 100 + i))
        say("graph replay", i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_refusals(torch_dev):
    torch, dev = torch_dev
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.zeros((64, 32), dtype=torch.bfloat16, device=dev)
    dy = torch.zeros((4, 32), dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        mm.linear(x.float(), w.float())
    with pytest.raises(TypeError, match="w: expected"):
        mm.linear(x, w.half())
    with pytest.raises(ValueError, match="inner dimensions"):
        mm.linear(x, w[:60])
    with pytest.raises(ValueError, match="unknown activation 'tanh'"):
        mm.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="keep is"):
        mm.linear(x, w, keep="z")
    with pytest.raises(TypeError, match="residual"):
        mm.linear(x, w, residual=dy.float())
    with pytest.raises(ValueError, match="bias must have shape"):
        mm.linear(x, w, torch.zeros(31, device=dev))
    with pytest.raises(TypeError, match="out_dtype"):
        mm.linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="needs z"):
        mm.linear_backward(dy, x, w, activation="gelu")
    with pytest.raises(ValueError, match="differ"):
        mm.linear_backward(dy[:, :31], x, w)
    with pytest.raises(ValueError, match="shape"):
        mm.linear_backward(dy, x[:3], w)
    with pytest.raises(TypeError, match="dw_dtype"):
        mm.linear_backward(dy, x, w, dw_dtype=torch.float16)
