"""Layer norm, its backward pass and the 8-bit checkpoints on the GPU,
against float64 formulas (tests/ops_reference.py)."""
import pytest

import bit_exact_matrix_amd as mm
import ops_reference as ref
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = 1e-5
DT = ["fp16", "bf16", "fp32"]


def types(torch):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def rows_of(torch, dev, rows, cols, dtype, seed, pad=0, offset=0):
    """rows x cols of N(0, 1) with an offset and an outlying column, as the
    middle columns of a wider matrix of NaN (pad on either side)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    wide = torch.full((rows, cols + 2 * pad), float("nan"), dtype=dtype, device=dev)
    x = torch.randn((rows, cols), generator=g, device=dev) + offset
    x[:, cols // 2:cols // 2 + 1] *= 20
    view = wide[:, pad:pad + cols]
    view.copy_(x)
    return view


# one column; parts of a vector; the last of one vector plan and the first of
# the next; rows beyond registers
SHAPES = [(1, 1), (3, 7), (5, 33), (64, 512), (9, 513), (300, 1000), (2, 2049), (257, 4096),
          (3, 8200), (2, 16385), (2, 32769), (1, 70001)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", DT)
def test_layer_norm(torch_dev, dt, shape):
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    rows, cols = shape
    x = rows_of(torch, dev, rows, cols, dtype, rows + cols, pad=cols % 3, offset=1.5)
    g = torch.Generator(device=dev).manual_seed(1)
    wt = dtype if cols % 2 else torch.float32
    w = torch.randn(cols, generator=g, device=dev).to(wt)
    b = torch.randn(cols, generator=g, device=dev).to(wt)
    say("layer norm", dt, shape)
    y, mean, rstd, saved = mm.layer_norm(x, w, b, EPS, checkpoint=True)
    want, wm, wr, ey, em, er = ref.layer_norm(x, w, b, EPS)
    ref.close(mean, wm, em, "mean")
    ref.close(rstd, wr, er * wr, "rstd")
    ref.close(y, want, ey, "y")
    codes, scales, _ = ref.checkpoint(x.double(), dtype)
    assert torch.equal(saved.scales, scales)
    assert torch.equal(saved.codes.double(), codes)
    y2, _, _, none = mm.layer_norm(x, w, b, EPS)
    assert none is None and torch.equal(y2, y)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt,saved", [("fp16", False), ("fp16", True), ("bf16", False),
                                      ("bf16", True), ("fp32", False), ("fp32", True)])
def test_layer_norm_backward(torch_dev, dt, saved, shape):
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    rows, cols = shape
    x = rows_of(torch, dev, rows, cols, dtype, 3 * rows + cols, pad=cols % 2, offset=-0.5)
    dy = rows_of(torch, dev, rows, cols, dtype, 5 * rows + cols, pad=1 - cols % 2)
    w = torch.randn(cols, generator=torch.Generator(device=dev).manual_seed(2), device=dev)
    w = w.to(dtype) if rows % 2 else w
    _, mean, rstd, ck = mm.layer_norm(x, w, None, EPS, checkpoint=True)
    say("layer norm backward", dt, saved, shape)
    dx, dw, db = mm.layer_norm_backward(dy, ck if saved else x, w, mean, rstd)
    xr = ref.checkpoint(x.double(), dtype)[2] if saved else x.double()
    wx, ww, wb, ex, ew, eb = ref.layer_norm_backward(dy, xr, w, mean, rstd)
    ref.close(dx, wx, ex, "dx")
    ref.close(dw, ww, ew, "dweight")
    ref.close(db, wb, eb, "dbias")
    # parts on their own, and dx over dy through the C entry
    only, n1, n2 = mm.layer_norm_backward(dy, ck if saved else x, w, mean, rstd,
                                          need_dparams=False)
    assert torch.equal(only, dx) and n1 is None and n2 is None
    n0, dw2, db2 = mm.layer_norm_backward(dy, ck if saved else x, w, mean, rstd, need_dx=False)
    assert n0 is None and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("cols", [640, 40000])
def test_layer_norm_backward_in_place(torch_dev, cols):
    """dX == dY: also where the row is read in several passes."""
    from bit_exact_matrix_amd import ops
    torch, dev = torch_dev
    rows = 37
    x = rows_of(torch, dev, rows, cols, torch.bfloat16, 1)
    dy = rows_of(torch, dev, rows, cols, torch.bfloat16, 2)
    w = torch.randn(cols, device=dev).bfloat16()
    _, mean, rstd, _ = mm.layer_norm(x, w)
    dx, dw, db = mm.layer_norm_backward(dy, x, w, mean, rstd)
    n = ops.mma_layer_norm_backward_workspace(rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    say("layer norm backward in place", cols)
    rc = ops.mma_layer_norm_backward(
        1, 1, dy.data_ptr(), cols, x.data_ptr(), cols, None, None, w.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), cols, dw2.data_ptr(), db2.data_ptr(),
        rows, cols, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(dy, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_layer_norm_gradient_against_differences(torch_dev):
    """<dx, v>, <dw, v>, <db, v> against central differences of the float64
    formula of sum(c y).  With step h the difference is off by at most
    h^2/6 times the third derivative along v (below 1e3 at these sizes:
    rstd is about 1 and v of unit length) and by 1e-16 |L| / h; the
    gradient by its float32 roundings."""
    torch, dev = torch_dev
    rows, cols, h = 5, 48, 1e-4
    g = torch.Generator(device=dev).manual_seed(7)
    x, c, vx = (torch.randn((rows, cols), generator=g, device=dev) for _ in range(3))
    w, b, vw = (torch.randn(cols, generator=g, device=dev) for _ in range(3))
    vx, vw = vx / vx.norm(), vw / vw.norm()
    _, mean, rstd, _ = mm.layer_norm(x, w, b, EPS)
    dx, dw, db = mm.layer_norm_backward(c, x, w, mean, rstd)

    def loss(x, w, b):
        return float((c.double() * ref.layer_norm(x, w, b, EPS)[0]).sum())

    size = float(c.norm()) * float(ref.layer_norm(x, w, b, EPS)[0].norm())
    room = h * h / 6 * 1e3 + 1e-16 * size / h + 256 * ref.U * size
    xd, wd, bd, vxd, vwd = (t.double() for t in (x, w, b, vx, vw))
    for got, hi, lo in ((float((dx * vx).sum()), loss(xd + h * vxd, wd, bd),
                         loss(xd - h * vxd, wd, bd)),
                        (float((dw * vw).sum()), loss(xd, wd + h * vwd, bd),
                         loss(xd, wd - h * vwd, bd)),
                        (float((db * vw).sum()), loss(xd, wd, bd + h * vwd),
                         loss(xd, wd, bd - h * vwd))):
        assert abs(got - (hi - lo) / (2 * h)) <= room


def test_rows_without_spread_and_with_special_values(torch_dev):
    """A constant row has y = b; a row with a NaN or an infinity is NaN and
    leaves the other rows alone; a large offset keeps its spread."""
    torch, dev = torch_dev
    cols = 96
    x = rows_of(torch, dev, 6, cols, torch.float32, 4)
    clean = x.clone()
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = clean[4] + 1e4
    w, b = torch.randn(cols, device=dev), torch.randn(cols, device=dev)
    say("layer norm special rows")
    y, mean, rstd, _ = mm.layer_norm(x, w, b, EPS)
    assert torch.equal(y[1], b)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    y0, _, _, _ = mm.layer_norm(clean, w, b, EPS)
    assert torch.equal(y[0], y0[0]) and torch.equal(y[5], y0[5])
    want, _, _, ey, _, _ = ref.layer_norm(x[4:5], w, b, EPS)
    ref.close(y[4:5], want, ey, "offset row")


def test_empty(torch_dev):
    torch, dev = torch_dev
    x = torch.empty((0, 40), device=dev)
    y, mean, rstd, ck = mm.layer_norm(x, checkpoint=True)
    assert y.shape == (0, 40) and mean.shape == (0,) and ck.scales.shape == (0, 2)
    dx, dw, db = mm.layer_norm_backward(x, x, torch.ones(40, device=dev), mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()
    assert mm.restore(mm.checkpoint(torch.empty((3, 0), device=dev))).shape == (3, 0)
    with pytest.raises(mm.MmaOpsError, match="no columns"):
        mm.layer_norm(torch.empty((3, 0), device=dev))


# ------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (70, 32), (7, 33), (33, 1499), (2, 5000)],
                         ids=str)
@pytest.mark.parametrize("dt", DT)
def test_checkpoint(torch_dev, dt, shape):
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    x = rows_of(torch, dev, *shape, dtype, sum(shape), pad=shape[1] % 4)
    # every row at a magnitude of its own, over the type's range
    top = 15 if dt == "fp16" else 126
    k = torch.linspace(-top - 10, top - 5, shape[0], device=dev).round()
    x.copy_((x.double() * torch.exp2(k.double())[:, None]).clamp(-6e4 if top == 15 else -3e38,
                                                                6e4 if top == 15 else 3e38))
    say("checkpoint", dt, shape)
    ck = mm.checkpoint(x)
    codes, scales, values = ref.checkpoint(x.double(), dtype)
    assert torch.equal(ck.scales, scales)
    assert torch.equal(ck.codes.double(), codes)
    back = mm.restore(ck)
    assert back.dtype == dtype and torch.equal(back.double(), values)


@pytest.mark.parametrize("dt", DT)
def test_checkpoint_every_pattern(torch_dev, dt):
    """Every 16-bit pattern (for float32: followed by a fixed lower half),
    NaN and infinities among them, in blocks of 32 that hold neighbouring
    magnitudes, and each alone in its block."""
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    bits = torch.arange(65536, dtype=torch.int32, device=dev)
    if dt == "fp32":
        v = (bits << 16 | 0x7FFF).view(torch.float32)
    else:
        v = bits.to(torch.int16).view(dtype)
    alone = torch.zeros((65536, 32), dtype=dtype, device=dev)
    alone[torch.arange(65536), torch.arange(65536) % 32] = v
    for x in (v.view(64, 1024), alone):
        say("checkpoint patterns", dt, tuple(x.shape))
        ck = mm.checkpoint(x)
        codes, scales, values = ref.checkpoint(x.double(), dtype)
        assert torch.equal(ck.scales, scales)
        got = ck.codes.double()
        assert torch.equal(torch.isnan(got), torch.isnan(codes))
        assert torch.equal(got.nan_to_num(0), codes.nan_to_num(0))
        number = torch.isfinite(codes)
        assert torch.equal(torch.signbit(got)[number], torch.signbit(codes)[number])
        assert (ck.codes.view(torch.uint8)[~number] == 0xFF).all()
        back = mm.restore(ck).double()
        fine = torch.isfinite(x.double())
        assert torch.equal(back[fine], values[fine]) and torch.isnan(back[~fine]).all()


def test_restore_to_another_type_and_code_types(torch_dev):
    torch, dev = torch_dev
    x = rows_of(torch, dev, 9, 70, torch.bfloat16, 1)
    ck = mm.checkpoint(x)
    full = mm.restore(ck, torch.float32)
    assert full.dtype == torch.float32 and torch.equal(full, mm.restore(ck).float())
    bytes_ = mm.Checkpoint(ck.codes.view(torch.uint8), ck.scales, ck.dtype)
    assert torch.equal(mm.restore(bytes_), mm.restore(ck))
    with pytest.raises(ValueError, match="shape"):
        mm.restore(mm.Checkpoint(ck.codes, ck.scales[:, :2].contiguous(), ck.dtype))
    with pytest.raises(TypeError, match="1-byte"):
        mm.restore(mm.Checkpoint(ck.codes.float(), ck.scales, ck.dtype))
    with pytest.raises(TypeError, match="checkpoint of"):
        mm.layer_norm_backward(x.half(), ck, None, torch.ones(9, device=dev),
                               torch.ones(9, device=dev))


def test_offsets_past_32_bits(torch_dev):
    """A matrix of 2.2e9 elements: the last rows' results are those of the
    same rows on their own."""
    torch, dev = torch_dev
    rows, cols, last = 65600, 32768 + 1024, 3
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    x[:2] = 1.0
    x[-last:] = rows_of(torch, dev, last, cols, torch.bfloat16, 5)
    w = torch.randn(cols, device=dev).bfloat16()
    say("layer norm past 32 bits")
    y, mean, rstd, ck = mm.layer_norm(x, w, None, checkpoint=True)
    tail = x[-last:].clone()
    ty, tm, tr, tk = mm.layer_norm(tail, w, None, checkpoint=True)
    assert torch.equal(y[-last:], ty) and torch.equal(mean[-last:], tm)
    assert torch.equal(ck.codes[-last:].view(torch.uint8), tk.codes.view(torch.uint8))
    assert torch.equal(ck.scales[-last:], tk.scales)
    assert torch.equal(mm.restore(ck)[-last:], mm.restore(tk))
    del y
    x[:-last] = 0
    dx, dw, _ = mm.layer_norm_backward(x, ck, w, torch.nan_to_num(mean), torch.ones_like(rstd))
    td, _, _ = mm.layer_norm_backward(tail, tk, w, tm, torch.ones_like(tr))
    assert torch.equal(dx[-last:], td) and not dx[:-last].any()


def test_same_bits_on_every_call_and_stream(torch_dev):
    torch, dev = torch_dev
    x = rows_of(torch, dev, 3000, 1536, torch.bfloat16, 1)
    dy = rows_of(torch, dev, 3000, 1536, torch.bfloat16, 2)
    w = torch.randn(1536, device=dev).bfloat16()
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    say("layer norm repeats")
    runs = []
    for s in (None, side, None):
        y, mean, rstd, ck = mm.layer_norm(x, w, w, checkpoint=True, stream=s)
        g = mm.layer_norm_backward(dy, ck, w, mean, rstd, stream=s)
        (s or torch.cuda.current_stream()).synchronize()
        runs.append([y, mean, rstd, ck.codes.view(torch.uint8), ck.scales, *g])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_refusals(torch_dev):
    torch, dev = torch_dev
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    with pytest.raises(TypeError, match="float16"):
        mm.layer_norm(x.double())
    with pytest.raises(ValueError, match="matrix"):
        mm.layer_norm(x[0])
    with pytest.raises(ValueError, match="adjacent"):
        mm.layer_norm(x.t())
    with pytest.raises(ValueError, match="overlap"):
        mm.checkpoint(x[0:1].expand(4, 64))
    with pytest.raises(ValueError, match="shape"):
        mm.layer_norm(x, w[:63])
    with pytest.raises(TypeError, match="one type"):
        mm.layer_norm(x, w, w.bfloat16())
    with pytest.raises(TypeError, match="weight"):
        mm.layer_norm(x, w.half())
    with pytest.raises(ValueError, match="shape"):
        mm.layer_norm_backward(x, x[:3], w, w[:4], w[:4])
    with pytest.raises(TypeError, match="device tensor"):
        mm.layer_norm(x, torch.ones(64))
