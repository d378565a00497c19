"""Corners of the gated block's operators: what a call leaves out, elements past
a row's end beside large gradients, kept values near the largest float,
weights of one row or column, inputs and outputs on their own."""
import itertools
import math

import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
import ops_reference
from bit_exact_matrix_amd import block, ops
from test_gpu_gated_linear import NAMES, operands
from test_gpu_ops_linear import matrix
from test_gpu_parity import say, torch_dev  # noqa: F401
from test_gpu_residual_norm import vectors

pytestmark = pytest.mark.gpu


# ------------------------------------------- what a call leaves out (C entry points)
JOIN = ("dtype param_dtype post pre scale eps p seed offset state rows cols X ldx branch ldb gate "
        "post_weight post_bias pre_weight pre_bias R ldr H ldh post_mean post_rstd mean rstd").split()
JOIN_BACKWARD = (
    "dtype param_dtype post pre scale reserved p seed offset state rows cols dR lddr dH lddh R ldr "
    "branch ldb gate post_weight post_bias pre_weight post_mean post_rstd mean rstd dX lddx dbranch "
    "lddb dgate dpost_weight dpost_bias dpre_weight dpre_bias").split()


def raw(torch, names, packed, call, values, *more):
    """A call of the C entry point; tensors are given as their pointers, the rest is 0."""
    v = [values.get(n, 0) for n in names]
    args = packed.pack(*(t.data_ptr() if isinstance(t, torch.Tensor) else t for t in v))
    return call(args, *more, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("cols", [72, 640, 4096, 8256, 16392])
def test_vectors_of_a_norm_that_is_not_there_are_not_read(torch_dev, cols):
    """They hold NaN, or are the memory of an output."""
    torch, dev = torch_dev
    rows, dt = 5, torch.bfloat16
    x, b, dr, dh = (matrix(torch, dev, rows, cols, dt, i) for i in range(4))
    nan = torch.full((cols,), math.nan, dtype=dt, device=dev)
    v = vectors(torch, dev, cols, dt, "rms", "rms", True, True)
    base = dict(dtype=ops.BF16, param_dtype=ops.BF16, scale=1.0, eps=1e-5, rows=rows, cols=cols,
                gate=v.gate)
    ld = {k: cols for k in ("ldx", "ldb", "ldr", "ldh", "lddr", "lddh", "lddx", "lddb")}
    for post, pre in itertools.product((None, "rms"), repeat=2):
        say("vectors without their norm", cols, post, pre)
        p = mm.ResidualParams(v.gate, v.post_weight if post else None, None,
                              v.pre_weight if pre else None, None)
        r, h, stats = mm.residual_norm(x, b, p, post=post, pre=pre)
        dx, db, grads = mm.residual_norm_backward(dr, dh if pre else None, r, b, p, stats,
                                                  post=post, pre=pre)
        R, H, dX, dB = (torch.empty_like(x) for _ in range(4))
        dgate = torch.empty_like(nan)
        kinds = dict(post=block.NORMS[post], pre=block.NORMS[pre])
        # the vectors: of a norm that is there its own, else NaN, and (for the biases) R's memory
        own = dict(post_weight=v.post_weight if post else nan, post_bias=0 if post else R,
                   pre_weight=v.pre_weight if pre else nan, pre_bias=0 if pre else R)
        rc = raw(torch, JOIN, block._JOIN, ops.mma_residual_norm,
                 {**base, **ld, **kinds, **own, "X": x, "branch": b, "R": R, "H": H})
        assert rc == 0 and torch.equal(R, r) and (h is None or torch.equal(H, h))
        # statistics of a norm that is not there, and an rms norm's mean: an output's memory
        s = {n: t if t is not None else dX for n, t in stats._asdict().items()}
        own.update(post_bias=0 if post else dB, **s)
        args = {**base, **ld, **kinds, **own, "dR": dr, "dH": dh if pre else dX,
                "R": r if pre else dB, "branch": b, "dX": dX, "dbranch": dB, "dgate": dgate}
        need = raw(torch, JOIN_BACKWARD, block._JOIN_BACKWARD,
                   lambda a, _: ops.mma_residual_norm_backward_workspace(a), args)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = raw(torch, JOIN_BACKWARD, block._JOIN_BACKWARD, ops.mma_residual_norm_backward, args,
                 ws.data_ptr(), need)
        assert rc == 0 and torch.equal(dX, dx) and torch.equal(dB, db)
        assert torch.equal(dgate, grads.gate)


# --------------------------------------------------------- past a row's end
@pytest.mark.parametrize("cols", [60, 100, 200])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("post", ["layer", "rms"])
def test_large_equal_gradients_of_equal_rows(torch_dev, cols, dtype, post):
    """dh is 2^120 and r is 1 throughout: the layer norm before the next block gives
    no gradient, exactly (cols 2^120 < 2^128 is a float, and so is their mean), but an
    element that is not there would be 2^120 below the mean, times an rstd of 316 no
    float.  What is left is the gradient of the norm behind the block, of dr alone:
    its sums have at most 200 terms in no more than 16 additions each, so with some ten
    roundings of the products the error is below 32 2^-24 of the largest term."""
    torch, dev = torch_dev
    dt = getattr(torch, dtype)
    for rows in (1, 5):
        say("large equal gradients", cols, dtype, post, rows)
        one = torch.ones((rows, cols), device=dev, dtype=dt)
        dr, dh = matrix(torch, dev, rows, cols, dt, 1), one * 2.0 ** 120
        v = one[0].clone()
        bias = v if post == "layer" else None
        p = mm.ResidualParams(None, v, bias, v, v)
        how = dict(post=post, pre="layer")
        # each norm's statistics of rows of ones
        zero = torch.zeros_like(one)
        stats = mm.ResidualStats(*mm.residual_norm(zero, one, p, **how)[2][:2],
                                 *mm.residual_norm(one, zero, mm.ResidualParams(),
                                                   pre="layer")[2][2:])
        dx, db, grads = mm.residual_norm_backward(dr, dh, one, one, p, stats, **how)
        assert torch.equal(dx, dr)
        d, k = dr.double(), stats.post_rstd.double()[:, None]
        bh = (one.double() - (1.0 if post == "layer" else 0.0)) * k
        want = k * (d - (d.mean(1, keepdim=True) if post == "layer" else 0.0)
                    - bh * (d * bh).mean(1, keepdim=True))
        ops_reference.close(db, want, 2.0 ** -19 * k * d.abs().amax(1, keepdim=True) * 2, "dbranch")
        assert not bool(grads.pre_weight.any())
        assert torch.equal(grads.pre_bias, rows * dh[0])
        s = (d * bh).sum(0)
        ops_reference.close(grads.post_weight, s, 2.0 ** -20 * (d * bh).abs().sum(0), "post_weight")


# ------------------------------------------- kept values near the largest float
def one_sided(torch, dev, value, gate, dy, dtype):
    """dy, g and u of 6 x 40: u is `value` in the first columns, g is `gate`."""
    g = torch.full((6, 40), gate, dtype=dtype, device=dev)
    u = torch.randn((6, 40), generator=torch.Generator(dev).manual_seed(3), device=dev).to(dtype)
    u[:, :5] = value
    return torch.full_like(g, dy), g, u


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_a_kept_infinity_beside_no_gradient(torch_dev, act):
    """Slopes above 1 (gates of about 2) times the largest float are no float; times a
    dy of 0 they are 0."""
    torch, dev = torch_dev
    x = matrix(torch, dev, 6, 16, torch.bfloat16, 1)
    w = matrix(torch, dev, 16, 40, torch.bfloat16, 2)
    for value, gate in itertools.product((math.inf, -math.inf), (1.4, 2.4)):
        dy, g, u = one_sided(torch, dev, value, gate, 0.0, torch.bfloat16)
        say("kept infinity, no gradient", act, value, gate)
        got = mm.gated_linear_backward(dy, x, w, w, (g, u), activation=act)
        assert not any(bool(t.any()) for t in got)
        # a large number, and a small gradient: still a number
        got = mm.gated_linear_backward(dy + 2.0 ** -100, x, w, w, (g, u), activation=act)
        assert all(bool(torch.isfinite(t).all()) for t in got)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_a_checkpoint_at_its_bound(torch_dev, act):
    """u is 1.875 * 2^127, the largest value that a bf16 checkpoint keeps."""
    torch, dev = torch_dev
    dt = torch.bfloat16
    x = matrix(torch, dev, 6, 16, dt, 1)
    w = matrix(torch, dev, 16, 40, dt, 2)
    for dy, gate in itertools.product((0.0, 2.0 ** -100), (1.4, 2.4)):
        dy, g, u = one_sided(torch, dev, 1.875 * 2.0 ** 127, gate, dy, dt)
        say("saturated checkpoint", act)
        kept = mm.checkpoint(g), mm.checkpoint(u)
        gr, ur = (mm.restore(c).double() for c in kept)
        assert float(ur.max()) == 1.875 * 2.0 ** 127
        got = mm.gated_linear_backward(dy, x, w, w, kept, activation=act,
                                       bias_dtype=torch.float32)
        values, bounds = ref.gated_linear_backward(dy, x.double(), w, w, gr, ur, act, dt)
        for name, t, v, e in zip(NAMES, got, values, bounds):
            ops_reference.close(t, v, e, name)


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_the_largest_numbers_kept_whole(torch_dev, act):
    """Finite values of g and u are taken as they are, up to bf16's largest."""
    torch, dev = torch_dev
    dt = torch.bfloat16
    x = matrix(torch, dev, 6, 16, dt, 1)
    w = matrix(torch, dev, 16, 40, dt, 2)
    for top in (torch.finfo(dt).max, -torch.finfo(dt).max):
        dy, g, u = one_sided(torch, dev, top, 1.0, 2.0 ** -100, dt)
        g[:, 20:25] = abs(top)
        say("largest numbers", act, top)
        got = mm.gated_linear_backward(dy, x, w, w, (g, u), activation=act,
                                       bias_dtype=torch.float32)
        values, bounds = ref.gated_linear_backward(dy, x.double(), w, w, g.double(), u.double(),
                                                   act, dt)
        for name, t, v, e in zip(NAMES, got, values, bounds):
            ops_reference.close(t, v, e, name)


# ------------------------------------------------- weights of one row or column
@pytest.mark.parametrize("k,n", [(1, 24), (40, 1), (1, 1)])
def test_weights_of_one_row_or_column(torch_dev, k, n):
    """They are rows and columns at once: any two are stored alike."""
    torch, dev = torch_dev
    dt = torch.bfloat16
    x, dy = matrix(torch, dev, 9, k, dt, 1), matrix(torch, dev, 9, n, dt, 2)

    def ways(seed):
        w = matrix(torch, dev, k, n, dt, seed)
        wide = torch.full((k, n + 7), math.nan, dtype=dt, device=dev)
        wide[:, :n] = w
        tall = torch.full((n, k + 7), math.nan, dtype=dt, device=dev)
        tall[:, :k] = w.t()
        return [w, wide[:, :n], w.t().contiguous().t(), tall[:, :k].t()]

    for a, b in itertools.product(ways(3), ways(4)):
        say("one row or column", k, n, a.stride(), b.stride())
        y, kept = mm.gated_linear(x, a, b, keep="full")
        want, _, _, ey, _, _ = ref.gated_linear(x, a, b, None, None, "silu")
        ops_reference.close(y, want, ey, "y")
        values, bounds = ref.gated_linear_backward(dy, x.double(), a, b, kept[0].double(),
                                                   kept[1].double(), "silu", dt)
        for name, t, v, e in zip(NAMES, mm.gated_linear_backward(dy, x, a, b, kept), values,
                                 bounds):
            ops_reference.close(t, v, e, name)


# ------------------------------------------------ outputs and inputs on their own
@pytest.mark.parametrize("dtype,cols", [("bfloat16", 640), ("bfloat16", 1024), ("bfloat16", 4096),
                                        ("float32", 1000), ("float32", 1024), ("float32", 5120),
                                        ("bfloat16", 8256)])
@pytest.mark.parametrize("post,pre", [("rms", "layer"), (None, "rms")])
def test_without_the_gradient_of_the_sum(torch_dev, dtype, cols, post, pre):
    """dr=None, behind the last block: what dr=0 gives, and the formula."""
    torch, dev = torch_dev
    dt = getattr(torch, dtype)
    rows = 37
    x, b, dh = (matrix(torch, dev, rows, cols, dt, i) for i in range(3))
    v = vectors(torch, dev, cols, dt, post, pre, True, pre == "layer")
    how = dict(post=post, pre=pre, scale=0.7, dropout=0.25, seed=11, offset=12)
    say("no gradient of the sum", dtype, cols, post, pre)
    r, _, stats = mm.residual_norm(x, b, v, **how)
    got = mm.residual_norm_backward(None, dh, r, b, v, stats, **how)
    zero = mm.residual_norm_backward(torch.zeros_like(dh), dh, r, b, v, stats, **how)
    for s, t in zip((*got[:2], *got[2]), (*zero[:2], *zero[2])):
        assert (s is None) == (t is None) and (s is None or torch.equal(s, t))
    m = ref.mask(rows, cols, 0.25, 11, 12, dev)
    val, off = ref.residual_norm_backward(None, dh, r, b, v, stats, post, pre, 0.7, m)
    for k, t in {"dx": got[0], "dbranch": got[1], **got[2]._asdict()}.items():
        if t is not None:
            ops_reference.close(t, val[k], off[k], k)


@pytest.mark.parametrize("dtype,cols", [("bfloat16", 5120), ("bfloat16", 8192), ("float32", 1000),
                                        ("float32", 5120), ("float32", 8200)])
def test_gradients_without_those_of_the_vectors(torch_dev, dtype, cols):
    """dx and dbranch have the same bits on their own, rows of 9 to 16 waves and the
    gradients of biases among what is left out."""
    torch, dev = torch_dev
    dt = getattr(torch, dtype)
    x, b, dr, dh = (matrix(torch, dev, 600, cols, dt, i) for i in range(4))
    v = vectors(torch, dev, cols, dt, "layer", "layer", True, True)
    how = dict(post="layer", pre="layer")
    say("gradients without the vectors'", dtype, cols)
    r, _, stats = mm.residual_norm(x, b, v, **how)
    dx, db, _ = mm.residual_norm_backward(dr, dh, r, b, v, stats, **how)
    for need in itertools.product((False, True), repeat=2):
        got = mm.residual_norm_backward(dr, dh, r, b, v, stats, need_dx=need[0],
                                        need_dbranch=need[1], need_dparams=False, **how)
        assert got[0] is None or torch.equal(got[0], dx)
        assert got[1] is None or torch.equal(got[1], db)


@pytest.mark.parametrize("m,n,k", [(1, 1024, 1024), (64, 48, 40), (299, 260, 640), (520, 1040, 96),
                                   (1100, 1300, 65), (2048, 512, 512)])
@pytest.mark.parametrize("saved", [False, True])
def test_bias_gradients_on_their_own(torch_dev, m, n, k, saved):
    """The same bits from the small pass's second launch and from a kernel of their own."""
    torch, dev = torch_dev
    x, wg, wu = operands(torch, dev, m, n, k, torch.bfloat16, "kn", 1, 0)
    dy, g, u = (matrix(torch, dev, m, n, torch.bfloat16, i) for i in (3, 4, 5))
    kept = (mm.checkpoint(g), mm.checkpoint(u)) if saved else (g, u)
    say("bias gradients on their own", m, n, k, saved)
    want = mm.gated_linear_backward(dy, x, wg, wu, kept, bias_dtype=torch.float32)[3:]
    for need in itertools.product((False, True), repeat=2):
        got = mm.gated_linear_backward(dy, x, wg, wu, kept, need_dx=need[0], need_dw=need[1],
                                       bias_dtype=torch.float32)[3:]
        assert all(torch.equal(s, t) for s, t in zip(got, want)), need
