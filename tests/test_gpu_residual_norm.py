"""The sum into the residual stream with its norms, its gate and its dropout,
forward and backward, against float64 formulas (tests/block_reference.py)."""
import itertools
import math

import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
import ops_reference
from test_gpu_ops_linear import matrix
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
DT = ["fp16", "bf16", "fp32"]
EPS = 1e-5
SEED, OFFSET = 0x123456789ABCDEF, 77


def types(torch):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def vectors(torch, dev, cols, dtype, post, pre, gate, bias, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed + 50)

    def v(mean, there):
        t = mean + 0.3 * torch.randn(cols, generator=g, device=dev)
        return t.to(dtype) if there else None

    return mm.ResidualParams(v(0.6, gate), v(1.0, post), v(0.1, post and bias), v(1.0, pre),
                             v(0.1, pre and bias))


def check(torch, dev, rows, cols, dtype, vt, post, pre, gate, bias, p, scale, pad, seed=0,
          offset_rows=0.0):
    x = matrix(torch, dev, rows, cols, dtype, seed + 1, pad)
    b = matrix(torch, dev, rows, cols, dtype, seed + 2, pad)
    x += offset_rows
    v = vectors(torch, dev, cols, vt, post, pre, gate, bias, seed)
    how = dict(post=post, pre=pre, scale=scale, dropout=p, seed=SEED, offset=OFFSET)
    m = ref.mask(rows, cols, p, SEED, OFFSET, dev) if p else None
    say("residual norm", rows, cols, dtype, vt, post, pre, gate, bias, p, scale, pad)
    r, h, stats = mm.residual_norm(x, b, v, eps=EPS, **how)
    val, off = ref.residual_norm(x, b, v, post, pre, scale, EPS, m)
    got = {"r": r, "h": h, **stats._asdict()}
    assert {k for k, t in got.items() if t is not None} == {
        k for k in val if not ((post == "rms" and k == "post_mean")
                               or (pre == "rms" and k == "mean"))}
    for k, t in got.items():
        if t is not None:
            ops_reference.close(t, val[k], off[k], k)
    dr, dh = (matrix(torch, dev, rows, cols, dtype, seed + i, pad) for i in (3, 4))
    val, off = ref.residual_norm_backward(dr, dh, r, b, v, stats, post, pre, scale, m)
    dx, db, grads = mm.residual_norm_backward(dr, dh if pre else None, r, b, v, stats, **how)
    got = {"dx": dx, "dbranch": db, **grads._asdict()}
    for k, t in got.items():
        if t is not None:
            ops_reference.close(t, val[k], off[k], k)
    assert [t is None for t in grads] == [t is None for t in v]
    return x, b, v, how, r, h, stats, dr, dh, got


SHAPES = [(1, 1), (3, 7), (2, 64), (70, 33), (5, 513), (37, 1000), (9, 4096), (4, 4104), (3, 8200),
          (2, 16384), (2, 20001), (300, 96), (1100, 260), (1030, 640), (6, 1536), (5, 2560),
          (3, 5120), (3, 8192), (2, 10240)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(torch_dev, dt, shape):
    torch, dev = torch_dev
    dtype = types(torch)[dt]
    for i, (post, pre) in enumerate([("rms", "rms"), ("layer", "layer"), (None, "rms")]):
        check(torch, dev, *shape, dtype, dtype if i % 2 else torch.float32, post, pre, i != 2,
              i == 1, 0.3 if i != 1 else 0.0, (1.0, 0.7, 1.0)[i], (0, 3, 8)[i], seed=i)


@pytest.mark.parametrize("post,pre", itertools.product([None, "layer", "rms"], repeat=2))
@pytest.mark.parametrize("gate", [False, True])
def test_every_form(torch_dev, post, pre, gate):
    torch, dev = torch_dev
    for i, (bias, p, cols) in enumerate([(False, 0.0, 520), (True, 0.25, 520), (True, 1.0, 100),
                                         (True, 0.25, 8256)]):
        dtype = (torch.bfloat16, torch.float32, torch.float16, torch.bfloat16)[i]
        check(torch, dev, 41, cols, dtype, dtype, post, pre, gate, bias, p, 1.0, 0, seed=i)


def test_rows_far_from_zero(torch_dev):
    """A residual stream whose offset is large beside its spread: a layer
    norm's mean is corrected."""
    torch, dev = torch_dev
    for cols in (300, 4096, 20001):
        check(torch, dev, 3, cols, torch.float32, torch.float32, "layer", "layer", True, True,
              0.0, 1.0, 0, offset_rows=1000.0)


def test_parts_alone(torch_dev):
    """Each output has the same bits whatever else is asked for."""
    torch, dev = torch_dev
    for cols in (640, 8256):
        x, b, v, how, r, h, stats, dr, dh, got = check(
            torch, dev, 70, cols, torch.bfloat16, torch.bfloat16, "rms", "layer", True, True,
            0.2, 1.0, 0)
        for need in itertools.product([False, True], repeat=3):
            dx, db, grads = mm.residual_norm_backward(
                dr, dh, r, b, v, stats, need_dx=need[0], need_dbranch=need[1],
                need_dparams=need[2], **how)
            assert [dx is not None, db is not None, grads.gate is not None] == list(need)
            for k, t in {"dx": dx, "dbranch": db, **grads._asdict()}.items():
                assert t is None or torch.equal(t, got[k]), (k, need)
    # without the gradient of r, as behind the last block
    dx, db, _ = mm.residual_norm_backward(None, dh, r, b, v, stats, **how)
    zero, dz, _ = mm.residual_norm_backward(torch.zeros_like(dr), dh, r, b, v, stats, **how)
    assert torch.equal(dx, zero) and torch.equal(db, dz)


def test_against_layer_norm_and_dropout(torch_dev):
    """With nothing around it, the parts are the package's own operators."""
    torch, dev = torch_dev
    x = matrix(torch, dev, 33, 1000, torch.float32, 1)
    b = matrix(torch, dev, 33, 1000, torch.float32, 2)
    w, c = torch.randn(1000, device=dev), torch.randn(1000, device=dev)
    say("residual norm beside layer norm and dropout")
    r, h, stats = mm.residual_norm(x, b, mm.ResidualParams(pre_weight=w, pre_bias=c), pre="layer",
                                   dropout=0.3, seed=5, offset=6, eps=EPS)
    assert torch.equal(r, mm.dropout(b, 0.3, 5, 6, residual=x))
    y, mean, rstd, _ = mm.layer_norm(r, w, c, EPS)
    assert torch.allclose(h, y, rtol=1e-5, atol=1e-5)
    assert torch.allclose(stats.mean, mean, rtol=1e-5, atol=1e-6)
    assert torch.allclose(stats.rstd, rstd, rtol=1e-5)


@pytest.mark.parametrize("post,pre", [("layer", "rms"), ("rms", "layer"), (None, "rms"),
                                      ("layer", None)])
def test_gradients_against_differences(torch_dev, post, pre):
    """The change of sum(c r + e h) along random directions, in float64,
    against the kernels' gradients.  A central difference is off by h^2 / 6
    times the third derivative, which for rows of 40 elements of size 1 (rstd
    near 1) stays below 1e4 times the direction's size; the kernels' own errors
    are their bounds, and half a unit of float32's last place."""
    torch, dev = torch_dev
    rows, cols, step = 6, 40, 1e-4
    f32 = torch.float32
    x, b = matrix(torch, dev, rows, cols, f32, 1), matrix(torch, dev, rows, cols, f32, 2)
    v = vectors(torch, dev, cols, f32, post, pre, True, True)
    how = dict(post=post, pre=pre, scale=0.75, dropout=0.25, seed=3, offset=4)
    m = ref.mask(rows, cols, 0.25, 3, 4, dev)
    c, e = matrix(torch, dev, rows, cols, f32, 3), matrix(torch, dev, rows, cols, f32, 4)
    say("residual norm gradients", post, pre)
    r, h, stats = mm.residual_norm(x, b, v, eps=EPS, **how)
    dx, db, grads = mm.residual_norm_backward(c, e if pre else None, r, b, v, stats, **how)
    got = {"x": dx, "branch": db, **{k: t for k, t in grads._asdict().items() if t is not None}}
    point = {"x": x.double(), "branch": b.double(),
             **{k: t.double() for k, t in v._asdict().items() if t is not None}}

    def loss(at):
        p = mm.ResidualParams(**{k: at.get(k) for k in mm.ResidualParams._fields})
        val, _ = ref.residual_norm(at["x"], at["branch"], p, post, pre, 0.75, EPS, m)
        return float((c.double() * val["r"]).sum()
                     + ((e.double() * val["h"]).sum() if pre else 0.0))

    for i, (name, grad) in enumerate(got.items()):
        g = torch.Generator(device=dev).manual_seed(i)
        way = torch.randn(grad.shape, generator=g, device=dev).double()
        diff = (loss({**point, name: point[name] + step * way})
                - loss({**point, name: point[name] - step * way})) / (2 * step)
        mine = float((grad.double() * way).sum())
        size = float((grad.double() * way).abs().sum())
        # r and the statistics enter the backward pass rounded to float32: a
        # relative 2^-24 each, through sums of up to 240 terms
        room = (step ** 2 / 6 * 1e4 * float(way.abs().sum()) + 1e-15 * abs(loss(point)) / step
                + 1e3 * ref.U * (size + float(way.abs().sum())))
        assert abs(mine - diff) <= room, (name, mine, diff, room)


def test_special_values_stay_in_their_rows(torch_dev):
    torch, dev = torch_dev
    for cols in (96, 1000, 8256):
        x = matrix(torch, dev, 6, cols, torch.bfloat16, 1)
        b = matrix(torch, dev, 6, cols, torch.bfloat16, 2)
        v = vectors(torch, dev, cols, torch.bfloat16, "rms", "rms", True, False)
        how = dict(post="rms", pre="rms")
        clean = mm.residual_norm(x, b, v, **how)
        x2, b2 = x.clone(), b.clone()
        x2[2, 3], b2[4, 5] = math.inf, math.nan
        say("residual norm special values", cols)
        r, h, stats = mm.residual_norm(x2, b2, v, **how)
        rest = [0, 1, 3, 5]
        assert torch.equal(r[rest], clean[0][rest]) and torch.equal(h[rest], clean[1][rest])
        assert torch.isnan(h[4]).all() and torch.isinf(r[2, 3])
        fine = [i for i in range(cols) if i != 3]
        assert torch.equal(r[2, fine], clean[0][2, fine])
        dr, dh = torch.ones_like(x), torch.ones_like(x)
        dx, db, _ = mm.residual_norm_backward(dr, dh, r, b2, v, stats, **how)
        ex, eb, _ = mm.residual_norm_backward(dr, dh, clean[0], b, v, clean[2], **how)
        assert torch.equal(dx[rest], ex[rest]) and torch.equal(db[rest], eb[rest])


def test_what_is_dropped_has_no_part(torch_dev):
    """An infinity of the branch in a dropped place: neither in r nor in the
    gate's gradient."""
    torch, dev = torch_dev
    for cols in (200, 8256):
        m = ref.mask(12, cols, 0.5, 1, 2, dev)
        x = matrix(torch, dev, 12, cols, torch.bfloat16, 1)
        b = matrix(torch, dev, 12, cols, torch.bfloat16, 2)
        wild = torch.where(m > 0, b, torch.full_like(b, math.inf))
        wild[0] = torch.where(m[0] > 0, b[0], torch.full_like(b[0], math.nan))
        gate = torch.rand(cols, device=dev).bfloat16()
        v = mm.ResidualParams(gate=gate)
        how = dict(dropout=0.5, seed=1, offset=2)
        say("residual norm, dropped infinities", cols)
        r, _, st = mm.residual_norm(x, wild, v, **how)
        assert torch.equal(r, mm.residual_norm(x, b, v, **how)[0])
        got = mm.residual_norm_backward(x, None, None, wild, v, st, **how)
        want = mm.residual_norm_backward(x, None, None, b, v, st, **how)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2].gate, want[2].gate)


def test_empty_and_equal_rows(torch_dev):
    torch, dev = torch_dev
    e = torch.empty((0, 40), dtype=torch.bfloat16, device=dev)
    v = vectors(torch, dev, 40, torch.bfloat16, "layer", "rms", True, True)
    how = dict(post="layer", pre="rms")
    r, h, stats = mm.residual_norm(e, e, v, **how)
    assert r.shape == h.shape == (0, 40) and stats.rstd.shape == (0,) and stats.mean is None
    dx, db, grads = mm.residual_norm_backward(e, e, r, e, v, stats, **how)
    assert dx.shape == db.shape == (0, 40) and not any(g.any() for g in grads)
    with pytest.raises(mm.MmaOpsError, match="no columns"):
        mm.residual_norm(e[:, :0], e[:, :0])
    # a branch of zeros under an rms norm, a stream of one value under a layer norm
    x = torch.full((3, 500), 7.3, device=dev)
    z = torch.zeros_like(x)
    say("residual norm, equal rows")
    r, h, stats = mm.residual_norm(x, z, post="rms", pre="layer", eps=EPS)
    assert torch.equal(r, x) and not h.any()
    assert torch.allclose(stats.post_rstd, torch.full((3,), EPS ** -0.5, device=dev))


def test_offsets_past_32_bits(torch_dev):
    """Matrices of 2.2e9 elements: the last rows' results are those of the
    same rows on their own (no dropout: masks go by the row's number)."""
    torch, dev = torch_dev
    rows, cols, last = 530000, 4104, 5
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev)
    b = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev)
    x[-last:] = matrix(torch, dev, last, cols, torch.bfloat16, 1)
    b[-last:] = matrix(torch, dev, last, cols, torch.bfloat16, 2)
    v = vectors(torch, dev, cols, torch.bfloat16, "rms", "rms", True, False)
    how = dict(post="rms", pre="rms")
    say("residual norm past 32 bits")
    r, h, stats = mm.residual_norm(x, b, v, **how)
    tr, th, ts = mm.residual_norm(x[-last:], b[-last:], v, **how)
    assert torch.equal(r[-last:], tr) and torch.equal(h[-last:], th)
    assert torch.equal(stats.rstd[-last:], ts.rstd) and not r[:-last].any()
    dx, db, grads = mm.residual_norm_backward(x, h, r, b, v, stats, **how)
    ex, eb, eg = mm.residual_norm_backward(x[-last:], th, tr, b[-last:], v, ts, **how)
    assert torch.equal(dx[-last:], ex) and torch.equal(db[-last:], eb)
    for got, want in zip(grads, eg):
        assert want is None or torch.allclose(got.float(), want.float(), rtol=2.0 ** -7)


def test_repeats_streams_and_graphs(torch_dev):
    """The same bits on every call and stream, and in every replay of a
    captured pass on new inputs."""
    torch, dev = torch_dev
    for rows, cols in ((700, 1536), (40, 8256)):
        x, b, dr, dh = (matrix(torch, dev, rows, cols, torch.bfloat16, i) for i in range(4))
        v = vectors(torch, dev, cols, torch.bfloat16, "rms", "layer", True, True)
        seed = torch.tensor([5, 6], dtype=torch.int64, device=dev)
        how = dict(post="rms", pre="layer", dropout=0.1, seed=seed)

        def step(stream=None):
            r, h, stats = mm.residual_norm(x, b, v, stream=stream, **how)
            dx, db, grads = mm.residual_norm_backward(dr, dh, r, b, v, stats, stream=stream, **how)
            return [r, h, dx, db, *grads, *[s for s in stats if s is not None]]

        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream())
        say("residual norm repeats", rows, cols)
        first, other = step(), step(side)
        side.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(first, other))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(3):
            x.copy_(matrix(torch, dev, rows, cols, torch.bfloat16, 100 + i))
            seed.copy_(torch.tensor([i, 9]))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            assert all(torch.equal(s, t) for s, t in zip(got, step()))


def test_refusals(torch_dev):
    torch, dev = torch_dev
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    P, none = mm.ResidualParams, mm.ResidualStats(None, None, None, None)
    with pytest.raises(TypeError, match="float16"):
        mm.residual_norm(x.double(), x.double())
    with pytest.raises(ValueError, match="branch must have shape"):
        mm.residual_norm(x, x[:3])
    with pytest.raises(TypeError, match="branch: expected"):
        mm.residual_norm(x, x.float())
    with pytest.raises(ValueError, match="unknown norm 'batch'"):
        mm.residual_norm(x, x, pre="batch")
    with pytest.raises(ValueError, match="pre_weight without"):
        mm.residual_norm(x, x, P(pre_weight=w))
    with pytest.raises(ValueError, match="post_bias without"):
        mm.residual_norm(x, x, P(post_bias=w), pre="rms")
    with pytest.raises(TypeError, match="one type"):
        mm.residual_norm(x, x, P(gate=w, pre_weight=w.float()), pre="rms")
    with pytest.raises(ValueError, match="gate must have shape"):
        mm.residual_norm(x, x, P(gate=w[:9]))
    with pytest.raises(TypeError, match="ResidualParams"):
        mm.residual_norm(x, x, (w,))
    with pytest.raises(ValueError, match="probability"):
        mm.residual_norm(x, x, dropout=2)
    with pytest.raises(TypeError, match="ResidualStats"):
        mm.residual_norm_backward(x, None, None, x, P(), None)
    with pytest.raises(ValueError, match="dh without"):
        mm.residual_norm_backward(x, x, None, x, P(), none)
    with pytest.raises(TypeError, match="dh must"):
        mm.residual_norm_backward(x, None, x, x, P(), none, pre="rms")
    with pytest.raises(mm.MmaOpsError, match="NULL"):
        mm.residual_norm_backward(x, x, x, x, P(), none, pre="rms")
    with pytest.raises(mm.MmaOpsError, match="NULL"):
        mm.residual_norm_backward(x, None, None, None, P(gate=w), none)
    dx, db, _ = mm.residual_norm_backward(x + 1, None, None, None, P(), none, scale=2.0)
    assert (dx == 2).all() and (db == 1).all()
