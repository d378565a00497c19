"""Edges of the gated block's operators: the same tensor in two places, calls
from two threads, graphs side by side, rows so long that a tile spans more than
2^32 bytes, and rows of more columns than one row of a grid."""
import threading

import pytest

import bit_exact_matrix_amd as mm
import block_reference as ref
import ops_reference
from test_gpu_ops_linear import matrix
from test_gpu_ops_long_rows import STEP, inner, signs
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_same_tensor_in_two_places(torch_dev):
    torch, dev = torch_dev
    for m, n, k in ((1, 64, 128), (40, 72, 72), (300, 264, 200)):
        x = matrix(torch, dev, m, k, torch.bfloat16, 1)
        w = matrix(torch, dev, k, n, torch.bfloat16, 2, scale=k ** -0.5)
        say("gated, one weight twice", m, n, k)
        y, (g, u) = mm.gated_linear(x, w, w, activation="none", keep="full")
        assert torch.equal(g, u)
        want, _, _, ey, _, _ = ref.gated_linear(x, w, w, None, None, "none")
        ops_reference.close(y, want, ey, "y")
        dy = matrix(torch, dev, m, n, torch.bfloat16, 3)
        apart = mm.gated_linear_backward(dy, x, w, w.clone(), (g, g.clone()))
        same = mm.gated_linear_backward(dy, x, w, w, (g, g))
        assert all(torch.equal(a, b) for a, b in zip(apart, same))
        # the gradient of y is the input itself, where the sizes allow it
        if n == k:
            a = mm.gated_linear_backward(x, x, w, w, (g, u))
            b = mm.gated_linear_backward(x.clone(), x, w, w, (g, u))
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    x = matrix(torch, dev, 30, 520, torch.bfloat16, 1)
    v = torch.rand(520, device=dev).bfloat16()
    params = mm.ResidualParams(v, v, v, v, v)
    how = dict(post="layer", pre="layer", dropout=0.2, seed=1)
    say("residual norm, one tensor everywhere")
    r, h, stats = mm.residual_norm(x, x, params, **how)
    again = mm.residual_norm(x, x.clone(), mm.ResidualParams(*(v.clone() for _ in range(5))),
                             **how)
    assert torch.equal(r, again[0]) and torch.equal(h, again[1])
    a = mm.residual_norm_backward(x, x, r, x, params, stats, **how)
    b = mm.residual_norm_backward(x.clone(), x.clone(), r, x.clone(), params, stats, **how)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(s, t) for s, t in zip(a[2], b[2]))
    assert torch.equal(mm.dropout(x, 0.5, 1, residual=x),
                       mm.dropout(x, 0.5, 1, residual=x.clone()))


def test_two_threads_on_two_streams(torch_dev):
    torch, dev = torch_dev
    sizes = ((700, 520, 264), (5, 1024, 512))
    work, want = [], []
    for i, (m, n, k) in enumerate(sizes):
        x = matrix(torch, dev, m, k, torch.bfloat16, i)
        w = [matrix(torch, dev, k, n, torch.bfloat16, i + j, scale=k ** -0.5) for j in (5, 9)]
        dy = matrix(torch, dev, m, n, torch.bfloat16, i + 20)

        def step(x=x, w=w, dy=dy):
            y, kept = mm.gated_linear(x, *w, keep="checkpoint")
            r, h, stats = mm.residual_norm(dy, y, pre="rms", post="rms", dropout=0.1, seed=7)
            back = mm.residual_norm_backward(dy, y, r, y, mm.ResidualParams(), stats, pre="rms",
                                             post="rms", dropout=0.1, seed=7)
            return [y, r, h, *back[:2], *mm.gated_linear_backward(dy, x, *w, kept)]

        work.append(step)
        want.append(step())
    torch.cuda.synchronize()
    say("two threads")
    got, failed = [None, None], []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream(device=dev)):
                for _ in range(10):
                    got[i] = work[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001  shown by the assertion below
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for g, w in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(g, w))


def test_two_graphs_in_turn(torch_dev):
    """Two captured passes, replayed in turn: neither's workspace is the
    other's."""
    torch, dev = torch_dev
    parts = []
    for m, n, k in ((64, 2048, 512), (1, 2048, 2048)):
        x = matrix(torch, dev, m, k, torch.bfloat16, m)
        w = [matrix(torch, dev, n, k, torch.bfloat16, j, scale=k ** -0.5).t() for j in (1, 2)]
        dy = matrix(torch, dev, m, n, torch.bfloat16, 9)

        def step(x=x, w=w, dy=dy):
            y, kept = mm.gated_linear(x, *w, keep="checkpoint")
            return [y, *mm.gated_linear_backward(dy, x, *w, kept)]

        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        parts.append((graph, out, step, x))
    for i in range(3):
        for graph, _, _, x in parts:
            x.copy_(matrix(torch, dev, *x.shape, torch.bfloat16, 70 + i))
        say("two graphs, turn", i)
        for graph, _, _, _ in parts:
            graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in out] for _, out, _, _ in parts]
        for g, (_, _, step, _) in zip(got, parts):
            assert all(torch.equal(s, t) for s, t in zip(g, step()))


@pytest.mark.parametrize("m,n,k", [(100, 40_000_000, 64), (20, 20_000_001, 72)])
def test_long_rows_of_the_weights(torch_dev, m, n, k):
    """Weights stored K x N.  The elements are -1, 0 and 1: every sum is exact,
    and so is the product of two of them, up to its one rounding."""
    torch, dev = torch_dev
    x, wg, wu = signs(torch, dev, m, k, 1), signs(torch, dev, k, n, 2), signs(torch, dev, k, n, 3)
    say("gated, long rows of the weights", m, n, k)
    y, _ = mm.gated_linear(x, wg, wu, activation="none")
    for c in range(0, n, STEP):
        g, u = (x.float() @ w[:, c:c + STEP].float() for w in (wg, wu))
        assert torch.equal(y[:, c:c + STEP], (g * u).bfloat16())


@pytest.mark.parametrize("m,n,k", [(256, 64, 20_000_000), (16, 64, 40_000_000),
                                   (20, 66, 20_000_001)])
def test_long_inner_size(torch_dev, m, n, k):
    """Weights stored N x K: rows of all operands are long.  g and u below 2^24
    are exact in float32; their product is rounded there once."""
    torch, dev = torch_dev
    x, wg, wu = signs(torch, dev, m, k, 3), signs(torch, dev, n, k, 4), signs(torch, dev, n, k, 5)
    say("gated, long inner size", m, n, k)
    y, _ = mm.gated_linear(x, wg.t(), wu.t(), activation="none", out_dtype=torch.float32)
    assert torch.equal(y, inner(torch, x, wg) * inner(torch, x, wu))


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_long_inner_size_of_the_input_gradient(torch_dev, layout):
    """dX sums over two long rows: dg = dY and du = dY for u = 1, g = 1 without an
    activation, all exact."""
    torch, dev = torch_dev
    m, n, k = 16, 20_000_000, 64
    dy = signs(torch, dev, m, n, 1)
    w = [signs(torch, dev, *((k, n) if layout == "kn" else (n, k)), i) for i in (2, 3)]
    w = w if layout == "kn" else [t.t() for t in w]
    one = torch.ones((m, n), dtype=torch.bfloat16, device=dev)
    say("gated backward, long rows", layout)
    dx = mm.gated_linear_backward(dy, one[:, :k], *w, (one, one), activation="none",
                                  need_dw=False, need_dbias=False)[0]
    want = sum(inner(torch, dy, t) for t in w)
    assert torch.equal(dx, want.bfloat16())


def test_more_columns_than_a_grid_has(torch_dev):
    """Rows of 2^25 + 2^20 + 3 elements: the vectors' gradients take more than
    one row of the last kernel's grid.  Ones and twos: exact sums."""
    torch, dev = torch_dev
    cols = (1 << 25) + (1 << 20) + 3
    dr = torch.ones((2, cols), dtype=torch.bfloat16, device=dev)
    dr[1] = 2
    b = torch.full_like(dr, 0.5)
    gate = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    params = mm.ResidualParams(gate=gate)
    say("residual norm, long rows")
    r, h, stats = mm.residual_norm(dr, b, params)
    assert torch.equal(r, dr + 0.5) and h is None
    dx, db, grads = mm.residual_norm_backward(dr, None, None, b, params, stats)
    assert torch.equal(dx, dr) and torch.equal(db, dr)
    assert (grads.gate == 1.5).all()
    y = mm.dropout(dr, 0.5, 3, 4)
    m = ref.mask([1], 64, 0.5, 3, 4, dev)
    assert torch.equal(y[1:, :64].double(), 2 * m)


@pytest.mark.parametrize("cols", [512, 500, 1024, 1536, 2048])
@pytest.mark.parametrize("post", [None, "rms"])
def test_last_rows_that_are_not_finite_where_they_are_dropped(torch_dev, cols, post):
    """A workgroup works on several of these rows, and where the matrix has fewer, the
    places of the others take no part: not with what the last row holds."""
    torch, dev = torch_dev
    for rows in (1, 3, 5, 2049):
        say("dropped infinities in the last row", cols, post, rows)
        how = dict(post=post, dropout=0.5, seed=3, offset=rows)
        branch = matrix(torch, dev, rows, cols, torch.bfloat16, 1)
        dr = matrix(torch, dev, rows, cols, torch.bfloat16, 2)
        v = torch.rand(cols, device=dev).bfloat16()
        params = mm.ResidualParams(gate=v, post_weight=v if post else None)
        kept = ref.mask(rows, cols, 0.5, 3, rows, dev)[-1] != 0
        x = torch.zeros_like(branch)
        _, _, stats = mm.residual_norm(x, branch, params, **how)
        _, _, want = mm.residual_norm_backward(dr, None, None, branch, params, stats, **how)
        branch[-1, ~kept] = float("inf")
        if post:
            stats.post_rstd[-1] = float("nan")
        _, _, got = mm.residual_norm_backward(dr, None, None, branch, params, stats, **how)
        for a, b in zip(got, want):
            if a is not None:
                assert torch.equal(a[~kept], b[~kept])
                assert bool(torch.isfinite(a[~kept]).all())


@pytest.mark.parametrize("cols", [1, 8, 60, 100])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_equal_rows_of_large_values(torch_dev, cols, dtype):
    """A row of equal values has an rstd of 1 / sqrt(eps): with a mean of 2^120 their
    product is past a float, and no element of the row is that far from its mean.
    (The row's sum has to be a float: 100 2^120 < 2^127.)"""
    torch, dev = torch_dev
    dt = getattr(torch, dtype)
    for rows in (1, 5):
        say("equal rows", cols, dtype, rows)
        big = torch.full((rows, cols), 2.0 ** 120, device=dev, dtype=dt)
        none = torch.zeros_like(big)
        how = dict(post="layer", pre="layer")
        # the norm of equal values is 0, in both places
        r, h, stats = mm.residual_norm(big, big, mm.ResidualParams(), **how)
        assert torch.equal(r, big) and not bool(h.any())
        dr, dh = (matrix(torch, dev, rows, cols, dt, s) for s in (1, 2))
        v = torch.ones(cols, device=dev, dtype=dt)
        p = mm.ResidualParams(None, v, v, v, v)
        dx, db, grads = mm.residual_norm_backward(dr, dh, r, big, p, stats, **how)
        centred = dh.double() - dh.double().mean(dim=1, keepdim=True)
        want = dr.double() + stats.rstd.double()[:, None] * centred
        for t in (dx, db, *grads[1:]):
            assert bool(torch.isfinite(t).all())
        assert not bool(grads.pre_weight.any()) and not bool(grads.post_weight.any())
        # the mean's sum and the rounding of dx: half a step, and 2^-20 of what is added
        far = dr.double().abs() + stats.rstd.double()[:, None] * dh.double().abs().amax(
            dim=1, keepdim=True)
        bound = want.abs() * torch.finfo(dt).eps + far * 2.0 ** -18
        assert bool(((dx.double() - want).abs() <= bound).all())
