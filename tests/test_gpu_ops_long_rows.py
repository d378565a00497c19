"""Products whose operands have rows so long that a tile of them spans more
than 2^32 bytes.  The elements are -1, 0 and 1: every sum is exact in
float32, whatever its order, so results are compared bit for bit."""
import pytest

import bit_exact_matrix_amd as mm
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu
STEP = 1 << 22  # columns compared at a time


def signs(torch, dev, rows, cols, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    for c in range(0, cols, STEP):
        part = out[:, c:c + STEP]
        part.copy_(torch.randint(-1, 2, part.shape, generator=g, device=dev, dtype=torch.int8))
    return out


def inner(torch, a, b):
    """a b^T over their long rows, exact in float32."""
    s = torch.zeros((a.shape[0], b.shape[0]), device=a.device)
    for c in range(0, a.shape[1], STEP):
        s += a[:, c:c + STEP].float() @ b[:, c:c + STEP].float().t().contiguous()
    return s


@pytest.mark.parametrize("m,n,k", [(128, 40_000_000, 64), (40, 40_000_001, 72),
                                   (128, 70_000_000, 16)])
def test_long_rows_of_the_weight(torch_dev, m, n, k):
    """W stored K x N; the last has more tiles than one row of a grid."""
    torch, dev = torch_dev
    x, w = signs(torch, dev, m, k, 1), signs(torch, dev, k, n, 2)
    say("linear, long rows of W", m, n, k)
    y, _ = mm.linear(x, w)
    for c in range(0, n, STEP):
        assert torch.equal(y[:, c:c + STEP], (x.float() @ w[:, c:c + STEP].float()).bfloat16())


@pytest.mark.parametrize("m,n,k", [(1024, 1024, 9_500_000), (256, 64, 36_000_000),
                                   (16, 64, 40_000_000),
                                   (20, 66, 40_000_001)])
def test_long_inner_size(torch_dev, m, n, k):
    """W stored N x K: rows of both operands are long."""
    torch, dev = torch_dev
    x, w = signs(torch, dev, m, k, 3), signs(torch, dev, n, k, 4)
    say("linear, long inner size", m, n, k)
    y, _ = mm.linear(x, w.t(), out_dtype=torch.float32)
    assert torch.equal(y, inner(torch, x, w))


def test_long_rows_in_the_backward_pass(torch_dev):
    """dW over long rows of X, dX over long rows of dY and W."""
    torch, dev = torch_dev
    m, n, k = 64, 16, 40_000_000
    x, dy, w = (signs(torch, dev, r, c, 5 + r) for r, c in ((m, k), (m, n), (k, n)))
    say("linear backward, long rows of X")
    _, dw, _ = mm.linear_backward(dy, x, w, need_dx=False, need_dbias=False)
    for c in range(0, k, STEP):
        want = x[:, c:c + STEP].float().t().contiguous() @ dy.float()
        assert torch.equal(dw[c:c + STEP], want.bfloat16())
    del x, w, dw
    m, n, k = 16, 40_000_000, 24
    x, dy, w = (signs(torch, dev, r, c, 5 + r) for r, c in ((m, k), (m, n), (k, n)))
    say("linear backward, long rows of dY and W")
    dx, _, db = mm.linear_backward(dy, x, w, need_dw=False, bias_dtype=torch.float32)
    assert torch.equal(dx, inner(torch, dy, w).bfloat16())
    for c in range(0, n, STEP):
        assert torch.equal(db[c:c + STEP], dy[:, c:c + STEP].float().sum(0))
