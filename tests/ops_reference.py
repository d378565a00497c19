"""The native operators' formulas in float64, and error bounds for results
computed with float32 sums and one rounding of the output.

Bounds.  u is the unit roundoff of the output type, U = 2^-24 that of
float32.  A float32 sum of terms t_i over a tree or chain of depth d is off
by at most d U sum |t_i| (to first order); the kernels' sums have a depth
of at most 128 for the row and column sums tested here, and of at most
K + 64 for a product's K terms (their order inside a matrix instruction is
not known).  Each bound adds these along the formula, u |result| for the
output, and the smallest positive output for its underflow.
"""
import math

import torch

U = 2.0 ** -24
DEPTH = 128
ROUND = {t: torch.finfo(t).eps / 2 for t in (torch.float16, torch.bfloat16, torch.float32)}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
BLOCK = 32


def close(got, want, bound, what, dtype=None):
    """|got - want| <= bound everywhere, non-finite values alike."""
    dt = dtype or got.dtype
    got = got.double()
    # beyond the output type's range a result is infinite (within its bound
    # of the range's end, either)
    top = torch.finfo(dt).max
    past = torch.isinf(got) & (want.abs() + bound >= top) & (torch.sign(got) == torch.sign(want))
    want = torch.where(past, got, want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite where it should be"
    room = bound + ROUND[dt] * want.abs() + TINY[dt]
    over = ((got - want).abs() - room)[fine]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: over its bound by {worst:.3g}"


# ------------------------------------------------------------ layer norm
def layer_norm(x, w, b, eps):
    """(y, mean, rstd, bound of y, of mean, of rstd relative)."""
    x = x.double()
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(n, dtype=torch.float64, device=x.device) if b is None else b.double()
    mean = x.sum(1) / n
    d = x - mean[:, None]
    var = (d * d).sum(1) / n
    rstd = 1.0 / torch.sqrt(var + eps)
    y = d * rstd[:, None] * w + b
    size = x.abs().mean(1)
    em = DEPTH * U * size
    # d is off by em and a rounding; the variance by 2 |d| em and DEPTH U
    er = DEPTH * U + rstd * (em + U * size)
    ey = ((rstd * em)[:, None] + (d * rstd[:, None]).abs() * (er[:, None] + 4 * U)
          + U * (x * rstd[:, None]).abs()) * w.abs() + 2 * U * (y.abs() + b.abs())
    return y, mean, rstd, ey, em, er


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db, and their bounds); x in float64 already."""
    dy = dy.double()
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    r, m = rstd.double()[:, None], mean.double()[:, None]
    xh = (x - m) * r
    h = dy * w
    m0, m1 = h.sum(1, keepdim=True) / n, (h * xh).sum(1, keepdim=True) / n
    dx = r * (h - m0 - xh * m1)
    a0, a1 = h.abs().mean(1, keepdim=True), (h * xh).abs().mean(1, keepdim=True)
    edx = (DEPTH + 8) * U * r * (h.abs() + a0 + xh.abs() * a1)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return (dx, dw, db, edx, (DEPTH + 4) * U * (dy * xh).abs().sum(0),
            DEPTH * U * dy.abs().sum(0))


# ------------------------------------------------------------- checkpoint
def limit(dtype):
    return 61440.0 if dtype == torch.float16 else 1.875 * 2.0 ** 127


def e4m3(v):
    """float64 |v| <= 448 to the nearest E4M3 value, ties to an even code."""
    mag = v.abs()
    lead = torch.frexp(mag)[1] - 1          # 2^lead <= mag < 2^(lead + 1)
    step = torch.exp2((lead.clamp(min=-6) - 3).double())
    return torch.copysign(torch.round(mag / step) * step, v)


def checkpoint(x, dtype):
    """(code values, scale bytes, restored values) of float64 x."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    p = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, nb, BLOCK)
    fine = torch.isfinite(p)
    q = torch.where(fine, p.clamp(-limit(dtype), limit(dtype)), torch.zeros_like(p))
    q = torch.where(fine, torch.copysign(q, p), q)
    amax = q.abs().amax(2)
    e = torch.full(amax.shape, -117, dtype=torch.int64, device=x.device)
    for t in range(-117, 121):              # the definition, one exponent at a time
        e = torch.where(amax > 448.0 * 2.0 ** t, torch.full_like(e, t + 1), e)
    s = torch.exp2(e.double())[:, :, None]
    codes = torch.where(fine, e4m3(q / s), torch.full_like(q, math.nan))
    flat = lambda t: t.reshape(rows, -1)[:, :cols]  # noqa: E731
    return flat(codes), (e + 127).to(torch.uint8), flat(codes * s)


# ---------------------------------------------------------------- products
def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return (0.5 * torch.special.erfc(-z * math.sqrt(0.5))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# No activation here is steeper than 1.13, and each evaluation is a few
# float32 operations on values of at most |z| and 1: 16 U (|z| + 1) covers
# their roundings and the library functions' own errors of a few ulp.
STEEP, EVAL = 1.2, 16 * U


def linear(x, w, bias, name, residual):
    """(y, z, bound of y, bound of z)."""
    x, w = x.double(), w.double()
    k = x.shape[1]
    z = x @ w
    ez = (k + 64) * U * (x.abs() @ w.abs())
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * z.abs()
    y = act(z, name)
    ey = ez if name == "none" else STEEP * ez + EVAL * (z.abs() + 1)
    if residual is not None:
        y = y + residual.double()
        ey = ey + U * y.abs()
    return y, z, ey, ez


def linear_backward(dy, x, w, z, name, dtype):
    """(dx, dw, db, and their bounds); x and z in float64 already."""
    dy, w = dy.double(), w.double()
    m, n = dy.shape
    slope = act_slope(z, name) if name != "none" else torch.ones_like(dy)
    dz = dy * slope
    edz = torch.zeros_like(dz)
    if name != "none":
        edz = dy.abs() * EVAL * (z.abs() + 1) + U * dz.abs()
    # the products take dz rounded to the operands' type
    erz = edz if name == "none" else edz + ROUND[dtype] * (dz.abs() + edz) + TINY[dtype]
    dx, dw, db = dz @ w.t(), x.t() @ dz, dz.sum(0)
    a = dz.abs() + erz
    edx = erz @ w.abs().t() + (n + 64) * U * (a @ w.abs().t())
    edw = x.abs().t() @ erz + (m + 64) * U * (x.abs().t() @ a)
    return dx, dw, db, edx, edw, edz.sum(0) + DEPTH * U * (dz.abs() + edz).sum(0)
