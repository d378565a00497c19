"""The gated block's formulas in float64, and error bounds for results
computed with float32 sums and one rounding of the output (as in
ops_reference: U = 2^-24, a row or column sum has a depth of at most DEPTH)."""
import numpy as np
import torch

import ops_reference
from ops_reference import DEPTH, ROUND, TINY, U


# ---------------------------------------------------------------- dropout
def philox(counter, key):
    """Philox4x32 with ten rounds: four words of each counter.  counter: four
    arrays of 32-bit words, key: two words."""
    low = np.uint64(0xFFFFFFFF)
    x = [np.asarray(c, dtype=np.uint64) for c in counter]
    k0, k1 = key
    for _ in range(10):
        p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(p1 >> np.uint64(32)) ^ x[1] ^ np.uint64(k0), p1 & low,
             (p0 >> np.uint64(32)) ^ x[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return x


def numbers(rows, cols, seed, offset):
    """The 16-bit numbers of the elements; rows: how many, or which ones."""
    rows = range(rows) if isinstance(rows, int) else rows
    out = np.empty((len(rows), cols), dtype=np.int64)
    col = np.arange(cols)
    for i, row in enumerate(rows):
        count = [(row * 2 ** 24 + int(c) // 8) for c in col[::8]]
        words = philox([np.array([c % 2 ** 32 for c in count]), np.array([c >> 32 for c in count]),
                        np.full(len(count), offset % 2 ** 32), np.full(len(count), offset >> 32)],
                       (seed % 2 ** 32, seed >> 32))
        words = np.stack(words, axis=1)                       # [columns / 8][word]
        out[i] = words[col // 8, col % 8 // 2] >> (16 * (col % 2)).astype(np.uint64) & 0xFFFF
    return out


def threshold(p):
    return int(np.floor(65536 * p + 0.5))


def mask(rows, cols, p, seed, offset, dev):
    """float64 0 or 65536 / (65536 - T)."""
    t = threshold(p)
    up = 65536 / (65536 - t) if t < 65536 else 0.0
    return torch.from_numpy((numbers(rows, cols, seed, offset) >= t) * up).to(dev)


def dropped(x, m):
    """What is dropped is 0, an infinity or NaN too."""
    return torch.where(m > 0, x * m, torch.zeros_like(x))


# --------------------------------------------- sum into the residual stream
def _one(v, n, dev, fill=1.0):
    return (torch.full((n,), fill, dtype=torch.float64, device=dev) if v is None else v.double())


def norm(x, kind, w, b, eps, ex=None):
    """(y, mean, rstd, bound of y, of mean, of rstd relative); ex: how far each
    element of x may be off already (None: not at all)."""
    n = x.shape[1]
    w, b = _one(w, n, x.device), _one(b, n, x.device, 0.0)
    mean = x.sum(1) / n if kind == "layer" else torch.zeros_like(x[:, 0])
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / n + eps)
    y = d * rstd[:, None] * w + b
    size = x.abs().mean(1)
    em = DEPTH * U * size if kind == "layer" else torch.zeros_like(size)
    # d is off by em and a rounding, the variance by 2 |d| em and DEPTH U
    er = DEPTH * U + rstd * (em + U * size)
    ey = ((rstd * em)[:, None] + (d * rstd[:, None]).abs() * (er[:, None] + 4 * U)
          + U * (x * rstd[:, None]).abs()) * w.abs() + 2 * U * (y.abs() + b.abs())
    if ex is not None:
        # to first order: d moves by ed, the variance by 2 mean |d| ed, and
        # twice that for what is of higher order
        ed = ex + (ex.mean(1, keepdim=True) if kind == "layer" else 0.0)
        rel = rstd ** 2 * (d.abs() * ed).mean(1)
        ey = ey + 2 * w.abs() * rstd[:, None] * (ed + d.abs() * rel[:, None])
        em = em + (ex.mean(1) if kind == "layer" else 0.0)
        er = er + 2 * rel
    return y, mean, rstd, ey, em, er


def residual_norm(x, branch, p, post, pre, scale, eps, m):
    """Dictionaries of values and bounds; m: the mask with its factor, or None."""
    x, b = x.double(), branch.double()
    n, dev = x.shape[1], x.device
    val, off = {}, {}
    v, ev = b, torch.zeros_like(b)
    if post:
        v, mean, rstd, ev, em, er = norm(b, post, p.post_weight, p.post_bias, eps)
        val["post_mean"], off["post_mean"] = mean, em
        val["post_rstd"], off["post_rstd"] = rstd, er * rstd
    if m is not None:
        v, ev = dropped(v, m), torch.where(m > 0, ev * m, torch.zeros_like(ev))
    g = _one(p.gate, n, dev)
    val["r"] = r = scale * x + g * v
    off["r"] = ex = 4 * U * ((scale * x).abs() + (g * v).abs()) + g.abs() * ev
    if pre:
        h, mean, rstd, eh, em, er = norm(r, pre, p.pre_weight, p.pre_bias, eps, ex)
        val["h"], off["h"] = h, eh
        val["mean"], off["mean"] = mean, em
        val["rstd"], off["rstd"] = rstd, er * rstd
    return val, off


def residual_norm_backward(dr, dh, r, branch, p, stats, post, pre, scale, m):
    """The same for the gradients: dx, dbranch and the vectors' names."""
    lead = dh if pre else dr
    n, dev = lead.shape[1], lead.device
    val, off = {}, {}
    t = torch.zeros(lead.shape, dtype=torch.float64, device=dev) if dr is None else dr.double()
    et = torch.zeros_like(t)
    if pre:
        d, rr, q = dh.double(), r.double(), stats.rstd.double()[:, None]
        mu = stats.mean.double()[:, None] if pre == "layer" else torch.zeros_like(q)
        rh, erh = (rr - mu) * q, 3 * U * (rr.abs() + mu.abs()) * q
        hq = d * _one(p.pre_weight, n, dev)
        m1, em1 = (hq * rh).mean(1, keepdim=True), (DEPTH * U * (hq * rh).abs()
                                                    + hq.abs() * erh).mean(1, keepdim=True)
        m0 = hq.mean(1, keepdim=True) if pre == "layer" else torch.zeros_like(m1)
        em0 = (DEPTH * U * hq.abs().mean(1, keepdim=True) if pre == "layer"
               else torch.zeros_like(m1))
        et = (6 * U * (t.abs() + q * (hq.abs() + m0.abs() + (rh * m1).abs()))
              + q * (em0 + rh.abs() * em1 + erh * m1.abs()))
        t = t + q * (hq - m0 - rh * m1)
        val["pre_weight"] = (d * rh).sum(0)
        off["pre_weight"] = (d.abs() * erh + (DEPTH + 4) * U * (d * rh).abs()).sum(0)
        val["pre_bias"], off["pre_bias"] = d.sum(0), DEPTH * U * d.abs().sum(0)
    val["dx"], off["dx"] = scale * t, abs(scale) * et + 2 * U * (scale * t).abs()
    td, etd = t, et
    if m is not None:
        td = dropped(t, m)
        etd = et * m + 2 * U * td.abs()
    g = _one(p.gate, n, dev)
    if branch is None:
        val["dbranch"], off["dbranch"] = td * g, etd * g.abs() + 2 * U * (td * g).abs()
        return val, off
    b = branch.double()
    if post:
        k = stats.post_rstd.double()[:, None]
        mu = stats.post_mean.double()[:, None] if post == "layer" else torch.zeros_like(k)
    else:
        k, mu = torch.ones_like(b[:, :1]), torch.zeros_like(b[:, :1])
    bh, ebh = (b - mu) * k, 3 * U * (b.abs() + mu.abs()) * k
    w, wb = ((_one(p.post_weight, n, dev), _one(p.post_bias, n, dev, 0.0)) if post else
             (torch.ones_like(g), torch.zeros_like(g)))
    qq = td * g * w
    eqq = etd * (g * w).abs() + 3 * U * qq.abs()
    if post:
        k1 = (qq * bh).mean(1, keepdim=True)
        ek1 = (DEPTH * U * (qq * bh).abs() + eqq * bh.abs() + qq.abs() * ebh).mean(1, keepdim=True)
        k0, ek0 = torch.zeros_like(k1), torch.zeros_like(k1)
        if post == "layer":
            k0 = qq.mean(1, keepdim=True)
            ek0 = (DEPTH * U * qq.abs() + eqq).mean(1, keepdim=True)
        val["dbranch"] = k * (qq - k0 - bh * k1)
        off["dbranch"] = k * (eqq + ek0 + bh.abs() * ek1 + ebh * k1.abs()
                              + 6 * U * (qq.abs() + k0.abs() + (bh * k1).abs()))
    else:
        val["dbranch"], off["dbranch"] = qq, eqq
    kept = bh if m is None else dropped(bh, (m > 0).double())
    s1, s0 = (td * kept).sum(0), td.sum(0)
    e1 = (etd * kept.abs() + td.abs() * ebh + (DEPTH + 4) * U * (td * kept).abs()).sum(0)
    e0 = (etd + DEPTH * U * td.abs()).sum(0)
    val["gate"] = w * s1 + wb * s0
    off["gate"] = w.abs() * e1 + wb.abs() * e0 + 3 * U * ((w * s1).abs() + (wb * s0).abs())
    if post:
        val["post_weight"], off["post_weight"] = g * s1, g.abs() * e1 + U * (g * s1).abs()
        val["post_bias"], off["post_bias"] = g * s0, g.abs() * e0 + U * (g * s0).abs()
    return val, off


# ------------------------------------------------------------ gated layer
def gated_linear(x, wg, wu, bg, bu, act):
    """(y, g, u, and their bounds)."""
    g, _, eg, _ = ops_reference.linear(x, wg, bg, "none", None)
    u, _, eu, _ = ops_reference.linear(x, wu, bu, "none", None)
    a = ops_reference.act(g, act)
    ea = eg if act == "none" else (ops_reference.STEEP * eg
                                   + ops_reference.EVAL * (g.abs() + 1))
    return a * u, g, u, u.abs() * ea + a.abs() * eu + ea * eu + U * (a * u).abs(), eg, eu


def gated_linear_backward(dy, x, wg, wu, g, u, act, dtype):
    """dx, dw_gate, dw_up, dbias_gate, dbias_up and their bounds; x, g and u in
    float64 already."""
    dy, wg, wu = dy.double(), wg.double(), wu.double()
    m, n = dy.shape
    a, slope = ops_reference.act(g, act), ops_reference.act_slope(g, act)
    ev = 0.0 if act == "none" else ops_reference.EVAL * (g.abs() + 1)
    dg, du = dy * u * slope, dy * a
    eg, eu = (dy * u).abs() * ev + 3 * U * dg.abs(), dy.abs() * ev + U * du.abs()
    # the products take both rounded to the operands' type
    rg = eg + ROUND[dtype] * (dg.abs() + eg) + TINY[dtype]
    ru = eu + ROUND[dtype] * (du.abs() + eu) + TINY[dtype]
    ag, au, xa = dg.abs() + rg, du.abs() + ru, x.abs()
    dx = dg @ wg.t() + du @ wu.t()
    ex = (rg @ wg.abs().t() + ru @ wu.abs().t()
          + (2 * n + 64) * U * (ag @ wg.abs().t() + au @ wu.abs().t()))
    values = dx, x.t() @ dg, x.t() @ du, dg.sum(0), du.sum(0)
    bounds = (ex, xa.t() @ rg + (m + 64) * U * (xa.t() @ ag),
              xa.t() @ ru + (m + 64) * U * (xa.t() @ au),
              eg.sum(0) + DEPTH * U * (dg.abs() + eg).sum(0),
              eu.sum(0) + DEPTH * U * (du.abs() + eu).sum(0))
    return values, bounds
