"""The measured cases of the gated block's operators, with their plain forms.

They are what one gated feed-forward block of a training step runs beside the
products that are there already: the projections with their gate, the dropout
inside the block, and the sum into the residual stream with the norms around it.

  gated_linear            g = x Wg + bg, u = x Wu + bu, y = act(g) u; with
                          `save`, the 8-bit checkpoints of g and u too
  gated_linear_backward   dg = dy u act'(g), du = dy act(g), their column sums,
                          dx = dg Wg^T + du Wu^T, dWg = x^T dg, dWu = x^T du;
                          x, g and u whole, or as 8-bit checkpoints
  dropout                 y = mask x / (1 - p) + residual
  residual_norm           v = post(branch), r = scale x + gate drop(v),
                          h = pre(r); post and pre are a layer norm, an rms norm
                          or nothing
  residual_norm_backward  its gradients, from those of r and h

The mask of an element goes by its place alone.  Philox4x32 with ten rounds
(Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011) is run on the counter (row 2^24 + column / 8, offset), both of 64 bits,
with the seed as its key; element c of a row has half c mod 2 of word
(c mod 8) / 2.  An element is kept where these 16 bits are at least
T = round(65536 p), and 1 / (1 - p) is 65536 / (65536 - T).

Checkpoints: E4M3 codes (OCP "FN") and one power of two for each 32 consecutive
elements of a row, the smallest 2^e, -117 <= e <= 120, with max |x| <= 448 * 2^e
over the block's finite elements.

Where `own` is false, `run` computes the plain form: elementary torch operations
in float32, rounded once at the end.  Where it is true, it calls the package's
operators.  `exact` computes the same in float64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32
EPS = 1e-5


def listed():
    return [
        # one token of a decoding step: both weights are read once
        dict(name="gated_token", op="gated_linear", m=1, n=4096, k=4096, dtype="bf16",
             act="silu", layout="nk", bias=False, save=False),
        # a few tokens against a wide block
        dict(name="gated_few", op="gated_linear", m=16, n=8192, k=4096, dtype="fp16",
             act="gelu_tanh", layout="kn", bias=False, save=False),
        # the square sizes of the package's other products
        dict(name="gated_square", op="gated_linear", m=4096, n=4096, k=4096, dtype="bf16",
             act="gelu", layout="kn", bias=True, save=False),
        # odd sizes, and what a training step keeps in 8 bits
        dict(name="gated_ragged", op="gated_linear", m=1999, n=1499, k=1024, dtype="fp16",
             act="silu", layout="kn", bias=True, save=True),
        # the backward pass of a training step's block from 8-bit checkpoints
        dict(name="gated_back_saved", op="gated_linear_backward", m=4096, n=4096, k=1024,
             dtype="bf16", act="silu", layout="kn", saved=True),
        # a small backward pass with odd sizes, from whole activations
        dict(name="gated_back_small", op="gated_linear_backward", m=299, n=260, k=640,
             dtype="fp16", act="gelu", layout="nk", saved=False),
        # a training batch inside a block
        dict(name="dropout_batch", op="dropout", rows=8192, cols=4096, dtype="bf16", p=0.1,
             residual=False),
        # a small ragged batch, added to the residual stream
        dict(name="dropout_ragged", op="dropout", rows=70, cols=1499, dtype="fp32", p=0.5,
             residual=True),
        # one token between two blocks of a decoding step
        dict(name="join_token", op="residual_norm", rows=1, cols=4096, dtype="bf16", post="none",
             pre="rms", gate=False, p=0.0, scale=1.0),
        # a training batch: norms on both sides, the gate, and dropout
        dict(name="join_train", op="residual_norm", rows=8192, cols=4096, dtype="bf16",
             post="rms", pre="rms", gate=True, p=0.1, scale=1.0),
        # the backward pass of that batch
        dict(name="join_back", op="residual_norm_backward", rows=8192, cols=4096, dtype="bf16",
             post="rms", pre="rms", gate=True, p=0.1, scale=1.0),
        # layer norms, a scaled residual, a width off the vector sizes
        dict(name="join_back_ragged", op="residual_norm_backward", rows=4097, cols=1000,
             dtype="fp32", post="layer", pre="layer", gate=True, p=0.0, scale=0.8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi], even over its logarithm; half of the larger ones are multiples of 320."""
    v = _log(rng, lo, hi)
    return v // 320 * 320 if v >= 320 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["gated_linear", "gated_linear", "gated_linear_backward", "dropout",
                     "residual_norm", "residual_norm_backward"])
    if op in ("dropout", "residual_norm", "residual_norm_backward"):
        cols = _size(rng, 33, 16384)
        rows = _size(rng, 1, max(1, min(65536, 8192 * 4096 // 2 // cols)))
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    p=rng.choice([0.0, 0.05, 0.1, 0.3]))
        if op == "dropout":
            case["p"] = case["p"] or 0.2
            case["residual"] = rng.random() < 0.5
        else:
            case["post"] = rng.choice(["none", "rms", "layer"])
            case["pre"] = rng.choice(["none", "rms", "rms", "layer"])
            case["gate"] = rng.random() < 0.6
            case["scale"] = rng.choice([1.0, 1.0, 0.7])
        return case
    # 8 M N K of the backward pass stays below the largest listed one
    k = _size(rng, 48, 8192)
    n = _size(rng, 48, 16384 if op == "gated_linear" else 8192)
    budget = 4096 ** 3 // (2 if op == "gated_linear" else 4)
    m = _size(rng, 1, max(1, min(8192, budget // (n * k))))
    case = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "fp16"]),
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "silu"]),
                layout=rng.choice(["kn", "nk"]))
    if op == "gated_linear":
        case["bias"] = rng.random() < 0.5
        case["save"] = rng.random() < 0.5
    else:
        case["saved"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _activations(g, rows, cols, dtype):
    """N(0, 1) with a few outlying channels and a small offset of each row."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x[:, :: max(1, cols // 7)] *= 12.0
    x += 0.2 * torch.randn((rows, 1), generator=g, device="cuda")
    return x.to(dtype)


def _blocks(x):
    """float32 rows, zero-padded to whole blocks: [rows, blocks, 32]."""
    rows, cols = x.shape
    n = -(-cols // BLOCK)
    p = torch.zeros((rows, n * BLOCK), dtype=torch.float32, device=x.device)
    p[:, :cols] = x
    return p.view(rows, n, BLOCK)


def _encode(x, limit):
    """(codes as float8, scale exponents + 127) of float32 x."""
    p = _blocks(x)
    fine = torch.isfinite(p)
    mag = torch.where(fine, p.abs(), torch.zeros_like(p)).clamp(max=limit)
    f, e = torch.frexp(mag.amax(dim=2))
    e = torch.where(f == 0, torch.full_like(e, -117), (e - 9 + (f > 0.875)).clamp(-117, 120))
    v = torch.ldexp(torch.copysign(mag, p), -e.unsqueeze(2))
    v = torch.where(fine, v, torch.full_like(v, math.nan))
    codes = v.to(torch.float8_e4m3fn).view(x.shape[0], -1)[:, : x.shape[1]].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _decode(codes, scales):
    """The float32 values of a checkpoint."""
    v = torch.ldexp(_blocks(codes.float()), (scales.to(torch.int32) - 127).unsqueeze(2))
    return v.view(codes.shape[0], -1)[:, : codes.shape[1]]


def _limit(dtype):
    return 61440.0 if dtype == torch.float16 else 1.875 * 2.0 ** 127


def _threshold(p):
    return int(math.floor(65536.0 * p + 0.5))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    dt = DTYPES[case["dtype"]]
    # the generator's seed and offset are the step's: the sampler's state of a training run
    s = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63, "offset": 7 + seed}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "dropout":
        s["x"] = _activations(g, case["rows"], case["cols"], dt)
        s["residual"] = (_activations(g, case["rows"], case["cols"], dt)
                         if case["residual"] else None)
        return s
    if case["op"] in ("residual_norm", "residual_norm_backward"):
        rows, cols = case["rows"], case["cols"]
        x, b = _activations(g, rows, cols, dt), normal(rows, cols).to(dt)
        s["branch"] = b

        def vector(mean, there):
            return (mean + 0.2 * normal(cols)).to(dt) if there else None

        s["gate"] = vector(0.5, case["gate"])
        for side in ("post", "pre"):
            s[side + "_weight"] = vector(1.0, case[side] != "none")
            s[side + "_bias"] = vector(0.0, case[side] == "layer")
        if case["op"] == "residual_norm":
            s["x"] = x
            return s
        # what the forward pass left: r in the stream's type, statistics in float32
        r, _, stats = _join64(case, x, s)
        s["r"] = r.to(dt)
        s["stats"] = tuple(None if t is None else t.float() for t in stats)
        s["dr"] = normal(rows, cols).to(dt)
        s["dh"] = normal(rows, cols).to(dt) if case["pre"] != "none" else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    x = _activations(g, m, k, dt)
    for name in ("w_gate", "w_up"):
        w = (normal(k, n) * (0.7 / math.sqrt(k))).to(dt)
        s[name] = w if case["layout"] == "kn" else w.t().contiguous().t()
    if case["op"] == "gated_linear":
        s["x"] = x
        s["bias_gate"] = (0.2 * normal(n)).to(dt) if case["bias"] else None
        s["bias_up"] = (0.2 * normal(n)).to(dt) if case["bias"] else None
        return s
    s["dy"] = normal(m, n).to(dt)
    kept = (1.5 * normal(m, n)).to(dt), (1.5 * normal(m, n)).to(dt)
    if case["saved"]:
        s["x"] = _encode(x.float(), _limit(dt))
        s["kept"] = tuple(_encode(t.float(), _limit(dt)) for t in kept)
    else:
        s["x"], s["kept"] = x, kept
    return s


# ------------------------------------------------------- plain forms (fp32)
def _act(z, name):
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _whole(v):
    return _decode(*v) if isinstance(v, tuple) else v.float()


def _kept_elements(rows, cols, p, seed, offset, device):
    """The mask: Philox4x32-10 in 64-bit integers."""
    low = 0xFFFFFFFF
    row = torch.arange(rows, dtype=torch.int64, device=device)[:, None]
    at = (row << 24) + torch.arange(-(-cols // 8), dtype=torch.int64, device=device)[None, :]
    a, b = at & low, (at >> 32) & low
    c, d = torch.full_like(a, offset & low), torch.full_like(a, offset >> 32 & low)
    for r in range(10):
        # a 32-bit product's words; past 2^63 it wraps, and its bits stay
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        k0, k1 = (seed + r * 0x9E3779B9) & low, ((seed >> 32) + r * 0xBB67AE85) & low
        a, b, c, d = (v >> 32 & low) ^ b ^ k0, v & low, (u >> 32 & low) ^ d ^ k1, u & low
    words = torch.stack([a, b, c, d], dim=2)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=3)
    return halves.view(rows, -1)[:, :cols] >= _threshold(p)


def _dropped(v, s):
    """v / (1 - p) where it is kept, else 0."""
    p = s["case"]["p"]
    if p == 0.0:
        return v
    keep = _kept_elements(*v.shape, p, s["seed"], s["offset"], v.device)
    return torch.where(keep, v * (65536.0 / (65536 - _threshold(p))), torch.zeros_like(v))


def _normed(v, kind, weight, bias):
    """(the norm of v's rows, mean, rstd)."""
    if kind == "none":
        return v, None, None
    mean = v.mean(dim=1) if kind == "layer" else None
    d = v if mean is None else v - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(dim=1) + EPS)
    y = d * rstd[:, None] * weight.float()
    return (y if bias is None else y + bias.float()), mean, rstd


def _normed_backward(dy, v, kind, weight, mean, rstd):
    """(gradient of v, of the weight, of the bias) of _normed."""
    if kind == "none":
        return dy, None, None
    vh = (v if mean is None else v - mean[:, None]) * rstd[:, None]
    h = dy * weight.float()
    g = h - vh * (h * vh).mean(dim=1, keepdim=True)
    if mean is not None:
        g = g - h.mean(dim=1, keepdim=True)
    return (rstd[:, None] * g, (dy * vh).sum(dim=0),
            dy.sum(dim=0) if mean is not None else None)


def _named(names, values):
    return {n: v for n, v in zip(names, values) if v is not None}


def _plain_join(s, dt):
    case = s["case"]
    v, post_mean, post_rstd = _normed(s["branch"].float(), case["post"], s["post_weight"],
                                      s["post_bias"])
    v = _dropped(v, s)
    if s["gate"] is not None:
        v = v * s["gate"].float()
    r = case["scale"] * s["x"].float() + v
    h, mean, rstd = _normed(r, case["pre"], s["pre_weight"], s["pre_bias"])
    out = {"r": r.to(dt)}
    if case["pre"] != "none":
        out["h"] = h.to(dt)
    return out | _named(("post_mean", "post_rstd", "mean", "rstd"),
                        (post_mean, post_rstd, mean, rstd))


def _plain_join_backward(s, dt):
    case = s["case"]
    post_mean, post_rstd, mean, rstd = s["stats"]
    t, dw, db = s["dr"].float(), None, None
    if case["pre"] != "none":
        g, dw, db = _normed_backward(s["dh"].float(), s["r"].float(), case["pre"],
                                     s["pre_weight"], mean, rstd)
        t = t + g
    b = s["branch"].float()
    dv = _dropped(t, s)
    dgate = None
    if s["gate"] is not None:
        v = b
        if case["post"] != "none":
            v = (b if post_mean is None else b - post_mean[:, None]) * post_rstd[:, None]
            v = v * s["post_weight"].float()
            if s["post_bias"] is not None:
                v = v + s["post_bias"].float()
        dgate = (dv * v).sum(dim=0)
        dv = dv * s["gate"].float()
    dbranch, dpw, dpb = _normed_backward(dv, b, case["post"], s["post_weight"], post_mean,
                                         post_rstd)
    out = _named(("dx", "dbranch", "dgate", "dpost_weight", "dpost_bias", "dpre_weight",
                  "dpre_bias"), (case["scale"] * t, dbranch, dgate, dpw, dpb, dw, db))
    return {n: v.to(dt) for n, v in out.items()}


def _plain(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    op = case["op"]
    if op == "dropout":
        y = _dropped(s["x"].float(), s)
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(dt)}
    if op == "residual_norm":
        return _plain_join(s, dt)
    if op == "residual_norm_backward":
        return _plain_join_backward(s, dt)
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    if op == "gated_linear":
        x = s["x"].float()
        g, u = x @ wg, x @ wu
        if s["bias_gate"] is not None:
            g, u = g + s["bias_gate"].float(), u + s["bias_up"].float()
        out = {"y": (_act(g, case["act"]) * u).to(dt)}
        if case["save"]:
            out["g"] = _decode(*_encode(g, _limit(dt))).to(dt)
            out["u"] = _decode(*_encode(u, _limit(dt))).to(dt)
        return out
    g, u = (_whole(t) for t in s["kept"])
    dy, x = s["dy"].float(), _whole(s["x"])
    dg, du = dy * u * _act_slope(g, case["act"]), dy * _act(g, case["act"])
    return {"dx": (dg @ wg.t() + du @ wu.t()).to(dt), "dw_gate": (x.t() @ dg).to(dt),
            "dw_up": (x.t() @ du).to(dt), "dbias_gate": dg.sum(dim=0).to(dt),
            "dbias_up": du.sum(dim=0).to(dt)}


# ------------------------------------------------- the package's operators
def _own(s):
    import bit_exact_matrix_amd as mm

    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    op = case["op"]

    def saved(v):
        return mm.Checkpoint(v[0], v[1], dt) if isinstance(v, tuple) else v

    if op == "dropout":
        return {"y": mm.dropout(s["x"], case["p"], s["seed"], s["offset"],
                                residual=s["residual"])}
    if op in ("residual_norm", "residual_norm_backward"):
        params = mm.ResidualParams(s["gate"], s["post_weight"], s["post_bias"], s["pre_weight"],
                                   s["pre_bias"])
        how = dict(post=None if case["post"] == "none" else case["post"],
                   pre=None if case["pre"] == "none" else case["pre"], scale=case["scale"],
                   dropout=case["p"], seed=s["seed"], offset=s["offset"])
        if op == "residual_norm":
            r, h, stats = mm.residual_norm(s["x"], s["branch"], params, eps=EPS, **how)
            return _named(("r", "h", "post_mean", "post_rstd", "mean", "rstd"), (r, h, *stats))
        dx, dbranch, grads = mm.residual_norm_backward(
            s["dr"], s["dh"], s["r"], s["branch"], params, mm.ResidualStats(*s["stats"]), **how)
        return _named(("dx", "dbranch", "dgate", "dpost_weight", "dpost_bias", "dpre_weight",
                       "dpre_bias"), (dx, dbranch, *grads))
    if op == "gated_linear":
        y, kept = mm.gated_linear(s["x"], s["w_gate"], s["w_up"], s["bias_gate"], s["bias_up"],
                                  activation=case["act"],
                                  keep="checkpoint" if case["save"] else None)
        out = {"y": y}
        if case["save"]:
            out["g"], out["u"] = mm.restore(kept[0]), mm.restore(kept[1])
        return out
    kept = saved(s["kept"][0]), saved(s["kept"][1])
    grads = mm.gated_linear_backward(s["dy"], saved(s["x"]), s["w_gate"], s["w_up"], kept,
                                     activation=case["act"])
    return dict(zip(("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up"), grads))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the work
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op in ("dropout", "residual_norm", "residual_norm_backward"):
        r, c = case["rows"], case["cols"]
        # ten rounds of two products and four exclusive ors for eight elements
        draws = 8 * r * c if case["p"] else 0
        if op == "dropout":
            return {"bytes": r * c * e * (3 if case["residual"] else 2), "flops": 2 * r * c + draws}
        vectors = (int(case["gate"]) + sum((case[s] != "none") + (case[s] == "layer")
                                           for s in ("post", "pre")))
        stats = 4 * r * sum((case[s] != "none") + (case[s] == "layer") for s in ("post", "pre"))
        if op == "residual_norm":
            n = 4 if case["pre"] != "none" else 3
            return {"bytes": n * r * c * e + vectors * c * e + stats, "flops": 16 * r * c + draws}
        n = 3 + (2 if case["pre"] != "none" else 0)  # dr, dx, dbranch; dh and r
        n += 1 if case["gate"] or case["post"] != "none" else 0  # the branch
        return {"bytes": n * r * c * e + 2 * vectors * c * e + stats, "flops": 30 * r * c + draws}
    m, n, k = case["m"], case["n"], case["k"]
    packed = 2 * m * (n + -(-n // BLOCK))  # two checkpoints of m x n
    if op == "gated_linear":
        b = m * k + 2 * k * n + m * n + (2 * n if case["bias"] else 0)
        # saved, and read again by the caller that looks at their values
        z = 2 * packed + 2 * m * n * e if case["save"] else 0
        return {"bytes": b * e + z, "flops": 4 * m * n * k + 12 * m * n}
    x = m * (k + -(-k // BLOCK)) if case["saved"] else m * k * e
    z = packed if case["saved"] else 2 * m * n * e
    return {"bytes": x + z + (m * n + 4 * k * n + m * k + 2 * n) * e,
            "flops": 8 * m * n * k + 30 * m * n}


# --------------------------------------------------------- float64, on its own
def _mask64(rows, cols, p, seed, offset):
    """Element by element from the definition, in numpy's unsigned integers."""
    mask = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    col = np.arange(-(-cols // 8), dtype=np.uint64)
    count = (np.arange(rows, dtype=np.uint64)[:, None] * np.uint64(2 ** 24) + col[None, :]).ravel()
    x = [count & mask, count >> half, np.full_like(count, offset & 0xFFFFFFFF),
         np.full_like(count, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(p1 >> half) ^ x[1] ^ np.uint64(key[0]), p1 & mask,
             (p0 >> half) ^ x[3] ^ np.uint64(key[1]), p0 & mask]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.empty((count.size, 8), dtype=np.uint16)
    for i in range(8):
        bits[:, i] = (x[i // 2] >> np.uint64(16 * (i % 2))).astype(np.uint16)
    keep = bits.reshape(rows, -1)[:, :cols].astype(np.int32) >= _threshold(p)
    return torch.from_numpy(np.ascontiguousarray(keep)).cuda()


def _drop64(v, case, s):
    if case["p"] == 0.0:
        return v
    keep = _mask64(*v.shape, case["p"], s["seed"], s["offset"])
    return torch.where(keep, v * 65536.0 / (65536 - _threshold(case["p"])), torch.zeros_like(v))


def _norm64(v, kind, weight, bias):
    if kind == "none":
        return v, None, None
    mean = torch.sum(v, 1) / v.shape[1] if kind == "layer" else None
    d = v - mean[:, None] if kind == "layer" else v
    rstd = 1.0 / torch.sqrt(torch.sum(d * d, 1) / v.shape[1] + EPS)
    y = weight.double() * (d * rstd[:, None])
    if bias is not None:
        y += bias.double()
    return y, mean, rstd


def _join64(case, x, s):
    """(r, h, statistics) of residual_norm."""
    v, pm, pr = _norm64(s["branch"].double(), case["post"], s["post_weight"], s["post_bias"])
    v = _drop64(v, case, s)
    r = x.double() * case["scale"] + (v if s["gate"] is None else s["gate"].double() * v)
    h, m, q = _norm64(r, case["pre"], s["pre_weight"], s["pre_bias"])
    return r, h, (pm, pr, m, q)


def _exact_values(x):
    """The matrix, or what a checkpoint stands for."""
    if not isinstance(x, tuple):
        return x.double()
    codes, scales = x
    step = torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=1)
    return codes.double() * step[:, : codes.shape[1]]


def _gate64(z, name):
    """(activation, slope) in float64, by other forms than the plain ones."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.maximum(z, torch.zeros_like(z)), torch.where(z > 0, 1.0, 0.0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * torch.sigmoid(-z)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    t = c * (z + 0.044715 * z ** 3)
    sg = torch.sigmoid(t)
    return z * sg, sg + z * sg * torch.sigmoid(-t) * c * (1.0 + 3 * 0.044715 * z * z)


def _unnorm64(dy, v, kind, weight, mean, rstd):
    if kind == "none":
        return dy, None, None
    n = v.shape[1]
    vh = (v - mean.double()[:, None] if kind == "layer" else v) * rstd.double()[:, None]
    w = weight.double()
    g = dy * w - vh * (((dy * vh) @ w)[:, None] / n)
    if kind == "layer":
        g -= (dy @ w)[:, None] / n
    return (g * rstd.double()[:, None], torch.sum(dy * vh, 0),
            torch.sum(dy, 0) if kind == "layer" else None)


def _exact_join_backward(case, s):
    pm, pr, m, q = s["stats"]
    t, dw, db = s["dr"].double(), None, None
    if case["pre"] != "none":
        g, dw, db = _unnorm64(s["dh"].double(), s["r"].double(), case["pre"], s["pre_weight"], m, q)
        t = t + g
    b = s["branch"].double()
    dv, dgate = _drop64(t, case, s), None
    if s["gate"] is not None:
        v = b
        if case["post"] != "none":
            vh = (b if pm is None else b - pm.double()[:, None]) * pr.double()[:, None]
            v = vh * s["post_weight"].double()
            if s["post_bias"] is not None:
                v += s["post_bias"].double()
        dgate = torch.sum(dv * v, 0)
        dv = dv * s["gate"].double()
    dbranch, dpw, dpb = _unnorm64(dv, b, case["post"], s["post_weight"], pm, pr)
    return _named(("dx", "dbranch", "dgate", "dpost_weight", "dpost_bias", "dpre_weight",
                   "dpre_bias"), (case["scale"] * t, dbranch, dgate, dpw, dpb, dw, db))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        y = _drop64(s["x"].double(), case, s)
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    if op == "residual_norm":
        r, h, stats = _join64(case, s["x"], s)
        out = {"r": r}
        if case["pre"] != "none":
            out["h"] = h
        return out | _named(("post_mean", "post_rstd", "mean", "rstd"), stats)
    if op == "residual_norm_backward":
        return _exact_join_backward(case, s)
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    if op == "gated_linear":
        x = s["x"].double()
        g, u = torch.mm(x, wg), torch.mm(x, wu)
        if s["bias_gate"] is not None:
            g += s["bias_gate"].double()
            u += s["bias_up"].double()
        out = {"y": _gate64(g, case["act"])[0] * u}
        # rounding to 8 bits is a step function: no value to compare with
        return out | {"g": None, "u": None} if case["save"] else out
    g, u = (_exact_values(t) for t in s["kept"])
    x, dy = _exact_values(s["x"]), s["dy"].double()
    a, slope = _gate64(g, case["act"])
    dg, du = dy * slope * u, dy * a
    return {"dx": torch.addmm(torch.mm(dg, wg.t()), du, wu.t()), "dw_gate": torch.mm(x.t(), dg),
            "dw_up": torch.mm(x.t(), du), "dbias_gate": torch.sum(dg, 0),
            "dbias_up": torch.sum(du, 0)}
