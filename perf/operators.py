"""The measured cases of the native training operators, with their plain forms.

The operators stand next to the emulated GEMM in a program that replays and
audits a training or serving step on one MI355X: the layer norm before a
product, the product itself with its epilogue, the 8-bit checkpoints that a
forward pass leaves for the backward pass, and both backward passes.

  layer_norm           y = (x - mu) rstd w + b for each row, with mu and rstd
                       in float32; with `save`, the 8-bit checkpoint of x too
  layer_norm_backward  dx, dw and db from dy and x (or x's checkpoint)
  linear               y = act(x W + b) + r, z = x W + b; with `save`, the
                       8-bit checkpoint of z too
  linear_backward      dz = dy act'(z), db = sum over rows of dz, dx = dz W^T,
                       dW = x^T dz; x and z whole, or as 8-bit checkpoints
  checkpoint           x to 8 bits and back

A checkpoint holds E4M3 codes (OCP "FN") and one power of two for each 32
consecutive elements of a row: the smallest 2^e, -117 <= e <= 120, with
max |x| <= 448 * 2^e over the block's finite elements.

Where `own` is false, `run` computes the plain form: elementary torch
operations in float32, rounded once at the end.  Where it is true, it calls
the package's operators.  `exact` computes the same in float64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32


def listed():
    return [
        # one token of a decoding step through a block's first layer norm
        dict(name="norm_token", op="layer_norm", rows=1, cols=4096, dtype="bf16", save=False),
        # a training batch: the layer norm also leaves the checkpoint of its input
        dict(name="norm_train", op="layer_norm", rows=8192, cols=4096, dtype="bf16", save=True),
        # the backward pass of that batch
        dict(name="norm_back", op="layer_norm_backward", rows=8192, cols=4096, dtype="bf16",
             saved=False),
        # backward from the checkpoint: odd row count, a width off the vector sizes
        dict(name="norm_back_saved", op="layer_norm_backward", rows=4097, cols=1000,
             dtype="fp32", saved=True),
        # one token through a square projection: the weight is read once
        dict(name="linear_token", op="linear", m=1, n=4096, k=4096, dtype="bf16", act="silu",
             layout="kn", residual=True, save=False),
        # a few tokens against a wide output, weight stored with a row for each output
        dict(name="linear_narrow", op="linear", m=16, n=50000, k=4096, dtype="fp16", act="none",
             layout="nk", residual=False, save=False),
        # the square product of the emulator's own benchmark, whole epilogue
        dict(name="linear_square", op="linear", m=4096, n=4096, k=4096, dtype="bf16", act="gelu",
             layout="kn", residual=True, save=False),
        # odd sizes, and the checkpoint of the pre-activation beside the output
        dict(name="linear_ragged", op="linear", m=1999, n=1499, k=1024, dtype="fp16", act="gelu",
             layout="kn", residual=False, save=True),
        # a training step's backward pass from 8-bit checkpoints
        dict(name="linear_back_saved", op="linear_backward", m=4096, n=4096, k=4096,
             dtype="bf16", act="gelu", layout="kn", saved=True),
        # a small backward pass with odd sizes, from whole activations
        dict(name="linear_back_small", op="linear_backward", m=299, n=260, k=640, dtype="fp16",
             act="silu", layout="nk", saved=False),
        # the checkpoint of a training batch, written and used
        dict(name="checkpoint_batch", op="checkpoint", rows=8192, cols=4096, dtype="bf16"),
        # a small ragged checkpoint: the last block of each row is a part of one
        dict(name="checkpoint_ragged", op="checkpoint", rows=70, cols=1499, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi], even over its logarithm; half of the larger ones are multiples of 320."""
    v = _log(rng, lo, hi)
    return v // 320 * 320 if v >= 320 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "linear", "linear", "linear_backward",
                     "checkpoint"])
    if op in ("layer_norm", "layer_norm_backward", "checkpoint"):
        cols = _size(rng, 33, 16384)
        rows = _size(rng, 1, max(1, min(65536, 8192 * 4096 // 2 // cols)))
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        if op == "layer_norm":
            case["save"] = rng.random() < 0.5
        if op == "layer_norm_backward":
            case["saved"] = rng.random() < 0.5
        return case
    # 4 M N K of the backward pass stays below the largest listed one
    k = _size(rng, 48, 8192)
    n = _size(rng, 48, 50000 if op == "linear" else 8192)
    m = _size(rng, 1, max(1, min(8192, 4096 ** 3 // 2 // (n * k))))
    case = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "fp16"]),
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                layout=rng.choice(["kn", "nk"]))
    if op == "linear":
        case["residual"] = rng.random() < 0.5
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
    """(codes as float8, scale exponents + 127) of float32 x, in float32."""
    p = _blocks(x)
    mag = p.abs()
    mag = torch.where(torch.isfinite(p), mag, torch.zeros_like(mag)).clamp(max=limit)
    f, e = torch.frexp(mag.amax(dim=2))
    e = (e - 9 + (f > 0.875)).clamp(-117, 120)
    e = torch.where(f == 0, torch.full_like(e, -117), e)
    v = torch.ldexp(torch.copysign(mag, p), -e.unsqueeze(2))
    v = torch.where(torch.isfinite(p), v, torch.full_like(v, math.nan))
    codes = v.to(torch.float8_e4m3fn).view(x.shape[0], -1)[:, : x.shape[1]].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _decode(codes, scales):
    """The float32 values of a checkpoint."""
    v = _blocks(codes.float())
    v = torch.ldexp(v, (scales.to(torch.int32) - 127).unsqueeze(2))
    return v.view(codes.shape[0], -1)[:, : codes.shape[1]]


def _limit(dtype):
    return 61440.0 if dtype == torch.float16 else 1.875 * 2.0 ** 127


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] in ("layer_norm", "layer_norm_backward", "checkpoint"):
        x = _activations(g, case["rows"], case["cols"], dt)
        if case["op"] == "checkpoint":
            s["x"] = x
            return s
        s["weight"] = (1.0 + 0.2 * normal(case["cols"])).to(dt)
        if case["op"] == "layer_norm":
            s["x"] = x
            s["bias"] = (0.2 * normal(case["cols"])).to(dt)
            return s
        s["dy"] = normal(case["rows"], case["cols"]).to(dt)
        xf = x.double()
        mean = xf.mean(dim=1)
        var = (xf - mean[:, None]).square().mean(dim=1)
        s["mean"], s["rstd"] = mean.float(), (var + 1e-5).rsqrt().float()
        s["x"] = _encode(x.float(), _limit(dt)) if case["saved"] else x
        return s
    m, n, k = case["m"], case["n"], case["k"]
    x = _activations(g, m, k, dt)
    w = (normal(k, n) * (0.7 / math.sqrt(k))).to(dt)
    s["w"] = w if case["layout"] == "kn" else w.t().contiguous().t()
    if case["op"] == "linear":
        s["x"] = x
        s["bias"] = (0.2 * normal(n)).to(dt)
        s["residual"] = _activations(g, m, n, dt) if case["residual"] else None
        return s
    s["dy"] = normal(m, n).to(dt)
    z = (1.5 * normal(m, n)).to(dt) if case["act"] != "none" else None
    if case["saved"]:
        s["x"] = _encode(x.float(), _limit(dt))
        s["z"] = _encode(z.float(), _limit(dt)) if z is not None else None
    else:
        s["x"], s["z"] = x, z
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


def _plain(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    op = case["op"]
    if op == "checkpoint":
        return {"x": _decode(*_encode(s["x"].float(), _limit(dt))).to(dt)}
    if op == "layer_norm":
        x = s["x"].float()
        mean = x.mean(dim=1)
        d = x - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(dim=1) + 1e-5)
        out = {"y": (d * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt),
               "mean": mean, "rstd": rstd}
        if case["save"]:
            out["codes"], out["scales"] = _encode(x, _limit(dt))
        return out
    if op == "layer_norm_backward":
        xh = (_whole(s["x"]) - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        h = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (h - h.mean(dim=1, keepdim=True)
                                   - xh * (h * xh).mean(dim=1, keepdim=True))
        return {"dx": dx.to(dt), "dweight": (dy * xh).sum(dim=0).to(dt),
                "dbias": dy.sum(dim=0).to(dt)}
    w = s["w"].float()
    if op == "linear":
        z = s["x"].float() @ w + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(dt)}
        if case["save"]:
            out["z"] = _decode(*_encode(z, _limit(dt))).to(dt)
        return out
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(_whole(s["z"]), case["act"])
    x = _whole(s["x"])
    return {"dx": (dz @ w.t()).to(dt), "dw": (x.t() @ dz).to(dt), "dbias": dz.sum(dim=0).to(dt)}


# ------------------------------------------------- the package's operators
def _own(s):
    import bit_exact_matrix_amd as mm

    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    op = case["op"]

    def saved(v):
        return mm.Checkpoint(v[0], v[1], dt) if isinstance(v, tuple) else v

    if op == "checkpoint":
        return {"x": mm.restore(mm.checkpoint(s["x"]))}
    if op == "layer_norm":
        y, mean, rstd, ck = mm.layer_norm(s["x"], s["weight"], s["bias"], eps=1e-5,
                                          checkpoint=case["save"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if ck is not None:
            out["codes"], out["scales"] = ck.codes, ck.scales
        return out
    if op == "layer_norm_backward":
        dx, dw, db = mm.layer_norm_backward(s["dy"], saved(s["x"]), s["weight"], s["mean"],
                                            s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "linear":
        y, z = mm.linear(s["x"], s["w"], s["bias"], activation=case["act"],
                         residual=s["residual"], keep="checkpoint" if case["save"] else None)
        return {"y": y, "z": mm.restore(z)} if case["save"] else {"y": y}
    dx, dw, db = mm.linear_backward(s["dy"], saved(s["x"]), s["w"], saved(s["z"]),
                                    activation=case["act"])
    return {"dx": dx, "dw": dw, "dbias": db}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the work
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op in ("layer_norm", "layer_norm_backward", "checkpoint"):
        r, c = case["rows"], case["cols"]
        n, saved = r * c, r * (c + -(-c // BLOCK))
        if op == "checkpoint":
            return {"bytes": 2 * n * e + 2 * saved, "flops": 4 * n}
        if op == "layer_norm":
            return {"bytes": 2 * n * e + 2 * c * e + 8 * r + (saved if case["save"] else 0),
                    "flops": 8 * n}
        return {"bytes": 2 * n * e + (saved if case["saved"] else n * e) + 3 * c * e + 8 * r,
                "flops": 15 * n}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        b = m * k + k * n + n + m * n * (2 if case["residual"] else 1)
        z = 2 * m * (n + -(-n // BLOCK)) + m * n * e if case["save"] else 0
        return {"bytes": b * e + z, "flops": 2 * m * n * k + 10 * m * n}
    x = m * (k + -(-k // BLOCK)) if case["saved"] else m * k * e
    z = 0 if case["act"] == "none" else m * (n + -(-n // BLOCK)) if case["saved"] else m * n * e
    return {"bytes": x + z + (m * n + 2 * k * n + m * k + n) * e, "flops": 4 * m * n * k}


# --------------------------------------------------------- float64, on its own
def _exact_codes(x, top):
    """(the E4M3 values, scale exponents + 127) by rounding on the grid."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    p = torch.nn.functional.pad(x, (0, pad)).view(rows, -1, BLOCK)
    ok = torch.isfinite(p)
    p = torch.where(ok, p.clamp(-top, top), torch.zeros_like(p))
    big = p.abs().amax(dim=2)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 448.0))
    e = torch.where(big > 448.0 * torch.exp2(e), e + 1, e)          # log2's own rounding
    e = torch.where(big <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(big > 0, e, torch.full_like(e, -117.0)).clamp(-117, 120)
    v = p / torch.exp2(e).unsqueeze(2)
    mag = v.abs()
    lead = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    lead = torch.where(mag >= torch.exp2(lead + 1), lead + 1, lead)
    step = torch.exp2(lead.clamp(min=-6) - 3)
    v = torch.round(v / step) * step
    v = torch.where(ok, v, torch.full_like(v, math.nan))
    return v, e


def _exact_values(v, e, cols):
    return (v * torch.exp2(e).unsqueeze(2)).reshape(v.shape[0], -1)[:, :cols]


def _exact_whole(v):
    if not isinstance(v, tuple):
        return v.double()
    codes, scales = v
    step = torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=1)
    return codes.double() * step[:, : codes.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    top = _limit(DTYPES[case["dtype"]])
    if op == "checkpoint":
        x = s["x"].double()
        return {"x": _exact_values(*_exact_codes(x, top), x.shape[1])}
    if op == "layer_norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + 1e-5)
        y = (x - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double()
        out = {"y": y, "mean": mean, "rstd": rstd}
        if case["save"]:
            v, e = _exact_codes(x, top)
            out["codes"] = v.reshape(x.shape[0], -1)[:, : x.shape[1]]
            out["scales"] = (e + 127).to(torch.uint8)
        return out
    if op == "layer_norm_backward":
        r = s["rstd"].double()[:, None]
        x, dy, w = _exact_whole(s["x"]), s["dy"].double(), s["weight"].double()
        n = x.shape[1]
        xh = (x - s["mean"].double()[:, None]) * r
        p = (dy @ w)[:, None] / n
        q = ((dy * xh) @ w)[:, None] / n
        return {"dx": r * (dy * w - p - xh * q), "dweight": torch.sum(dy * xh, 0),
                "dbias": torch.sum(dy, 0)}
    w = s["w"].double()

    def cdf(t):
        return 0.5 * torch.special.erfc(-t / math.sqrt(2.0))

    def inner(t):
        return 2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)

    if op == "linear":
        z = torch.addmm(s["bias"].double(), s["x"].double(), w)
        y = {"none": lambda t: t, "relu": lambda t: torch.maximum(t, torch.zeros_like(t)),
             "silu": lambda t: t * torch.sigmoid(t), "gelu": lambda t: t * cdf(t),
             "gelu_tanh": lambda t: t * torch.sigmoid(inner(t))}[case["act"]](z)
        if s["residual"] is not None:
            y += s["residual"].double()
        # rounding z to 8 bits is a step function of z: no value to compare with
        return {"y": y, "z": None} if case["save"] else {"y": y}
    dz = s["dy"].double()
    if s["z"] is not None:
        z = _exact_whole(s["z"])
        if case["act"] == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif case["act"] == "silu":
            sg = torch.sigmoid(z)
            dz = dz * (sg + z * sg * torch.sigmoid(-z))
        elif case["act"] == "gelu":
            dz = dz * (cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        else:
            sg = torch.sigmoid(inner(z))
            slope = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * z * z)
            dz = dz * (sg + z * sg * torch.sigmoid(-inner(z)) * slope)
    return {"dx": dz @ w.t(), "dw": _exact_whole(s["x"]).t() @ dz, "dbias": torch.sum(dz, 0)}
