"""A training step of a feed-forward block, replayed for an audit.

    h = layer_norm(x);  a = gelu(h w1 + b1);  y = a w2 + b2 + x

The forward pass runs on the native operators and leaves 8-bit checkpoints
of x, of the pre-activation h w1 + b1 and of a; the backward pass uses them
(and makes h again from the checkpoint of x).  The gated block, from the sum of
the stream and the block before it to the sum behind it,

    r, h = x + branch, rms(x + branch);  a = silu(h wg) * (h wu)
    y = drop(a) wd;  r2 = r + gate drop(rms(y)), h2 = rms(r2)

leaves checkpoints of h, of both projections and of a; its dropout masks are
not kept but made again, from the seed, in the backward pass as in the replay.
Two things are then checked:

  repeats     the step run twice gives the same bits everywhere, in what it
              saves as in its output and gradients: the forward/recompute comparison of the AEGIS
              chapter ("Redundancy already exists in the training
              computation"), which a provider's step must pass too
  emulated    sampled rows of the first product, emulated as a Hopper or
              Ampere GPU computes it, beside the native product: how far
              the card's own arithmetic is from the one that is audited
              (the emulated rows are what mma_verify_gemm compares with);
              of the gated block, both projections, and a made of them

    python -m bit_exact_matrix_amd.replay --rows 4096 --dim 1024 --hidden 4096
    python -m bit_exact_matrix_amd.replay --block gated --dropout 0.1
"""
from __future__ import annotations

import argparse
import json
from typing import NamedTuple

from . import block as blk
from . import gemm, ops


class Block(NamedTuple):
    """Parameters: norm weight and bias (dim), w1 dim x hidden, b1 (hidden),
    w2 hidden x dim, b2 (dim)."""
    norm_w: object
    norm_b: object
    w1: object
    b1: object
    w2: object
    b2: object


class Saved(NamedTuple):
    """What the forward pass leaves for the backward pass."""
    x: ops.Checkpoint
    mean: object
    rstd: object
    z: ops.Checkpoint
    a: ops.Checkpoint


def forward(x, p: Block):
    """(y, Saved) of the block on x (rows x dim, float16 or bfloat16)."""
    h, mean, rstd, xs = ops.layer_norm(x, p.norm_w, p.norm_b, checkpoint=True)
    a, zs = ops.linear(h, p.w1, p.b1, activation="gelu", keep="checkpoint")
    y, _ = ops.linear(a, p.w2, p.b2, residual=x)
    return y, Saved(xs, mean, rstd, zs, ops.checkpoint(a))


def backward(dy, s: Saved, p: Block):
    """(dx, Block of the parameters' gradients) from dy and what was saved."""
    h, _, _, _ = ops.layer_norm(ops.restore(s.x), p.norm_w, p.norm_b)
    da, dw2, db2 = ops.linear_backward(dy, s.a, p.w2)
    dh, dw1, db1 = ops.linear_backward(da, h, p.w1, s.z, activation="gelu")
    dx, dnw, dnb = ops.layer_norm_backward(dh, s.x, p.norm_w, s.mean, s.rstd)
    return dx + dy, Block(dnw, dnb, dw1, db1, dw2, db2)


def emulated_rows(x, p: Block, rows, model="hopper"):
    """Rows of h w1 + b1 (float32) as the emulated GPU computes the product,
    and of the native product of the step: over all rows, for the number of
    rows chooses the kernel and the order of its sums."""
    import torch
    h, _, _, _ = ops.layer_norm(x, p.norm_w, p.norm_b)
    native, _ = ops.linear(h, p.w1, p.b1, out_dtype=torch.float32)
    c = p.b1.float().expand(len(rows), -1).contiguous()
    dtype = "bf16" if x.dtype == torch.bfloat16 else "fp16"
    d, _ = gemm(model, dtype, h[rows].contiguous().view(torch.int16),
                p.w1.contiguous().view(torch.int16), c)
    return d, native[rows]


class GatedBlock(NamedTuple):
    """Parameters: norm_w (dim) before the block, w_gate and w_up dim x hidden,
    w_down hidden x dim; gate and post_w (dim) of the sum behind it, next_w (dim)
    of the norm before the next block."""
    norm_w: object
    w_gate: object
    w_up: object
    w_down: object
    gate: object
    post_w: object
    next_w: object


class GatedSaved(NamedTuple):
    """What the gated block's forward pass leaves for its backward pass: the
    stream at both ends, the statistics, y, and checkpoints."""
    r: object
    stats: blk.ResidualStats
    h: ops.Checkpoint
    g: ops.Checkpoint
    u: ops.Checkpoint
    a: ops.Checkpoint
    y: object
    r2: object
    stats2: blk.ResidualStats


# the offsets of a step's two masks
_INSIDE, _BEHIND = 0, 1


def _ends(p: GatedBlock):
    """The vectors of the sums before and behind the block."""
    return (blk.ResidualParams(pre_weight=p.norm_w),
            blk.ResidualParams(gate=p.gate, post_weight=p.post_w, pre_weight=p.next_w))


def gated_forward(x, branch, p: GatedBlock, drop=0.0, seed=0):
    """(r2, h2, GatedSaved) of the gated block on the stream x and the output of
    the block before it (rows x dim, float16 or bfloat16)."""
    before, behind = _ends(p)
    r, h, stats = blk.residual_norm(x, branch, before, pre="rms")
    a, (g, u) = blk.gated_linear(h, p.w_gate, p.w_up, keep="checkpoint")
    y, _ = ops.linear(blk.dropout(a, drop, seed, _INSIDE), p.w_down)
    r2, h2, stats2 = blk.residual_norm(r, y, behind, post="rms", pre="rms", dropout=drop,
                                       seed=seed, offset=_BEHIND)
    return r2, h2, GatedSaved(r, stats, ops.checkpoint(h), g, u, ops.checkpoint(a), y, r2, stats2)


def gated_backward(dr, dh, s: GatedSaved, p: GatedBlock, drop=0.0, seed=0):
    """(dx, dbranch, GatedBlock of the parameters' gradients) from the gradients
    of r2 and h2 and what was saved."""
    before, behind = _ends(p)
    dr, dy, ends = blk.residual_norm_backward(
        dr, dh, s.r2, s.y, behind, s.stats2, post="rms", pre="rms", dropout=drop, seed=seed,
        offset=_BEHIND)
    a = blk.dropout(ops.restore(s.a), drop, seed, _INSIDE)
    da, dwd, _ = ops.linear_backward(dy, a, p.w_down, need_dbias=False)
    da = blk.dropout_backward(da, drop, seed, _INSIDE)
    dh, dwg, dwu, _, _ = blk.gated_linear_backward(da, s.h, p.w_gate, p.w_up, (s.g, s.u),
                                                   need_dbias=False)
    dx, dbranch, first = blk.residual_norm_backward(dr, dh, s.r, None, before, s.stats, pre="rms")
    return dx, dbranch, GatedBlock(first.pre_weight, dwg, dwu, dwd, ends.gate, ends.post_weight,
                                   ends.pre_weight)


def emulated_gate(x, branch, p: GatedBlock, rows, model="hopper"):
    """Rows of silu(h wg) * (h wu) in float32, with both products as the emulated
    GPU computes them, and of the step's own: over all rows, for their number
    chooses the kernel and the order of its sums."""
    import torch
    _, h, _ = blk.residual_norm(x, branch, _ends(p)[0], pre="rms")
    native, _ = blk.gated_linear(h, p.w_gate, p.w_up, out_dtype=torch.float32)
    dtype = "bf16" if x.dtype == torch.bfloat16 else "fp16"
    g, u = (gemm(model, dtype, h[rows].contiguous().view(torch.int16),
                 w.contiguous().view(torch.int16))[0] for w in (p.w_gate, p.w_up))
    return torch.nn.functional.silu(g) * u, native[rows]


def _flat(values):
    """The tensors of a tuple of tensors, Checkpoints and tuples of them."""
    for v in values:
        if isinstance(v, ops.Checkpoint):
            yield from v[:2]
        elif isinstance(v, tuple):
            yield from _flat(v)
        elif v is not None:
            yield v


def outputs(y, s: Saved, dx, grads: Block):
    """Every tensor that a step leaves."""
    return [y, dx, *grads, *_flat(s)]


def gated_outputs(r2, h2, s: GatedSaved, dx, dbranch, grads: GatedBlock):
    """Every tensor that a step of the gated block leaves (r2 is among what it
    saves)."""
    return [h2, dx, dbranch, *grads, *_flat(s)]


def same_bits(a, b):
    """Whether two tensors are the same word for word: a zero of the other
    sign differs, a NaN does not."""
    import torch
    word = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.dtype == b.dtype and torch.equal(a.contiguous().view(word), b.contiguous().view(word))


def _normal(dtype, seed, device):
    import torch
    g = torch.Generator(device=device).manual_seed(seed)

    def n(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=g, device=device)).to(dtype)

    return n


def make(rows, dim, hidden, dtype, seed=0, device="cuda"):
    """A block of random parameters, an input and a gradient of its output."""
    n = _normal(dtype, seed, device)
    p = Block(1 + n(dim, scale=0.1), n(dim, scale=0.1), n(dim, hidden, scale=dim ** -0.5),
              n(hidden, scale=0.1), n(hidden, dim, scale=hidden ** -0.5), n(dim, scale=0.1))
    return p, n(rows, dim), n(rows, dim)


def make_gated(rows, dim, hidden, dtype, seed=0, device="cuda"):
    """A gated block of random parameters, a stream, the output of the block
    before it, and gradients of r2 and h2."""
    n = _normal(dtype, seed, device)
    p = GatedBlock(1 + n(dim, scale=0.1), n(dim, hidden, scale=dim ** -0.5),
                   n(dim, hidden, scale=dim ** -0.5), n(hidden, dim, scale=hidden ** -0.5),
                   0.5 + n(dim, scale=0.1), 1 + n(dim, scale=0.1), 1 + n(dim, scale=0.1))
    return p, n(rows, dim), n(rows, dim), n(rows, dim), n(rows, dim)


def replay_gated(rows=4096, dim=1024, hidden=4096, dtype="bf16", model="hopper", seed=0,
                 dropout=0.1):
    """replay of the gated block."""
    import torch
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    p, x, branch, dr, dh = make_gated(rows, dim, hidden, dt, seed)
    mask = seed % 2 ** 64  # torch's generators take negative seeds, dropout does not
    runs = []
    for _ in range(2):
        r2, h2, saved = gated_forward(x, branch, p, dropout, mask)
        back = gated_backward(dr, dh, saved, p, dropout, mask)
        runs.append(gated_outputs(r2, h2, saved, *back))
    same = all(same_bits(a, b) for a, b in zip(*runs))
    sample = torch.linspace(0, rows - 1, min(rows, 16), device=x.device).long()
    emulated, native = emulated_gate(x, branch, p, sample, model)
    kept = [saved.h, saved.g, saved.u, saved.a]
    return {"rows": rows, "dim": dim, "hidden": hidden, "dtype": dtype, "model": model,
            "block": "gated", "dropout": dropout, "repeats": same,
            "emulated_relative_difference":
                float((emulated - native).norm() / native.norm().clamp(min=1e-30)),
            "saved_bytes": sum(c.codes.numel() + c.scales.numel() for c in kept),
            "whole_bytes": sum(c.codes.numel() * x.element_size() for c in kept),
            "mask_bytes": 0}


def replay(rows=4096, dim=1024, hidden=4096, dtype="bf16", model="hopper", seed=0):
    """Runs the step twice and emulates 16 rows; the findings as a dict."""
    import torch
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    p, x, dy = make(rows, dim, hidden, dt, seed)
    runs = []
    for _ in range(2):
        y, saved = forward(x, p)
        dx, grads = backward(dy, saved, p)
        runs.append(outputs(y, saved, dx, grads))
    same = all(same_bits(a, b) for a, b in zip(*runs))
    sample = torch.linspace(0, rows - 1, min(rows, 16), device=x.device).long()
    emulated, native = emulated_rows(x, p, sample, model)
    kept = [saved.x, saved.z, saved.a]
    return {"rows": rows, "dim": dim, "hidden": hidden, "dtype": dtype, "model": model,
            "repeats": same,
            "emulated_relative_difference":
                float((emulated - native).norm() / native.norm().clamp(min=1e-30)),
            "saved_bytes": sum(c.codes.numel() + c.scales.numel() for c in kept),
            "whole_bytes": sum(c.codes.numel() * x.element_size() for c in kept)}


def main():
    ap = argparse.ArgumentParser(description="replay a feed-forward block's training step")
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--dtype", choices=["bf16", "fp16"], default="bf16")
    ap.add_argument("--model", choices=["ampere", "hopper"], default="hopper")
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--block", choices=["plain", "gated"], default="plain")
    ap.add_argument("--dropout", type=float, default=None,
                    help="of the gated block (0.1 unless given)")
    args = vars(ap.parse_args())
    gated, drop = args.pop("block") == "gated", args.pop("dropout")
    if drop is not None and not gated:
        ap.error("--dropout is of the gated block")
    if gated:
        found = replay_gated(**args, dropout=0.1 if drop is None else drop)
    else:
        found = replay(**args)
    print(json.dumps(found), flush=True)


if __name__ == "__main__":
    main()
