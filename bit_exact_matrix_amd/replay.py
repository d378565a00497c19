"""A training step of one feed-forward block, replayed for an audit.

    h = layer_norm(x);  a = gelu(h w1 + b1);  y = a w2 + b2 + x

The forward pass runs on the native operators and leaves 8-bit checkpoints
of x, of the pre-activation h w1 + b1 and of a; the backward pass uses them
(and makes h again from the checkpoint of x).  Two things are then checked:

  repeats     the step run twice gives the same bits everywhere, in what it
              saves as in its output and gradients: the forward/recompute comparison of the AEGIS
              chapter ("Redundancy already exists in the training
              computation"), which a provider's step must pass too
  emulated    sampled rows of the first product, emulated as a Hopper or
              Ampere GPU computes it, beside the native product: how far
              the card's own arithmetic is from the one that is audited
              (the emulated rows are what mma_verify_gemm compares with)

    python -m bit_exact_matrix_amd.replay --rows 4096 --dim 1024 --hidden 4096
"""
from __future__ import annotations

import argparse
import json
from typing import NamedTuple

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


def outputs(y, s: Saved, dx, grads: Block):
    """Every tensor that a step leaves."""
    saved = [t for part in s for t in (part[:2] if isinstance(part, ops.Checkpoint) else (part,))]
    return [y, dx, *grads, *saved]


def same_bits(a, b):
    """Whether two tensors are the same word for word: a zero of the other
    sign differs, a NaN does not."""
    import torch
    word = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.dtype == b.dtype and torch.equal(a.contiguous().view(word), b.contiguous().view(word))


def make(rows, dim, hidden, dtype, seed=0, device="cuda"):
    """A block of random parameters, an input and a gradient of its output."""
    import torch
    g = torch.Generator(device=device).manual_seed(seed)

    def n(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=g, device=device)).to(dtype)

    p = Block(1 + n(dim, scale=0.1), n(dim, scale=0.1), n(dim, hidden, scale=dim ** -0.5),
              n(hidden, scale=0.1), n(hidden, dim, scale=hidden ** -0.5), n(dim, scale=0.1))
    return p, n(rows, dim), n(rows, dim)


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
    print(json.dumps(replay(**vars(ap.parse_args()))), flush=True)


if __name__ == "__main__":
    main()
