"""The gated block's formulas in float64, and error bounds for results
computed with float32 sums and one rounding of the output (as in
ops_reference: U = 2^-24, a row or column sum has a depth of at most DEPTH)."""
import numpy as np
import torch

from ops_reference import DEPTH, ROUND, TINY, U  # noqa: F401


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
