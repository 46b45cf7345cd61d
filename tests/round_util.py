"""Plain 64-bit implementations of the norms and rotations of queries and keys
and of the log probabilities (numpy, CPU), with how far the kernels may be off."""
import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rotated(x, pos, rope, weight=None, eps=None):
    """(y, size) in float64: x [B][T][H][D] normed and turned; pos [B][T] whole
    numbers; size, which the tolerances are made of: the sum of a channel's pair's
    magnitudes (its own where it does not turn)."""
    y = x.astype(np.float64)
    D = x.shape[-1]
    if eps is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps)))
        if weight is not None:
            y = y * weight
    size = np.abs(y)
    if rope is None:
        return y, size
    dim, scale = rope["dim"], float(np.float32(rope["scale"]))
    freq = rope["freq"].cpu().tolist()
    B, T = len(pos), len(pos[0])
    turn = np.array([[[(int(pos[b][t]) * f % (1 << 64)) / 2.0 ** 64 for f in freq]
                      for t in range(T)] for b in range(B)])[:, :, None]
    c, s = np.cos(2 * np.pi * turn) * scale, np.sin(2 * np.pi * turn) * scale
    if rope["interleaved"]:
        i, j = np.arange(0, dim, 2), np.arange(1, dim, 2)
    else:
        i, j = np.arange(dim // 2), np.arange(dim // 2, dim)
    u, v = y[..., i], y[..., j]
    y[..., i], y[..., j] = u * c - v * s, v * c + u * s
    size[..., i] = size[..., j] = (np.abs(u) + np.abs(v)) * abs(scale)
    assert D >= dim
    return y, size


def rotation_bound(size):
    """How far 32-bit results may be off.  The norm: a sum of D squares (chains of
    16 and four shuffles: 20 roundings, of which the root halves the effect),
    mean, eps, root, quotient and two products, 16 * 2^-24.  The turn: half turns
    rounded to 24 bits (pi 2^-25), sine and cosine (2^-23), their scale (2^-24),
    two products and a sum (2^-23): 7 * 2^-24.  Together below 2^-19."""
    return size * 2.0 ** -19


def rounding(dtype, y, off):
    """... and rounded once to dtype."""
    t = TYPES[dtype]
    return off + torch.finfo(t).eps / 2 * (np.abs(y) + off) + float(
        torch.finfo(t).smallest_normal) * torch.finfo(t).eps


def positions(start, offset, B, T):
    return [[int(start[b] if start is not None else 0) +
             int(offset[b][t] if offset is not None else t) for t in range(T)] for b in range(B)]


# ------------------------------------------------------- log probabilities

class Row:
    """One row of logits (float64 values of the stored ones) at temperature t."""

    def __init__(self, x, t=1.0):
        t = float(np.float32(t)) or 1.0
        self.x, self.t = x, t
        self.m = x.max()
        with np.errstate(invalid="ignore"):
            d = (x - self.m) / t
        w = np.exp(d)
        z = w.sum()
        self.log_z = math.log(z)
        self.lp = d - self.log_z
        some = w > 0
        self.spread = float((w[some] * -d[some]).sum() / z)   # mean distance to the maximum
        self.entropy = self.log_z + self.spread

    def bounds(self):
        """(of log probabilities [V], of the entropy).  A weight: its exponent has
        three roundings (2^-24 each of itself), ex2 is off by 2^-22 of the result,
        and at most eight times on its way to the row's sum the reference rises
        (2^-22 and three roundings of the rise, which are less than the
        exponent's own).  The sum: at most 64 roundings on the way.  So Z is off
        by (36 + 64 + 12 + 6 spread) 2^-24 of itself; the logarithm and the
        differences add three roundings of what they are made of."""
        z = (112 + 6 * self.spread) * 2.0 ** -24
        with np.errstate(invalid="ignore"):
            d = np.abs(self.x - self.m) / self.t
        lp = z + 4 * 2.0 ** -24 * (d + abs(self.log_z))
        # the mean exponent: Z's errors once more, relative to it
        h = z * (1 + 2 * self.spread) + 8 * 2.0 ** -24 * (abs(self.log_z) + self.spread)
        return np.where(np.isfinite(lp), lp, 0.0), h

    def top(self, n):
        """Ids of the n largest, lower ids first among equals, without -inf."""
        order = np.lexsort((np.arange(len(self.x)), -self.x))[:n]
        return order[self.x[order] > -np.inf]
