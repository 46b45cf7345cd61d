"""Plain 64-bit implementation of the 8-bit key/value cache (numpy, CPU), and
the inputs its tests share.  The e4m3 grid is built from its definition: 1
sign, 4 exponent (bias 7) and 3 mantissa bits, 0x7f and 0xff NaN."""
import math

import numpy as np
import torch

EXP_LO, EXP_HI = -48, 48


def e4m3_values():
    """Value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[c] = math.nan if c & 0x7f == 0x7f else -x if c & 0x80 else x
    return out


E4M3 = e4m3_values()
_GRID = E4M3[:0x7f]  # the non-negative values, ascending


def encode(x):
    """Codes of x (float64): nearest, ties to the even code, saturated; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=448.0), 448.0)
    hi = np.searchsorted(_GRID, a)           # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _GRID[hi] - a, a - _GRID[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(_GRID[hi] == a, hi, pick)
    code = pick | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7f, code).astype(np.uint8)


def needed_exp(a):
    """The smallest e with a <= 448 * 2^e within the range."""
    if a == 0:
        return EXP_LO
    e = math.floor(math.log2(a / 448.0)) - 1
    while a > math.ldexp(448.0, e):
        e += 1
    return min(EXP_HI, max(EXP_LO, e))


class Cache:
    """codes k, v uint8 [pages][H][P][D], scales float64 [pages][H]."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v = k.copy(), v.copy()
        self.ks, self.vs = ks.astype(np.float64), vs.astype(np.float64)

    def side(self, s):
        return (self.k, self.ks) if s == "k" else (self.v, self.vs)

    def write(self, table, kv_len, num_new, k_new, v_new):
        P = self.k.shape[2]
        for name, new in (("k", k_new), ("v", v_new)):
            codes, scale = self.side(name)
            for b in range(table.shape[0]):
                at, n = int(kv_len[b]), int(num_new[b])
                for slot in range(at // P, (at + n - 1) // P + 1 if n else 0):
                    lo, hi = max(at, slot * P), min(at + n, (slot + 1) * P)
                    page, kept = table[b, slot], max(0, at - slot * P)
                    for h in range(codes.shape[1]):
                        x = new[b, lo - at:hi - at, h].astype(np.float64)
                        f = np.abs(x[np.isfinite(x)])
                        e = needed_exp(f.max() if f.size else 0.0)
                        if kept:
                            old = scale[page, h]
                            e = max(e, int(math.log2(old)))
                            s = math.ldexp(1.0, e)
                            if s > old:
                                codes[page, h, :kept] = encode(
                                    E4M3[codes[page, h, :kept]] * (old / s))
                        s = math.ldexp(1.0, e)
                        scale[page, h] = s
                        codes[page, h, lo - slot * P:hi - slot * P] = encode(x / s)

    def values(self, side, table_row, positions):
        codes, scale = self.side(side)
        P = codes.shape[2]
        pos = np.asarray(positions, np.int64)
        page = table_row[pos // P]
        return E4M3[codes[page, :, pos % P]] * scale[page][:, :, None]  # [n][H][D]


def attention(q, cache, table, kv_len, num_new, mask, scale):
    """(out, lse, spread, xerr) in float64: spread [B][T][Hq][D] is the
    weighted mean of |v|, xerr [B][T][Hq] the largest sum |q k| scale, which
    the tolerances are made of.  mask: bool [B][T][T] or None (causal)."""
    B, T, Hq, D = q.shape
    H = cache.k.shape[1]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse, xerr = np.full((B, T, Hq), -np.inf), np.zeros((B, T, Hq))
    for b in range(B):
        n, at = int(num_new[b]), int(kv_len[b])
        if n == 0:
            continue
        k, v = (cache.values(s, table[b], np.arange(at + n)) for s in "kv")
        for t in range(n):
            see = np.ones(at + n, bool)
            see[at:] = (np.arange(n) <= t) if mask is None else mask[b, t, :n]
            if not see.any():
                continue
            for j in range(Hq):
                h = j * H // Hq
                x = k[see, h] @ q[b, t, j] * scale
                xerr[b, t, j] = (np.abs(k[see, h]) @ np.abs(q[b, t, j])).max() * abs(scale)
                m = x.max()
                w = np.exp(x - m)
                lse[b, t, j] = m + np.log(w.sum())
                w /= w.sum()
                out[b, t, j] = w @ v[see, h]
                spread[b, t, j] = w @ np.abs(v[see, h])
    return out, lse, spread, xerr


def out_bounds(out, spread, xerr, D, dtype):
    """How far the kernel's out and lse may be off.  x: at most D roundings of
    products and sums in 32 bits, and the exponential's own 2^-21; the weights
    are rounded to fp16 (2^-11) for the second product, whose sums add less
    than 2^-12; the result is rounded once."""
    dx = D * 2.0 ** -24 * xerr + 2.0 ** -21
    half = torch.finfo(dtype).eps / 2
    d = spread * (2.0 ** -11 + 2.0 ** -12 + 2 * dx[..., None])
    return d + half * (np.abs(out) + d) + 2.0 ** -24, dx


# ------------------------------------------------------------------ inputs

def random_cache(rng, pages, H, P, D, spread=1.0):
    """A cache whose pages have scales between 2^-3 and 2^3 of each other."""
    k, v = (encode(rng.normal(size=(pages, H, P, D)) * 100.0 * spread) for _ in "kv")
    ks, vs = (2.0 ** rng.integers(-10, -4, (pages, H)) for _ in "kv")
    return Cache(k, v, ks, vs)


def tables(rng, pages, lens, P, slots=None):
    """Random disjoint page tables for `lens` tokens a request (-1 beyond)."""
    need = [-(-int(x) // P) for x in lens]
    assert sum(need) <= pages
    order = rng.permutation(pages).astype(np.int32)
    out = np.full((len(need), slots or max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        out[b, :n] = order[at:at + n]
        at += n
    return out


def to_device(cache, split=None):
    """The cache as the library takes it.  split "interleaved": k and v of a
    page side by side in one buffer; "heads": heads with a gap between them."""
    k, v = torch.from_numpy(cache.k).cuda(), torch.from_numpy(cache.v).cuda()
    pages, H, P, D = cache.k.shape
    if split == "interleaved":
        both = torch.empty((pages, 2, H, P, D), dtype=torch.uint8, device="cuda")
        both[:, 0], both[:, 1] = k, v
        k, v = both[:, 0], both[:, 1]
    elif split == "heads":
        wide = torch.full((2, pages, H, P + 1, D), 0x7f, dtype=torch.uint8, device="cuda")
        wide[0, :, :, :P], wide[1, :, :, :P] = k, v
        k, v = wide[0, :, :, :P], wide[1, :, :, :P]
    return dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn),
                k_scale=torch.from_numpy(cache.ks.astype(np.float32)).cuda(),
                v_scale=torch.from_numpy(cache.vs.astype(np.float32)).cuda())


def from_device(c):
    return (c["k"].view(torch.uint8).cpu().numpy(), c["v"].view(torch.uint8).cpu().numpy(),
            c["k_scale"].cpu().numpy(), c["v_scale"].cpu().numpy())


def mask_words(mask, words=None):
    """bool [B][T][T] as rows of 32-bit words (int32 storage)."""
    B, T, _ = mask.shape
    words = words or (T + 31) // 32
    out = np.zeros((B, T, words), np.uint32)
    for j in range(T):
        out[:, :, j // 32] |= mask[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def random_tree_mask(rng, B, T):
    m = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(T):
            if i:
                m[b, i] = m[b, rng.integers(max(0, i - 4), i)]
            m[b, i, i] = True
    return m
