"""The definition of attention over the 8-bit cache in float64, with a bound that holds weights to what two fp16 numbers hold
(test infrastructure, not product code)."""
import numpy as np

from tests import cache_ref as ref


def visible(b, i, p, window, sinks):
    """Pages and places of what position p of sequence i sees."""
    at = [b.place(i, j) for j in range(max(p + 1, 0)) if window == 0 or j > p - window or j < sinks]
    at = [x for x in at if x is not None]
    return np.array([x[0] for x in at], dtype=np.int64), np.array([x[1] for x in at], dtype=np.int64)


def attend(b, Q, scale, window=0, sinks=0, weights=None):
    """Results (T, H, D) and their tolerance.  weights: None, or what a kernel would make of the exact weights, which are 2^10 at
    the largest product with its value's scale, a function to (those of the values, those of the denominator).

    Scores: a sum of D exact products, at most 32 additions inside a matrix instruction and D/32 after them, each within 2^-23;
    the score's factor and the exponent's sum are three roundings of 2^-24 of them, exp2 and log2 within 2^-22.  Weights are
    the sum of two fp16 numbers, the first of them maybe truncated: 2^-10 of a weight, 2^-11 of what that leaves off, 2^-21
    together (of at most 2^-25, where the largest weight is 2^10 at least, nothing may be left: 2^-35).  The sums are 32 + L/8
    additions and scalings, both alike; the result is rounded to fp16."""
    T, H, D = Q.shape
    G, vals = H // b.heads, ref.values_of(b.fmt)
    out, tol = np.zeros((T, H, D)), np.full((T, H, D), 2.0 ** -25)
    for i, n in enumerate(b.new):
        for t in range(n):
            row, p = int(b.offsets[i]) + t, max(b.lens[i], 0) - n + t
            pg, pl = visible(b, i, p, window, sinks)
            if not len(pg):
                continue
            for h in range(b.heads):
                k = vals[b.K[pg, h, pl]] * b.ks[pg, h].astype(np.float64)[:, None]
                c, u = vals[b.V[pg, h, :, pl]], b.vs[pg, h].astype(np.float64)[:, None]
                q = Q[row, h * G:(h + 1) * G].astype(np.float64)
                x = scale * (q @ k.T)
                y = x / np.log(2) + np.log2(u).T
                w = 2.0 ** (y - y.max(1, keepdims=True) + 10)
                wv, wd = (w, w) if weights is None else weights(w)
                den = (wd / u.T).sum(1, keepdims=True)
                o = (wv @ c) / den
                A = abs(scale) * (np.abs(q) @ np.abs(k).T)
                lu = np.abs(np.log2(u)).max()
                e = A.max(1) * (36 + D / 32) * 2.0 ** -23 + 3 * 2.0 ** -24 * (np.abs(x).max(1) + lu + 10) + 2.0 ** -21
                rel = (2 * e + 2.0 ** -21 + (64 + len(pg) / 4) * 2.0 ** -23)[:, None]
                at = (row, slice(h * G, (h + 1) * G))
                out[at] = o
                tol[at] = (w @ np.abs(c)) / (w / u.T).sum(1, keepdims=True) * rel + 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + \
                    2.0 ** -35 * u.max() * np.abs(c).sum(0)
    return out, tol


def once(w):
    """Every weight rounded to one fp16, in both sums."""
    r = w.astype(np.float16).astype(np.float64)
    return r, r


def once_above(w):
    """Weights rounded to one fp16 over a denominator of unrounded ones."""
    return w.astype(np.float16).astype(np.float64), w


def twice(w):
    """Every weight as the sum of two fp16 numbers, the first truncated."""
    hi = w.astype(np.float16)
    hi = np.where(hi.astype(np.float64) > w, np.nextafter(hi, np.float16(0)), hi).astype(np.float64)
    return hi + (w - hi).astype(np.float16).astype(np.float64), w


def batch(rng, new, lens, heads, D, page, fmt, scale_steps=3):
    """Keys that make scores differ by little, values of one size and either sign: sums of weights cancel, roundings of single
    weights do not."""
    b = ref.Batch(rng, new, lens, heads, D, page, fmt)
    top = 100 if fmt == ref.INT8 else 0x58
    sign = rng.integers(0, 2, b.V.shape)
    b.V = (np.where(sign, 256 - top, top) if fmt == ref.INT8 else top + 128 * sign).astype(np.uint8)
    b.vs[:] = 2.0 ** -rng.integers(0, scale_steps, b.vs.shape)
    b.ks[:] = 2.0 ** -8 if fmt == ref.INT8 else 2.0 ** -6
    return b


def queries(rng, b, H):
    return (0.25 * rng.standard_normal((int(b.offsets[-1]), H, b.D))).astype(np.float16)


# new tokens, lengths, key/value heads, query heads of each: few rows of a head, tiles of many (with the steps shared by two
# groups of waves), many in one group
FEW = [([1], [3], 1, 4), ([2, 1], [9, 40], 2, 4), ([3], [7], 1, 8), ([4], [130], 1, 6)]
MANY = [([5], [7], 1, 8), ([5, 40], [12, 40], 2, 8), ([9], [130], 1, 4), ([1], [70], 1, 40)]


def flat(rng, n, L, fmt):
    """Equal scores (scale 0) and, in every dimension, equal values, but for the first four pages: zeros under a scale that makes
    all other weights 2^9 (1 + 0.98 * 2^-11), off by nearly half a step as one fp16."""
    b = ref.Batch(rng, [n], [L], 1, 64, 16, fmt)
    b.V[:] = (np.arange(64) + 60 if fmt == ref.INT8 else np.arange(64) % 24 + 0x40)[:, None]
    b.vs[:], b.ks[:] = 0.75, 0.01
    b.V[b.table[0, :4]] = 0
    b.vs[b.table[0, :4]] = 1.5 / (1 + 0.98 * 2.0 ** -11)
    return b
