"""Definitions of the heads' and the 8-bit cache's operators in float64 on the host (test infrastructure, not product code)."""
import numpy as np

import bit_mixed_precision_tri_amd as tri

INT8, E4M3 = tri.TRI_KV_INT8, tri.TRI_KV_E4M3
TOP = {INT8: 127.0, E4M3: 448.0}


def values_of(fmt):
    """What the 256 codes stand for."""
    b = np.arange(256)
    if fmt == INT8:
        return b.astype(np.uint8).view(np.int8).astype(np.float64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where(b & 128, -v, v)


def codes_of(x, fmt):
    """The code nearest to every value, ties to the even one; values within the largest code."""
    if fmt == INT8:
        return np.rint(x).astype(np.int8).view(np.uint8)
    mag = values_of(E4M3)[:127]                  # (0x7F is no number)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mag, a), 1, 126)
    lo = hi - 1
    dl, dh = a - mag[lo], mag[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need_scale(most, fmt):
    """The least power of two, 2^-30 or more, times which the largest code reaches `most`."""
    e = np.full(np.shape(most), -30)
    while np.any(most > TOP[fmt] * 2.0 ** e):
        e = np.where(most > TOP[fmt] * 2.0 ** e, e + 1, e)
    return 2.0 ** e


def rotate(x, pos, table, interleaved=False, norm=True, eps=1e-5, gain=None):
    """(T, heads, D) float64 -> (results, the magnitude that their errors go by)."""
    y = x.astype(np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if gain is not None:
            y = y * gain.astype(np.float64)
    out, mag = y.copy(), np.abs(y)
    if table is not None:
        cs = table.astype(np.float64)[pos][:, None]
        c, s, half = cs[..., 0], cs[..., 1], table.shape[1]
        ia = np.arange(half) * 2 if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return out, mag


class Batch:
    """A cache and a batch of sequences on the host."""

    def __init__(self, rng, new, lens, heads, D, page, fmt, spare=2, width=None, codes=True):
        self.new, self.lens, self.heads, self.D, self.page, self.fmt = list(new), list(lens), heads, D, page, fmt
        B = len(new)
        need = [-(-max(x, 0) // page) for x in lens]
        self.width = max(max(need), 1) if width is None else width
        need = [min(x, self.width) for x in need]
        total = sum(need) + spare
        ids = rng.permutation(total)
        self.table = np.full((B, self.width), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.offsets[-1])
        hi = 256 if codes else 1
        self.K = rng.integers(0, hi, (total, heads, page, D)).astype(np.uint8)
        self.V = rng.integers(0, hi, (total, heads, D, page)).astype(np.uint8)
        if fmt == E4M3 and codes:                # small numbers, most of them, none that is no number
            for x in (self.K, self.V):
                x[(x & 127) > 0x70] ^= 0x40
        if fmt == INT8:
            self.K[self.K == 128] = 0
            self.V[self.V == 128] = 0
        base = 1 / 64.0 if fmt == INT8 else 1 / 16.0
        self.ks = (base * 2.0 ** rng.integers(-3, 2, (total, heads))).astype(np.float32)
        self.vs = (base * 2.0 ** rng.integers(-3, 2, (total, heads))).astype(np.float32)

    def on_gpu(self, max_new=None, max_len=None):
        from tests.gpu_helpers import cuda
        cache = tri.KVCache(cuda(self.K), cuda(self.V), cuda(self.ks), cuda(self.vs), self.fmt)
        seqs = tri.Sequences(cuda(self.offsets), cuda(np.asarray(self.lens, dtype=np.int32)), cuda(self.table),
                             max_new=max(max(self.new), 1) if max_new is None else max_new, max_len=max_len)
        return cache, seqs

    def place(self, b, p):
        """The page and place of position p; None: there is none."""
        i = p // self.page
        if p < 0 or i >= self.width or not 0 <= self.table[b, i] < len(self.K):
            return None
        return int(self.table[b, i]), p % self.page

    def append(self, K, V, rows=None, max_new=1 << 30):
        """What the cache holds after the call, in place; rows: positions that the rotation's table has."""
        vals = values_of(self.fmt)
        for b in range(len(self.new)):
            n = self.new[b]
            pages = {}
            for i in range(min(n, max_new)):
                p = max(self.lens[b], 0) - n + i
                at = self.place(b, p)
                if at is None or (rows is not None and p >= rows):
                    continue
                pages.setdefault(at[0], []).append((at[1], int(self.offsets[b]) + i))
            for page, put in pages.items():
                first = put[0][0]
                places, src = [x for x, _ in put], [t for _, t in put]
                for X, C, S in ((K, self.K, self.ks), (V, self.V, self.vs)):
                    x = X[src].astype(np.float64)          # (tokens, heads, D)
                    x = np.where(np.isnan(x), np.copysign(0.0, x), np.clip(x, -65504.0, 65504.0))
                    for h in range(self.heads):
                        c = C[page, h] if C is self.K else C[page, h].T        # (page, D), a view
                        need = np.float32(need_scale(np.abs(x[:, h]).max(), self.fmt))
                        was = np.float32(S[page, h])
                        if first == 0 or not was >= need:
                            inv = np.float32(1) / need
                            if first > 0:
                                c[:first] = codes_of(vals[c[:first]] * float(was * inv), self.fmt)
                            S[page, h] = need
                        else:
                            inv = np.float32(1) / was
                        c[places] = codes_of(x[:, h] * float(inv), self.fmt)

    def attend(self, Q, scale, window=0, sinks=0, max_new=1 << 30):
        """Results (T, H, D), their tolerance, and which rows are written.

        A score is a sum of D exact products: inside a matrix instruction at most 32 additions, D/32 after them, each within
        2^-23 (a truncating adder); then a few roundings of fp32 and, in exp2 and log2, 2^-22.  A weight is rounded to
        fp16 (2^-11, or 2^-25 below 2^-14, the largest weight being 2^10); the sums are 32 + L/32 additions, and as many
        scalings as the maximum grows and waves and splits are joined (both sums alike)."""
        T, H, D = Q.shape
        G, vals = H // self.heads, values_of(self.fmt)
        out, tol, live = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros(T, dtype=bool)
        Q = Q.astype(np.float64)
        for b in range(len(self.new)):
            n, L = self.new[b], max(self.lens[b], 0)
            seen = [(j, self.place(b, j)) for j in range(L)]
            seen = [(j, a) for j, a in seen if a is not None]
            J = np.array([j for j, _ in seen], dtype=np.int64)
            pg, pl = np.array([a[0] for _, a in seen], dtype=np.int64), np.array([a[1] for _, a in seen], dtype=np.int64)
            for i in range(min(n, max_new)):
                t, p = int(self.offsets[b]) + i, L - n + i
                live[t] = True
                ok = J <= p
                if window > 0:
                    ok &= (J > p - window) | (J < sinks)
                if not ok.any():
                    tol[t] = 2.0 ** -24
                    continue
                for h in range(self.heads):
                    k = vals[self.K[pg[ok], h, pl[ok]]] * self.ks[pg[ok], h].astype(np.float64)[:, None]
                    c = vals[self.V[pg[ok], h, :, pl[ok]]]
                    u = self.vs[pg[ok], h].astype(np.float64)[:, None]
                    q = Q[t, h * G:(h + 1) * G]
                    x = scale * (q @ k.T)
                    m = x.max(1, keepdims=True)
                    w = np.exp(x - m)
                    w /= w.sum(1, keepdims=True)
                    o = w @ (c * u)
                    A = abs(scale) * (np.abs(q) @ np.abs(k).T)
                    lu = np.abs(np.log2(u)).max()
                    e = (A.max(1) * (40 + D / 32) * 2.0 ** -23 + (8 * 2.0 ** -24) * (3 * np.abs(x).max(1) + lu + 16) + 2.0 ** -20)[:, None]
                    rel = 2 * e + 2.0 ** -11 + (96 + len(J) / 8) * 2.0 ** -23
                    out[t, h * G:(h + 1) * G] = o
                    tol[t, h * G:(h + 1) * G] = (w @ np.abs(c * u)) * rel + 2.0 ** -11 * np.abs(o) + 2.0 ** -24 + \
                        2.0 ** -35 * u.max() * np.abs(c).sum(0)
        return out, tol, live
