"""Attention over the 8-bit cache with scores that are far from zero: the largest queries, keys at the scale that fp16's largest
number gives them, scales of the scores to the ends of fp32.  There a score's own rounding is more than any weight's exponent, so
that a row is the value of its largest score, or the mean of those that have the same."""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests import cache_ref as ref
from tests.gpu_helpers import cuda, host
from tests.test_gpu_cache import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


def values(b, L):
    """(L, D): what the first L tokens' values stand for."""
    at = [b.place(0, j) for j in range(L)]
    pg, pl = np.array([a[0] for a in at]), np.array([a[1] for a in at])
    return ref.values_of(b.fmt)[b.V[pg, 0, :, pl]] * b.vs[pg, 0].astype(np.float64)[:, None]


def place_keys(b, codes):
    """Token j's key: codes[j] in the first dimension, zeros in the others."""
    b.K[:] = 0
    b.ks[:] = 512.0
    for j, c in enumerate(codes):
        pg, pl = b.place(0, j)
        b.K[pg, 0, pl, 0] = c


def attend(b, G, scale, q0=65504.0):
    n = b.new[0]
    Q = np.zeros((n, G, b.D), dtype=np.float16)
    Q[..., 0] = q0
    cache, seqs = b.on_gpu()
    return host(tri.cache_attend(cache, seqs, cuda(Q), scale=scale))


SCALES = [1.0, -1.0, 2.0 ** 14, -1e25, 1e25]


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("n", [1, 4, 12, 40])
def test_the_largest_of_far_scores(n, D, page, fmt):
    """Keys that all differ: the value of the largest score that is seen (exact in fp16, as scales are powers of two)."""
    rng = np.random.default_rng([70, n, D, fmt])
    vals = ref.values_of(fmt)
    own = np.array([c for c in range(256) if c not in (0x80, *((0x7F, 0xFF) if fmt == ref.E4M3 else ()))])
    L = 170
    for scale in SCALES:
        b = ref.Batch(rng, [n], [L], 1, D, page, fmt)
        codes = rng.permutation(own)[:L]
        place_keys(b, codes)
        got = attend(b, 3, scale)
        x, v = np.sign(scale) * vals[codes], values(b, L)
        for t in range(n):
            best = v[np.argmax(x[:L - n + t + 1])]
            near(got[t], np.repeat(best[None], 3, 0), 2.0 ** -11 * np.abs(best) + 2.0 ** -25, (scale, t))


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("n,L", [(1, 300), (1, 5000), (12, 300), (40, 300), (40, 5000)])
def test_far_scores_that_are_the_same(n, L, fmt):
    """Equal keys, and one that is twice as large: those who see it take its value, the others the mean of what they see."""
    rng = np.random.default_rng([71, n, L, fmt])
    one, two = (50, 100) if fmt == ref.INT8 else (0x48, 0x50)
    for scale in SCALES:
        for big in (None, L - n // 2 - 1, 5):
            b = ref.Batch(rng, [n], [L], 1, 64, 32, fmt)
            b.vs[:] = 0.25
            codes = np.full(L, one)
            if big is not None:
                codes[big] = two
            place_keys(b, codes)
            got, v = attend(b, 2, scale), values(b, L)
            for t in range(n):
                seen = np.arange(L - n + t + 1)
                if big is not None and big in seen:
                    seen = seen[seen == big] if scale > 0 else seen[seen != big]
                want, size = v[seen].mean(0), np.abs(v[seen]).mean(0)
                # equal weights and a denominator of them: L/8 + 64 additions of fp32 each
                tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + (64 + L / 8) * 2.0 ** -23 * size
                near(got[t], np.repeat(want[None], 2, 0), tol, (scale, big, t))


@pytest.mark.parametrize("n", [1, 5, 50])
def test_any_far_scores(n):
    """Queries and keys at random: never anything but a mean of the values that are seen, and the largest score's own value where
    the next one is further behind than the scores' fp32 sums may be off."""
    rng = np.random.default_rng([72, n])
    for fmt in (ref.INT8, ref.E4M3):
        for D, spread in ((64, 65504.0), (128, 900.0), (128, 30.0)):
            L = 200
            b = ref.Batch(rng, [n], [L], 1, D, 16, fmt)
            b.ks[:] = 512.0
            Q = (rng.uniform(-1, 1, (n, 2, D)) * spread).astype(np.float16)
            cache, seqs = b.on_gpu()
            got = host(tri.cache_attend(cache, seqs, cuda(Q))).astype(np.float64)
            at = [b.place(0, j) for j in range(L)]
            pg, pl = np.array([a[0] for a in at]), np.array([a[1] for a in at])
            k = ref.values_of(fmt)[b.K[pg, 0, pl]] * 512.0
            v = values(b, L)
            sure = 0
            for t in range(n):
                seen = L - n + t + 1
                for h in range(2):
                    q = Q[t, h].astype(np.float64)
                    x, A = D ** -0.5 * (k[:seen] @ q), D ** -0.5 * (np.abs(k[:seen]) @ np.abs(q)).max()
                    hi, lo = v[:seen].max(0), v[:seen].min(0)
                    slack = 2.0 ** -10 * np.maximum(np.abs(hi), np.abs(lo)) + 2.0 ** -24
                    assert np.all((got[t, h] <= hi + slack) & (got[t, h] >= lo - slack)), (fmt, D, t)
                    first, second = np.sort(x)[[-1, -2]]
                    if first - second > 2 * (48 * 2.0 ** -23) * A + 40:
                        sure += 1
                        best = v[np.argmax(x)]
                        near(got[t, h], best, 2.0 ** -11 * np.abs(best) + 2.0 ** -25, (fmt, D, t))
            assert sure > n


@pytest.mark.parametrize("n", [2, 6, 40])
def test_scores_past_fp32_spoil_only_their_rows(n):
    """Every other row's query is 0 (all its scores are 0): the mean of what it sees, whatever becomes of the rows beside it."""
    rng = np.random.default_rng([73, n])
    for fmt in (ref.INT8, ref.E4M3):
        for scale in (3e38, -3e38, 1e36):
            L = 100
            b = ref.Batch(rng, [n], [L], 1, 64, 16, fmt)
            b.ks[:] = 512.0
            Q = (rng.uniform(-1, 1, (n, 3, 64)) * 65504).astype(np.float16)
            Q[:, 1] = 0
            cache, seqs = b.on_gpu()
            got, v = host(tri.cache_attend(cache, seqs, cuda(Q), scale=scale)), values(b, L)
            for t in range(n):
                x = v[:L - n + t + 1]
                tol = 2.0 ** -11 * np.abs(x.mean(0)) + 2.0 ** -25 + (64 + L / 8) * 2.0 ** -23 * np.abs(x).mean(0)
                tol = tol + 2.0 ** -21 * np.abs(x).mean(0) + 2.0 ** -35 * np.abs(x).sum(0)    # weights of two fp16 numbers
                near(got[t, 1], x.mean(0), tol, (fmt, scale, t))
