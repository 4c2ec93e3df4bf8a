"""Attention over the 8-bit cache on the GPU against the bound of tests/cache_exact.py: results do not carry a rounding of single
weights to fp16, whatever the size of the call."""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests import cache_exact as ex, cache_ref as ref
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


def check(b, Q, scale=None, window=0, sinks=0, what=""):
    scale = b.D ** -0.5 if scale is None else scale
    cache, seqs = b.on_gpu()
    got = host(tri.cache_attend(cache, seqs, cuda(Q), scale=scale, window=window, sinks=sinks))
    want, tol = ex.attend(b, Q, float(np.float32(scale)), window, sinks)
    near(got, want, tol, what)
    return got


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("rows", ["few", "many"])
def test_weights_of_two_halves(rows, D, page, fmt):
    for i, (new, lens, heads, G) in enumerate(ex.FEW if rows == "few" else ex.MANY):
        rng = np.random.default_rng([60, D, fmt, i])
        b = ex.batch(rng, new, lens, heads, D, page, fmt)
        check(b, ex.queries(rng, b, heads * G), what=(new, lens, heads, G))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_of_two_halves_in_splits_and_many_tiles(D):
    """Tiles whose steps are split and joined, and more tiles than two groups of waves share, over a window and first tokens."""
    rng = np.random.default_rng([63, D])
    b = ex.batch(rng, [9], [4100], 1, D, 64, ref.INT8)
    check(b, ex.queries(rng, b, 4), what="splits")
    B = 70
    b = ex.batch(rng, [5] * B, [int(x) for x in rng.integers(5, 150, B)], 8, D, 16, ref.E4M3)
    check(b, ex.queries(rng, b, 64), window=70, sinks=3, what="tiles")


def test_the_same_row_in_calls_of_any_size():
    """A token's result alone, among a few and among many new tokens is within one bound."""
    rng = np.random.default_rng(64)
    b = ex.batch(rng, [40], [100], 1, 128, 16, ref.INT8)
    Q = ex.queries(rng, b, 4)
    want, tol = ex.attend(b, Q, float(np.float32(128 ** -0.5)))
    for n in (1, 3, 8, 9, 40):
        b.new, b.offsets = [n], np.array([0, n], dtype=np.int32)
        cache, seqs = b.on_gpu()
        near(host(tri.cache_attend(cache, seqs, cuda(Q[40 - n:]))), want[40 - n:], tol[40 - n:], n)


@pytest.mark.parametrize("n", [1, 20, 100])
def test_flat_weights_that_are_no_fp16_numbers(n):
    """Equal scores whose common weight fp16 does not hold: nothing of its rounding is left in the mean of the values."""
    for fmt in (ref.INT8, ref.E4M3):
        for L in (n + 200, n + 1000):
            rng = np.random.default_rng([65, n, L, fmt])
            b = ex.flat(rng, n, L, fmt)
            check(b, ex.queries(rng, b, 2), scale=0.0, what=(L, fmt))
