"""What the bound of tests/cache_exact.py tells apart, on the host: weights of two fp16 numbers are within it, weights rounded to
one are not."""
import numpy as np
import pytest

from tests import cache_exact as ex, cache_ref as ref


def worst(b, Q, scale, weights):
    want, tol = ex.attend(b, Q, scale)
    got, _ = ex.attend(b, Q, scale, weights=weights)
    return (np.abs(got.astype(np.float16).astype(np.float64) - want) / tol).max()


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("D", [64, 256])
def test_weights_of_two_halves_are_told_from_rounded_ones(D, fmt):
    for i, (new, lens, heads, G) in enumerate((ex.FEW + ex.MANY)[1:]):
        rng = np.random.default_rng([60, D, fmt, i])
        b = ex.batch(rng, new, lens, heads, D, 16, fmt)
        Q = ex.queries(rng, b, heads * G)
        assert worst(b, Q, D ** -0.5, ex.twice) <= 1
        assert worst(b, Q, D ** -0.5, ex.once) > 1.5 and worst(b, Q, D ** -0.5, ex.once_above) > 1.5


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_flat_weights_that_are_no_fp16_numbers(fmt):
    rng = np.random.default_rng([61, fmt])
    for n, L in ((1, 300), (5, 1037)):
        b = ex.flat(rng, n, L, fmt)
        Q = ex.queries(rng, b, 2)
        assert worst(b, Q, 0.0, ex.twice) <= 1 and worst(b, Q, 0.0, ex.once_above) > 1


def test_the_bound_goes_by_the_same_definition():
    rng = np.random.default_rng(62)
    b = ref.Batch(rng, [3, 9], [30, 50], 2, 64, 16, ref.E4M3)
    Q = rng.standard_normal((12, 4, 64)).astype(np.float16)
    for window, sinks in ((0, 0), (7, 3)):
        want, _, live = b.attend(Q, 0.125, window, sinks)
        assert live.all() and np.allclose(ex.attend(b, Q, 0.125, window, sinks)[0], want, rtol=1e-12, atol=1e-14)
