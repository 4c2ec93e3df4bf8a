"""Heads and the 8-bit cache on the GPU: bounds and kernels that calls of other sizes do not reach."""
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


@pytest.mark.parametrize("n", [1, 3, 40])
def test_lengths_far_past_the_table(n):
    """A length that the table has no room for: what has a place is seen, and no time goes by the length (steps up to it would be
    33 million, seconds of a call)."""
    import torch
    rng = np.random.default_rng([80, n])
    for D, page, window, sinks in ((64, 16, 0, 0), (128, 64, 0, 0), (64, 16, 1000, 40), (64, 16, 2 ** 31 - 1, 0), (256, 128, 2 ** 31 - 300, 7)):
        b = ref.Batch(rng, [n, n], [5 * page] * 2, 1, D, page, ref.INT8)
        Q = rng.standard_normal((2 * n, 2, D)).astype(np.float16)
        cache, seqs = b.on_gpu(max_len=5 * page)
        wide = tri.Sequences(seqs.offsets, torch.full_like(seqs.lens, 2 ** 31 - 1), seqs.table, max_new=n, max_len=2 ** 31 - 200)
        tight = tri.Sequences(seqs.offsets, wide.lens, seqs.table, max_new=n, max_len=5 * page)
        # the same from nearer by: positions right behind the table with what is left of the window there, or a window behind it
        b.table, b.width = np.concatenate([b.table, np.full((2, 200), -1, dtype=np.int32)], 1), 205
        left = window - (2 ** 31 - 256 - n - 5 * page)
        b.lens = [5 * page + n + (window if left <= 0 else 0)] * 2
        want, tol = ex.attend(b, Q, float(np.float32(D ** -0.5)), left if left > 0 else window, sinks)
        for sq in (tight, wide):
            tri.cache_attend(cache, sq, cuda(Q), window=window, sinks=sinks)
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            q = cuda(Q)
            begin.record()
            got = tri.cache_attend(cache, sq, q, window=window, sinks=sinks)
            end.record()
            near(host(got), want, tol, (D, page, window))
            assert begin.elapsed_time(end) < 100, (D, page, window)
