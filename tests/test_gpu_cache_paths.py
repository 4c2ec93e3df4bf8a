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


def table_of(rows, dims):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, dims, 2) / dims)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


@pytest.mark.parametrize("D,sets,T", [(64, (33, 9), 1301), (64, (16, 5, 1), 2100), (128, (33, 9), 801), (128, (8, 1, 30, 3), 700),
                                      (256, (17, 2, 6), 700), (256, (32, 32), 300)])
def test_rotate_many_tokens(D, sets, T):
    """Calls of 4096 units of heads and more, where a wave takes two of them: odd numbers of units, units of two sets in one wave,
    rows apart, some outside the table; then in place."""
    import torch
    rng = np.random.default_rng([81, D, T])
    assert T * sum(-(-h * D // 1024) for h in sets) >= 4096
    rows, dims = 97, D // 2
    tab = table_of(rows, dims)
    x = rng.standard_normal((T, sum(sets) + 1, D)).astype(np.float16)
    at = np.concatenate([[0], np.cumsum(sets)])
    pos = rng.integers(-2, rows + 2, T).astype(np.int32)
    ok = (pos >= 0) & (pos < rows)
    gains = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float16) for _ in sets]
    gains[-1] = None
    for interleaved in (False, True):
        buf = cuda(x)
        views = [buf[:, at[i]:at[i + 1]] for i in range(len(sets))]
        r = tri.Rotary(cuda(tab), gains=[None if g is None else cuda(g) for g in gains], norm=True, interleaved=interleaved)
        out = [torch.full((T, h, D), float("nan"), dtype=torch.float16, device="cuda") for h in sets]
        tri.heads_rotate(views, r, cuda(pos), out=out)
        for i in range(len(sets)):
            want, mag = ref.rotate(x[:, at[i]:at[i + 1]], np.clip(pos, 0, rows - 1), tab, interleaved, True, float(np.float32(1e-5)), gains[i])
            got = host(out[i])
            assert np.isnan(got[~ok]).all()
            near(got[ok], want[ok], (32 * 2.0 ** -24 * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)[ok], (i, interleaved))
        tri.heads_rotate(views, r, cuda(pos), out=views)
        again = host(buf)
        for i in range(len(sets)):
            np.testing.assert_array_equal(again[ok, at[i]:at[i + 1]].view(np.uint16), host(out[i])[ok].view(np.uint16))
        np.testing.assert_array_equal(again[~ok].view(np.uint16), x[~ok].view(np.uint16))
        np.testing.assert_array_equal(again[:, -1].view(np.uint16), x[:, -1].view(np.uint16))


@pytest.mark.parametrize("D,page,dims,interleaved", [(64, 32, 16, False), (128, 16, 48, False), (128, 128, 64, True), (256, 32, 128, False), (256, 64, 240, True)])
def test_append_with_partial_rotation(D, page, dims, interleaved):
    """Keys of which only the first values turn, appended: codes and scales as of rotation and appending in two calls."""
    rng = np.random.default_rng([82, D, dims])
    tab = cuda(table_of(200, dims))
    for norm in (True, False):
        gains = [cuda((1 + 0.3 * rng.standard_normal(D)).astype(np.float16)) for _ in range(2)]
        r = tri.Rotary(tab, gains=gains, norm=norm, interleaved=interleaved)
        for new, lens in [([1, 1], [7, 150]), ([9, 140, 1], [60, 150, 33])]:
            b = ref.Batch(rng, new, lens, 3, D, page, ref.INT8)
            K, V, Q = (rng.standard_normal((b.T, h, D)).astype(np.float16) for h in (3, 3, 6))
            pos = np.concatenate([np.arange(l - n, l) for n, l in zip(new, lens)]).astype(np.int32)
            q2, k2 = tri.heads_rotate((cuda(Q), cuda(K)), r, cuda(pos))
            cache, seqs = b.on_gpu()
            q = tri.cache_append(cache, seqs, cuda(K), cuda(V), rotary=r, Q=cuda(Q))
            b.append(host(k2), V)
            for got, want in ((cache.K, b.K), (cache.V, b.V), (cache.K_scale, b.ks), (cache.V_scale, b.vs), (q, host(q2))):
                np.testing.assert_array_equal(host(got), want, err_msg=str((norm, new)))


def test_append_in_several_launches_with_queries():
    """max_new of thousands for sequences of one token each (more pieces than a launch takes): codes, scales and queries as with
    max_new of one."""
    import torch
    rng = np.random.default_rng(83)
    B, heads, H, D, page = 3000, 4, 6, 64, 16
    assert B * ((B + page - 2) // page + 1) * 2 * heads > 1 << 21
    K, V, Q = (cuda(rng.standard_normal((B, h, D)).astype(np.float16)) for h in (heads, heads, H))
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, lens = torch.arange(B + 1, **i32), torch.randint(1, page + 1, (B,), **i32)
    table = torch.randperm(B, device="cuda").to(torch.int32)[:, None].contiguous()
    r = tri.Rotary(cuda(table_of(page, D)))
    got = []
    for most in (B, 1):
        cache = tri.KVCache.empty(B, heads, D, page, ref.E4M3)
        q = tri.cache_append(cache, tri.Sequences(offsets, lens, table, max_new=most), K, V, rotary=r, Q=Q)
        got.append([host(x) for x in (cache.K, cache.V, cache.K_scale, cache.V_scale, q)])
    for x, y in zip(*got):
        np.testing.assert_array_equal(x, y)
    want = tri.heads_rotate((Q,), r, lens - 1)[0]
    np.testing.assert_array_equal(got[0][4].view(np.uint16), host(want).view(np.uint16))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,page,window,sinks", [(ref.E4M3, 128, 70, 3), (ref.INT8, 128, 0, 0), (ref.E4M3, 16, 0, 0), (ref.INT8, 16, 33, 130),
                                                   (ref.E4M3, 64, 100, 4), (ref.INT8, 32, 1, 0)])
def test_attend_many_rows_in_many_tiles_of_any_pages(D, fmt, page, window, sinks):
    """More tiles than two per CU, over pages shorter and longer than a step, with and without a window."""
    rng = np.random.default_rng([84, D, fmt, page])
    B = 70
    b = ref.Batch(rng, [5] * B, [int(x) for x in rng.integers(5, 300, B)], 8, D, page, fmt)
    Q = rng.standard_normal((5 * B, 64, D)).astype(np.float16)
    cache, seqs = b.on_gpu()
    got = host(tri.cache_attend(cache, seqs, cuda(Q), window=window, sinks=sinks))
    want, tol = ex.attend(b, Q, float(np.float32(D ** -0.5)), window, sinks)
    near(got, want, tol)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("D,G", [(64, 40), (64, 64), (128, 33), (128, 64), (256, 48), (128, 130)])
def test_attend_one_token_of_many_heads_per_key(D, G, fmt):
    """Single tokens with more than 32 query heads of a key/value head, whose steps are shared by workgroups and joined."""
    rng = np.random.default_rng([85, D, G, fmt])
    for lens, window in (([3000, 70], 0), ([1], 0), ([5000], 2000)):
        b = ref.Batch(rng, [1] * len(lens), lens, 1, D, 64, fmt)
        Q = rng.standard_normal((len(lens), G, D)).astype(np.float16)
        cache, seqs = b.on_gpu()
        got = host(tri.cache_attend(cache, seqs, cuda(Q), window=window, sinks=4))
        want, tol = ex.attend(b, Q, float(np.float32(D ** -0.5)), window, 4)
        near(got, want, tol, lens)
