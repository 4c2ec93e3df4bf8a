"""Heads and the 8-bit cache on the GPU against their definitions in float64 (tests/cache_ref.py): norm and rotation, appending
bit for bit, attention within a bound that counts its roundings, and a decoder's steps with all of them together.

Tolerance of a normalised and rotated value: the sum of squares is 16 fused steps and at most 4 additions, the mean, the added
eps, root, division, gain and two products a rounding each: under 32 roundings of 2^-24, of |a c| + |b s|; one rounding to
fp16, 2^-11, 2^-25 among its subnormal numbers."""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests import cache_ref as ref
from tests.gpu_helpers import cuda, host

pytestmark = pytest.mark.gpu
INT8, E4M3 = tri.TRI_KV_INT8, tri.TRI_KV_E4M3
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


def table_of(rows, dims):
    freq = 10000.0 ** (-np.arange(0, dims, 2) / dims)
    a = np.arange(rows)[:, None] * freq
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def near(got, want, tol, what=""):
    got = got.astype(np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %g at %s" % (
        what, bad.sum(), bad.size, (np.abs(got - want) / tol)[bad].max(), np.argwhere(bad)[0])


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dims,interleaved", [("all", False), ("all", True), ("half", False), (16, True), (48, False), (0, False)])
def test_rotate(D, dims, interleaved):
    import torch
    dims = {"all": D, "half": D // 2}.get(dims, dims)
    rng = np.random.default_rng([1, D, dims])
    rows = 50
    tab = table_of(rows, dims) if dims else None
    for T, H, Hk, norm, gains in [(1, 1, 1, True, True), (3, 5, 2, True, False), (67, 32, 8, True, True), (70, 17, 1, False, False)]:
        q, k = (rng.standard_normal((T, h, D)).astype(np.float16) for h in (H, Hk))
        q[0] *= 30
        k[-1] = 0                                # a row of zeros
        pos = rng.integers(0, rows, T).astype(np.int32)
        gq, gk = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float16) for _ in range(2)) if gains else (None, None)
        r = tri.Rotary(None if tab is None else cuda(tab), gains=(cuda(gq), cuda(gk)) if gains else None, norm=norm,
                       eps=1e-5, interleaved=interleaved)
        yq, yk = tri.heads_rotate((cuda(q), cuda(k)), r, cuda(pos))
        for x, y, g in ((q, yq, gq), (k, yk, gk)):
            want, mag = ref.rotate(x, pos, tab, interleaved, norm, float(np.float32(1e-5)), g)
            near(host(y), want, 32 * 2.0 ** -24 * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -25, (T, H, norm))


def test_rotate_strided_in_place_and_untouched_rows():
    import torch
    rng = np.random.default_rng(2)
    T, D = 9, 128
    x = rng.standard_normal((T, 7, D)).astype(np.float16)
    pos = np.array([0, -1, 3, 20, 5, 19, -2 ** 31, 2 ** 31 - 1, 1], dtype=np.int32)
    tab = table_of(20, D)
    ok = (pos >= 0) & (pos < 20)
    buf = cuda(x)
    q, k = buf[:, :5], buf[:, 5:6]               # heads of one buffer; the last head is nobody's
    r = tri.Rotary(cuda(tab), norm=True)
    out = torch.full((T, 6, D), NAN, dtype=torch.float16, device="cuda")
    tri.heads_rotate((q, k), r, cuda(pos), out=(out[:, 1:], torch.full((T, 1, D), NAN, dtype=torch.float16, device="cuda")))
    want, mag = ref.rotate(x[:, :5], np.clip(pos, 0, 19), tab)
    got = host(out)
    assert np.isnan(got[:, 0]).all() and np.isnan(got[~ok]).all()
    near(got[ok, 1:], want[ok], (32 * 2.0 ** -24 * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)[ok])
    tri.heads_rotate((q, k), r, cuda(pos), out=(q, k))
    again = host(buf)
    assert np.array_equal(again[ok, :5].view(np.uint16), got[ok, 1:].view(np.uint16))
    assert np.array_equal(again[~ok].view(np.uint16), x[~ok].view(np.uint16))
    assert np.array_equal(again[:, 6].view(np.uint16), x[:, 6].view(np.uint16))


def test_rotate_extreme_values():
    """The largest fp16 numbers stay finite under a norm; a row that is not finite spoils no other; no norm, no turn: the same bits."""
    D, T = 128, 4
    x = np.random.default_rng(3).standard_normal((T, 3, D)).astype(np.float16)
    x[0, 0] = 65504
    x[1, 1, 5] = np.inf
    x[2, 2] = 2.0 ** -24
    pos = np.zeros(T, dtype=np.int32)
    y = host(tri.heads_rotate((cuda(x),), tri.Rotary(None, eps=0.0), cuda(pos))[0])
    assert np.array_equal(y[0, 0], np.ones(D)) and np.array_equal(y[2, 2], np.ones(D))
    fine = np.ones((T, 3), dtype=bool)
    fine[1, 1] = False
    assert np.isfinite(y[fine]).all()
    z = host(tri.heads_rotate((cuda(x),), tri.Rotary(None, norm=False), cuda(pos - 5))[0])
    assert np.array_equal(z.view(np.uint16), x.view(np.uint16))


# ---------------------------------------------------------------- appending

def same_cache(cache, b, what=""):
    for got, want in ((cache.K, b.K), (cache.V, b.V)):
        np.testing.assert_array_equal(host(got), want, err_msg=str(what))
    for got, want in ((cache.K_scale, b.ks), (cache.V_scale, b.vs)):
        np.testing.assert_array_equal(host(got).view(np.uint32), want.view(np.uint32), err_msg=str(what))


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128), (256, 16), (256, 64), (256, 128)])
def test_append_bit_for_bit(D, page, fmt):
    rng = np.random.default_rng([4, D, page, fmt])
    for new, lens, heads in [([1], [1], 1), ([1, 1, 1, 1], [page, page + 1, 5, 2 * page + 3], 3), ([0, 1, 0], [0, 7, 9], 2),
                             ([3, page + 5, 0, 2 * page + 1, 1], [3, page + 9, 4, 2 * page + 1, 3 * page], 2),
                             ([7, 5], [page + 3, page], 1)]:
        b = ref.Batch(rng, new, lens, heads, D, page, fmt)
        K, V = (rng.standard_normal((b.T, heads, D)).astype(np.float16) for _ in range(2))
        for x in (K, V):
            x *= (10.0 ** rng.uniform(-3, 2, (b.T, 1, 1))).astype(np.float16)      # scales that grow, and that do not
        cache, seqs = b.on_gpu()
        for _ in range(2):                       # (the same tokens once more change nothing)
            tri.cache_append(cache, seqs, cuda(K), cuda(V))
            if _ == 0:
                b.append(K, V)
            same_cache(cache, b, (new, lens, heads))


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_append_token_by_token_through_a_page(fmt):
    """Forty single tokens of growing and shrinking size; the scale follows the definition at each."""
    rng = np.random.default_rng([5, fmt])
    b = ref.Batch(rng, [1, 1], [40, 45], 2, 64, 32, fmt)
    cache, seqs = b.on_gpu()
    last = list(b.lens)
    for s in range(40):
        b.lens = [s + 1, s + 6]
        seqs.lens.copy_(cuda(np.asarray(b.lens, dtype=np.int32)))
        K, V = ((rng.standard_normal((2, 2, 64)) * 2.0 ** rng.uniform(-6, 6)).astype(np.float16) for _ in range(2))
        tri.cache_append(cache, seqs, cuda(K), cuda(V))
        b.append(K, V)
        same_cache(cache, b, s)
    assert b.lens == last


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("n", [1, 4])
def test_append_values_that_are_not_finite_and_borders(n, fmt):
    rng = np.random.default_rng([6, n, fmt])
    top = ref.TOP[fmt]
    for fill in [0.0, -0.0, top, -top, top / 2, 65504.0, np.inf, -np.inf, NAN, 2.0 ** -24, 2.0 ** -14, np.nextafter(np.float16(top), np.float16(1e4))]:
        b = ref.Batch(rng, [n, n], [n, n + 3], 2, 64, 16, fmt)
        K, V = (rng.standard_normal((2 * n, 2, 64)).astype(np.float16) for _ in range(2))
        K[:, 0] = fill
        V[:, 1, ::2] = fill
        V[:, 1, 1::2] = 0
        K[0, 1, 3] = NAN
        cache, seqs = b.on_gpu()
        tri.cache_append(cache, seqs, cuda(K), cuda(V))
        b.append(K, V)
        same_cache(cache, b, fill)


def test_append_keeps_a_scale_that_is_no_power_of_two():
    rng = np.random.default_rng(7)
    for fmt in (INT8, E4M3):
        b = ref.Batch(rng, [2, 1], [9, 5], 2, 64, 16, fmt)
        b.ks[:], b.vs[:] = 0.0371, 0.0593
        K, V = (rng.standard_normal((3, 2, 64)).astype(np.float16) for _ in range(2))
        V[2] *= 100                              # this one's scale grows from 0.0593
        cache, seqs = b.on_gpu()
        tri.cache_append(cache, seqs, cuda(K), cuda(V))
        b.append(K, V)
        assert (b.ks == np.float32(0.0371)).any() and not (b.vs[b.table[1, 0]] == np.float32(0.0593)).any()
        same_cache(cache, b, fmt)


def test_append_leaves_out_what_has_no_place():
    """Pages outside the cache, positions before 0 and past the table, tokens behind max_new, rows of no sequence."""
    rng = np.random.default_rng(8)
    for fmt in (INT8, E4M3):
        for n in (1, 20):
            b = ref.Batch(rng, [n] * 6, [40, 40, 40, 40, 3, 60], 2, 64, 16, fmt, width=3)
            b.table[0, 2] = -1
            b.table[1, 1:] = len(b.K)
            b.table[2, 2] = 2 ** 31 - 1
            b.table[3, 2] = -2 ** 31
            b.offsets += 2                       # the first two rows are nobody's
            T = b.T + 2 + 3
            K, V = (rng.standard_normal((T, 2, 64)).astype(np.float16) for _ in range(2))
            for most in (n, max(1, n - 7)):
                cache, seqs = b.on_gpu(max_new=most)
                tri.cache_append(cache, seqs, cuda(K), cuda(V))
                old = [x.copy() for x in (b.K, b.V, b.ks, b.vs)]
                b.append(K, V, max_new=most)
                same_cache(cache, b, (fmt, n, most))
                b.K, b.V, b.ks, b.vs = old


def test_append_strided_rows():
    """Keys and values as views of one buffer of a layer's outputs."""
    rng = np.random.default_rng(9)
    b = ref.Batch(rng, [1, 30, 2], [33, 30, 7], 2, 128, 32, E4M3)
    x = rng.standard_normal((b.T, 9, 128)).astype(np.float16)
    buf = cuda(x)
    for new in (b.new, [1, 1, 1]):
        b.new, b.offsets = new, np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        cache, seqs = b.on_gpu()
        T = int(b.offsets[-1])
        tri.cache_append(cache, seqs, buf[:T, 5:7], buf[:T, 7:])
        b.append(x[:, 5:7], x[:, 7:])
        same_cache(cache, b, new)


@pytest.mark.parametrize("D,page,fmt,dims,interleaved", [(64, 16, INT8, 64, False), (128, 64, E4M3, 128, False), (128, 64, INT8, 64, True),
                                                         (256, 128, E4M3, 256, True), (128, 32, INT8, 0, False)])
def test_append_with_rotation_is_rotate_then_append(D, page, fmt, dims, interleaved):
    """The same codes, scales and queries, bit for bit, as two calls; tokens outside the rotation's table are left out."""
    import torch
    rng = np.random.default_rng([10, D, page])
    rows = 60
    tab = cuda(table_of(rows, dims)) if dims else None
    gains = [cuda((1 + 0.3 * rng.standard_normal(D)).astype(np.float16)) for _ in range(2)]
    r = tri.Rotary(tab, gains=gains, norm=True, interleaved=interleaved)
    for new, lens in [([1, 1, 1], [1, 50, 61]), ([5, 0, 40, 1], [5, 9, 70, 33]), ([1], [20]), ([1] * 70, list(range(1, 71))), ([3], [1])]:
        b = ref.Batch(rng, new, lens, 2, D, page, fmt)
        T = b.T + 3
        K, V = (rng.standard_normal((T, 2, D)).astype(np.float16) for _ in range(2))
        Q = cuda(rng.standard_normal((T, 6, D)).astype(np.float16))
        pos = np.concatenate([np.arange(l - n, l) for n, l in zip(new, lens)] + [np.full(3, -1)]).astype(np.int32)
        has = (pos >= 0) & ((pos < rows) if dims else True)
        k2, q2 = tri.heads_rotate((cuda(K), Q), tri.Rotary(tab, gains=gains[::-1], norm=True, interleaved=interleaved),
                                  cuda(np.where(has, pos, 0).astype(np.int32)))
        cache, seqs = b.on_gpu()
        out = torch.full_like(Q, NAN)
        got = tri.cache_append(cache, seqs, cuda(K), cuda(V), rotary=r, Q=Q, out=out)
        assert got is out
        b.append(host(k2), V, rows=rows if dims else None)
        same_cache(cache, b, (new, lens))
        q = host(out)
        assert np.isnan(q[~has]).all()
        np.testing.assert_array_equal(q[has].view(np.uint16), host(q2)[has].view(np.uint16))
        # in place
        tri.cache_append(cache, seqs, cuda(K), cuda(V), rotary=r, Q=Q, out=Q)
        np.testing.assert_array_equal(host(Q)[has].view(np.uint16), host(q2)[has].view(np.uint16))


# ---------------------------------------------------------------- attention

def check_attend(b, H, rng, scale=None, window=0, sinks=0, max_len=None, qsize=1.0, extra=0, what=""):
    import torch
    T = int(b.offsets[-1]) + extra
    scale = b.D ** -0.5 if scale is None else scale
    Q = (qsize * rng.standard_normal((T, H, b.D))).astype(np.float16)
    cache, seqs = b.on_gpu(max_len=max_len)
    out = torch.full((T, H, b.D), NAN, dtype=torch.float16, device="cuda")
    q = cuda(Q)
    got = host(tri.cache_attend(cache, seqs, q, scale=scale, window=window, sinks=sinks, out=out))
    want, tol, live = b.attend(Q, float(np.float32(scale)), window, sinks)
    assert np.isnan(got[~live]).all(), what
    near(got[live], want[live], tol[live], what)
    again = host(tri.cache_attend(cache, seqs, q, scale=scale, window=window, sinks=sinks))
    np.testing.assert_array_equal(again[live].view(np.uint16), got[live].view(np.uint16))
    return got


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128), (256, 16), (256, 32), (256, 128)])
def test_attend_one_token(D, page, fmt):
    rng = np.random.default_rng([20, D, page, fmt])
    for lens, heads, G in [([1], 1, 1), ([63, 64, 65, 1], 2, 4), ([700, 3, 129], 1, 7), ([300], 2, 17), ([2000], 1, 8)]:
        b = ref.Batch(rng, [1] * len(lens), lens, heads, D, page, fmt)
        check_attend(b, heads * G, rng, what=(lens, heads, G))


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 16), (256, 32), (128, 128)])
def test_attend_several_tokens(D, page, fmt):
    rng = np.random.default_rng([21, D, page, fmt])
    for new, lens, heads, G in [([2, 5, 0, 1], [2, 70, 0, 9], 2, 1), ([3, 8], [300, 8], 1, 4), ([33], [33], 1, 1), ([40, 17], [40, 200], 2, 3),
                                ([130], [190], 1, 2), ([65, 3, 64], [65, 500, 300], 1, 8)]:
        b = ref.Batch(rng, new, lens, heads, D, page, fmt)
        check_attend(b, heads * G, rng, extra=2, what=(new, lens, heads, G))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (64, 64), (100, 4), (100, 130), (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1),
                                          (17, 2 ** 31 - 1)])
def test_attend_window_and_sinks(window, sinks):
    rng = np.random.default_rng([22, window, sinks])
    for new, lens, heads, G, page, D in [([1, 1, 1], [700, 64, 5], 2, 2, 16, 64), ([50, 3], [400, 90], 1, 3, 64, 128), ([1], [1500], 1, 1, 128, 128),
                                         ([200], [200], 1, 1, 32, 64)]:
        b = ref.Batch(rng, new, lens, heads, D, page, E4M3 if D == 64 else INT8)
        check_attend(b, heads * G, rng, window=window, sinks=sinks, what=(new, lens))


def test_attend_rows_that_see_nothing():
    """Sequences without tokens, positions before 0, pages that are not there: 0; a window over missing pages likewise."""
    rng = np.random.default_rng(23)
    for n in (1, 3, 40):
        b = ref.Batch(rng, [n, n, 1, n], [max(0, n - 1), 5, 200, 0], 2, 64, 16, INT8, width=13)
        b.table[2] = -1
        got = check_attend(b, 4, rng, what=n)
        assert (got[2 * n] == 0).all() and (got[2 * n + 1:] == 0).all()
        b = ref.Batch(rng, [1, n], [200, 200], 1, 128, 16, E4M3)
        b.table[:, 3:7] = [-5, len(b.K), 2 ** 31 - 1, -2 ** 31]
        check_attend(b, 2, rng, what=n)
        b.table[:, 8:] = -1
        check_attend(b, 2, rng, window=50, sinks=0, what=n)
    # a length that the table has no room for: the tokens past it are not seen
    b = ref.Batch(rng, [1, 2], [100, 200], 1, 64, 16, INT8)
    b.table, b.width = np.ascontiguousarray(b.table[:, :5]), 5
    check_attend(b, 2, rng)


def test_attend_masked_places_may_hold_anything():
    """Codes that are no numbers, scales that are zero, huge or not finite where no token is visible change nothing."""
    rng = np.random.default_rng(24)
    for fmt in (INT8, E4M3):
        for new, lens, w in [([1, 4], [70, 5], 0), ([1, 100], [333, 130], 0), ([1, 3], [300, 290], 64)]:
            b = ref.Batch(rng, new, lens, 2, 128, 16, fmt)
            want = check_attend(b, 4, np.random.default_rng(1), window=w)
            for i, l in enumerate(lens):
                b.K[b.table[i, (l - 1) // 16], :, (l - 1) % 16 + 1:] = 0x7F
                b.V[b.table[i, (l - 1) // 16], :, :, (l - 1) % 16 + 1:] = 0xFF
                if w:                            # pages that the window has left behind
                    for page in range((l - new[i] - w) // 16):
                        b.K[b.table[i, page]], b.V[b.table[i, page]] = 0xFF, 0x7F
                        b.ks[b.table[i, page]], b.vs[b.table[i, page]] = NAN, [0.0, np.inf][page % 2]
            used = np.unique(b.table[b.table >= 0])
            spare = np.setdiff1d(np.arange(len(b.K)), used)
            b.ks[spare], b.vs[spare], b.K[spare], b.V[spare] = NAN, NAN, 0x7F, 0x7F
            got = check_attend(b, 4, np.random.default_rng(1), window=w)
            np.testing.assert_array_equal(got.view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("n", [1, 40])
def test_attend_sizes_of_scores_and_scales(n):
    """Sharp and flat softmax, negative and zero scale, scales of values far apart, the smallest scales."""
    rng = np.random.default_rng([25, n])
    for fmt in (INT8, E4M3):
        for scale, qsize in [(0.0, 1.0), (-0.1, 1.0), (1.0, 8.0), (0.088, 0.01), (3.0, 30.0)]:
            b = ref.Batch(rng, [n, 1], [260, 90], 1, 64, 32, fmt)
            check_attend(b, 2, rng, scale=scale, qsize=qsize, what=(fmt, scale))
        b = ref.Batch(rng, [n], [400], 1, 128, 16, fmt)
        b.vs[:] = (2.0 ** rng.integers(-30, 3, b.vs.shape)).astype(np.float32)
        check_attend(b, 4, rng, what="scales far apart")
        b.vs[:] = 2.0 ** -30
        b.ks[:] = 2.0 ** -30
        check_attend(b, 4, rng, scale=2.0 ** 28, what="small scales")


def test_attend_queries_that_are_not_finite_spoil_only_their_rows():
    rng = np.random.default_rng(26)
    for n in (1, 5, 50):
        b = ref.Batch(rng, [n], [n + 100], 1, 64, 16, INT8)
        Q = rng.standard_normal((n, 4, 64)).astype(np.float16)
        cache, seqs = b.on_gpu()
        want = host(tri.cache_attend(cache, seqs, cuda(Q)))
        Q[n // 2, 1, 3], Q[0, 2, 0] = NAN, np.inf
        got = host(tri.cache_attend(cache, seqs, cuda(Q)))
        bad = np.zeros((n, 4), dtype=bool)
        bad[n // 2, 1] = bad[0, 2] = True
        np.testing.assert_array_equal(got[~bad].view(np.uint16), want[~bad].view(np.uint16))
        assert np.isnan(got[bad]).all()


def test_attend_beyond_the_stated_length_and_new_tokens():
    """A length past max_len is taken whole; only the first max_new new tokens are taken."""
    import torch
    rng = np.random.default_rng(27)
    for n in (1, 3, 40):
        b = ref.Batch(rng, [n], [900], 1, 64, 16, INT8)
        check_attend(b, 2, rng, max_len=70, what=n)
    b = ref.Batch(rng, [9, 50], [30, 300], 2, 64, 32, E4M3)
    Q = rng.standard_normal((59, 2, 64)).astype(np.float16)
    for most in (1, 4, 40):
        cache, seqs = b.on_gpu(max_new=most)
        out = torch.full((59, 2, 64), NAN, dtype=torch.float16, device="cuda")
        got = host(tri.cache_attend(cache, seqs, cuda(Q), out=out))
        want, tol, live = b.attend(Q, 0.125, max_new=most)
        assert np.isnan(got[~live]).all() and live.sum() == min(9, most) + most
        near(got[live], want[live], tol[live], most)


def test_attend_strided_queries_and_results():
    import torch
    rng = np.random.default_rng(28)
    for new, lens in [([1, 1, 1], [100, 7, 64]), ([2, 40], [50, 90])]:
        b = ref.Batch(rng, new, lens, 2, 128, 64, E4M3)
        x = rng.standard_normal((b.T, 9, 128)).astype(np.float16)
        cache, seqs = b.on_gpu()
        out = torch.full((b.T, 8, 128), NAN, dtype=torch.float16, device="cuda")
        tri.cache_attend(cache, seqs, cuda(x)[:, 2:8], out=out[:, 1:7])
        want, tol, _ = b.attend(x[:, 2:8], float(np.float32(128 ** -0.5)))
        got = host(out)
        near(got[:, 1:7], want, tol)
        assert np.isnan(got[:, [0, 7]]).all()


def test_a_cache_past_four_gigabytes():
    """Pages at both ends of a cache of more than 4 GiB of keys, and as many of values."""
    import torch
    rng = np.random.default_rng(29)
    heads, page, D = 8, 128, 128
    pages = (1 << 32) // (heads * page * D) + 50
    big = tri.KVCache.empty(pages, heads, D, page, E4M3)
    assert big.K.numel() > 1 << 32
    ids = [0, pages - 1, 1, pages - 2, pages // 2]
    for new, total in [(600, 600), (1, 601)]:
        b = ref.Batch(rng, [new], [total], heads, D, page, E4M3, spare=0, codes=False) if new == 600 else b
        b.new, b.lens, b.offsets, b.T = [new], [total], np.array([0, new], dtype=np.int32), new
        table = cuda(np.array([ids], dtype=np.int32))
        seqs = tri.Sequences(cuda(b.offsets), cuda(np.array(b.lens, dtype=np.int32)), table, max_new=new)
        K, V = (rng.standard_normal((new, heads, D)).astype(np.float16) for _ in range(2))
        tri.cache_append(big, seqs, cuda(K), cuda(V))
        b.append(K, V)
        at = torch.tensor([ids[list(b.table[0]).index(i)] for i in range(5)], device="cuda")
        np.testing.assert_array_equal(host(big.K[at]), b.K)
        np.testing.assert_array_equal(host(big.V[at]), b.V)
        Q = rng.standard_normal((new, heads, D)).astype(np.float16)
        got = host(tri.cache_attend(big, seqs, cuda(Q)))
        want, tol, _ = b.attend(Q, float(np.float32(D ** -0.5)))
        near(got, want, tol, new)


@pytest.mark.parametrize("D,fmt", [(64, E4M3), (128, INT8), (256, INT8)])
def test_attend_many_rows_in_splits(D, fmt):
    """Tiles of many rows whose steps are shared by workgroups and joined, with and without a window."""
    rng = np.random.default_rng([41, D])
    for new, lens, heads, G, window, sinks in [([40], [5000], 1, 1, 0, 0), ([50, 3], [3000, 2000], 1, 4, 0, 0), ([33], [6000], 1, 2, 2500, 70)]:
        b = ref.Batch(rng, new, lens, heads, D, 64, fmt)
        check_attend(b, heads * G, rng, window=window, sinks=sinks, what=(new, lens))


@pytest.mark.parametrize("D", [64, 128])
def test_attend_many_rows_in_many_tiles(D):
    """More tiles than the two per CU up to which two groups of waves share one."""
    rng = np.random.default_rng([42, D])
    B, heads = 70, 8
    new = [int(x) for x in rng.integers(33, 50, B)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 150, B))]
    b = ref.Batch(rng, new, lens, heads, D, 16, INT8)
    check_attend(b, heads, rng)


def test_bounds_far_beyond_what_sequences_have():
    """max_new of thousands for sequences of one token each: more workgroups than one launch takes.  A token that sees itself
    alone gives its value."""
    import torch
    rng = np.random.default_rng(43)
    B, heads, D, page = 3000, 32, 64, 16
    K, V = (cuda(rng.standard_normal((B, heads, D)).astype(np.float16)) for _ in range(2))
    cache = tri.KVCache.empty(B, heads, D, page, INT8)
    i32 = dict(dtype=torch.int32, device="cuda")
    seqs = tri.Sequences(torch.arange(B + 1, **i32), torch.ones(B, **i32), torch.randperm(B, device="cuda").to(torch.int32)[:, None].contiguous(),
                         max_new=B)
    tri.cache_append(cache, seqs, K, V)
    one = tri.KVCache.empty(B, heads, D, page, INT8)
    single = tri.Sequences(seqs.offsets, seqs.lens, seqs.table, max_new=1)
    tri.cache_append(one, single, K, V)
    for x, y in ((cache.K, one.K), (cache.V, one.V), (cache.K_scale, one.K_scale), (cache.V_scale, one.V_scale)):
        assert torch.equal(x, y)
    at = seqs.table[:, 0].long()
    want = (cache.V.view(torch.int8)[at, :, :, 0].float() * cache.V_scale[at][..., None]).half()
    Q = torch.randn((B, heads, D), device="cuda").half()
    for sq in (seqs, single):
        assert torch.equal(tri.cache_attend(cache, sq, Q), want)


@pytest.mark.parametrize("n", [1, 20, 100])
def test_flat_weights_and_equal_values(n):
    """Equal scores and equal values: the mean of equal values is that value, whatever the number of tokens (roundings of equal
    weights must cancel)."""
    rng = np.random.default_rng([44, n])
    for L in (n, n + 37, n + 1000):
        for fmt, code in ((INT8, 77), (E4M3, 0x45)):
            b = ref.Batch(rng, [n], [L], 1, 64, 16, fmt)
            b.V[:], b.vs[:], b.ks[:] = code, 0.75, 0.01
            cache, seqs = b.on_gpu()
            Q = rng.standard_normal((n, 2, 64)).astype(np.float16)
            got = host(tri.cache_attend(cache, seqs, cuda(Q), scale=0.0)).astype(np.float64)
            v = ref.values_of(fmt)[code] * 0.75
            assert np.all(np.abs(got - v) <= 2.0 ** -11 * v + (L + 64) * 2.0 ** -23 * v), (L, fmt)


def test_long_contexts():
    """Splits of a long context, with and without a window, against sums taken in float64 on the GPU."""
    import torch
    rng = np.random.default_rng(30)
    for fmt, L, G, window, sinks in [(INT8, 70000, 8, 0, 0), (E4M3, 131077, 1, 0, 0), (INT8, 40000, 4, 9000, 100)]:
        b = ref.Batch(rng, [1], [L], 1, 128, 64, fmt)
        cache, seqs = b.on_gpu()
        Q = rng.standard_normal((1, G, 128)).astype(np.float16)
        got = host(tri.cache_attend(cache, seqs, cuda(Q), window=window, sinks=sinks))
        want, tol, _ = b.attend(Q, float(np.float32(128 ** -0.5)), window, sinks)
        near(got, want, tol, (fmt, L))


# ---------------------------------------------------------------- together

def block(rng, hidden, H, Hkv, D, fmt=tri.TRI_FMT_2BIT):
    from bit_mixed_precision_tri_amd import synth
    sizes = [H * D, Hkv * D, Hkv * D]
    W = [tri.pack(cuda(synth.trits(rng, n, hidden)), fmt) for n in sizes] + [tri.pack(cuda(synth.trits(rng, hidden, H * D)), fmt)]
    return W, sizes


def test_decoder_steps_with_the_layers():
    """A prompt and then single tokens of two sequences through norm, Q/K/V layers, rotation and appending, attention, O layer and
    residual: every step's attention against the definition on the queries and the cache that it read, and the whole captured
    in a graph whose replays follow lengths changed in place."""
    import torch
    rng = np.random.default_rng(31)
    hidden, H, Hkv, D, page = 256, 4, 2, 64, 16
    W, sizes = block(rng, hidden, H, Hkv, D)
    gains = [cuda((1 + 0.2 * rng.standard_normal(D)).astype(np.float16)) for _ in range(2)]
    rot = tri.Rotary(cuda(table_of(100, D)), gains=gains)
    b = ref.Batch(rng, [7, 3], [30, 40], Hkv, D, page, E4M3, codes=False)
    b.lens = [7, 3]
    cache, seqs = b.on_gpu()
    x = cuda(rng.standard_normal((10, hidden)).astype(np.float16))

    def step(x, seqs, bufs):
        M = x.shape[0]
        q, k, v, a, y = bufs
        tri.tri_linear_fused(x, W[:3], [0.05, 0.05, 0.05], M, sizes, hidden, tri.TRI_FMT_2BIT, [q, k, v], norm=True)
        q3 = q.view(M, H, D)
        tri.cache_append(cache, seqs, k.view(M, Hkv, D), v.view(M, Hkv, D), rotary=rot, Q=q3, out=q3)
        tri.cache_attend(cache, seqs, q3, out=a.view(M, H, D))
        tri.tri_linear_fused(a, W[3:], [0.05], M, [hidden], H * D, tri.TRI_FMT_2BIT, [y], residuals=[x])

    def bufs(M):
        return [torch.empty((M, n), dtype=torch.float16, device="cuda") for n in sizes + [H * D, hidden]]

    def check(bs):
        b.K, b.V, b.ks, b.vs = host(cache.K), host(cache.V), host(cache.K_scale), host(cache.V_scale)
        want, tol, _ = b.attend(host(bs[0]).reshape(-1, H, D), float(np.float32(D ** -0.5)))
        near(host(bs[3]).reshape(-1, H, D), want, tol)

    bs = bufs(10)
    step(x, seqs, bs)
    check(bs)
    y = bs[4]

    one = tri.Sequences(cuda(np.array([0, 1, 2], dtype=np.int32)), seqs.lens, seqs.table, max_new=1)
    b.new, b.offsets = [1, 1], np.array([0, 1, 2], dtype=np.int32)
    xs = y[[6, 9]].contiguous()
    bs = bufs(2)
    side = torch.cuda.Stream()
    saved = [t.clone() for t in (cache.K, cache.V, cache.K_scale, cache.V_scale)]
    seqs.lens += 1
    with torch.cuda.stream(side):                # warm-up off the graph
        side.wait_stream(torch.cuda.current_stream())
        step(xs, one, bs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(xs, one, bs)
    for t, s in zip((cache.K, cache.V, cache.K_scale, cache.V_scale), saved):
        t.copy_(s)
    seqs.lens -= 1
    first = xs.clone()
    replays = []
    for i in range(20):                          # past the ends of pages
        seqs.lens += 1
        b.lens = [7 + i + 1, 3 + i + 1]
        graph.replay()
        torch.cuda.synchronize()
        check(bs)
        replays.append(host(bs[4]).copy())
        xs.copy_(bs[4])
    # the same steps without the graph
    for t, s in zip((cache.K, cache.V, cache.K_scale, cache.V_scale), saved):
        t.copy_(s)
    seqs.lens.copy_(cuda(np.array([7, 3], dtype=np.int32)))
    xs.copy_(first)
    for i in range(20):
        seqs.lens += 1
        step(xs, one, bs)
        np.testing.assert_array_equal(host(bs[4]).view(np.uint16), replays[i].view(np.uint16))
        xs.copy_(bs[4])


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream with eager work between."""
    import torch
    rng = np.random.default_rng(32)
    calls = []
    for L, G in ((5000, 4), (9000, 2)):
        b = ref.Batch(rng, [1], [L], 2, 128, 64, INT8)
        cache, seqs = b.on_gpu()
        q = cuda(rng.standard_normal((1, 2 * G, 128)).astype(np.float16))
        calls.append((cache, seqs, q, torch.empty_like(q), host(tri.cache_attend(cache, seqs, q))))
    need = max(tri.cache_attend_workspace_bytes(c, s, 1, q.shape[1]) for c, s, q, _, _ in calls)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for c, s, q, o, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tri.cache_attend(c, s, q, workspace=ws, out=o)
        graphs.append(g)
    for i in range(6):
        for g, (_, _, _, o, want) in zip(graphs, calls):
            o.zero_()
            ws.fill_(0xFF)
            g.replay()
            np.testing.assert_array_equal(host(o).view(np.uint16), want.view(np.uint16))


def test_named_streams():
    """A call on a stream of its own gives what it gives on the current one, its results and workspace made for that stream."""
    import torch
    rng = np.random.default_rng(33)
    b = ref.Batch(rng, [1, 1], [3000, 400], 2, 128, 64, E4M3)
    cache, seqs = b.on_gpu()
    q = cuda(rng.standard_normal((2, 4, 128)).astype(np.float16))
    k, v = (cuda(rng.standard_normal((2, 2, 128)).astype(np.float16)) for _ in range(2))
    rot = tri.Rotary(cuda(table_of(4000, 128)))
    want_q = tri.cache_append(cache, seqs, k, v, rotary=rot, Q=q)
    want = host(tri.cache_attend(cache, seqs, want_q))
    want_k = host(tri.heads_rotate((k,), rot, seqs.lens - 1)[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del junk
    q2 = tri.cache_append(cache, seqs, k, v, rotary=rot, Q=q, stream=s)
    o = tri.cache_attend(cache, seqs, q2, stream=s)
    pos = seqs.lens - 1
    torch.cuda.synchronize()
    k2 = tri.heads_rotate((k,), rot, pos, stream=s.cuda_stream)[0]
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(o).view(np.uint16), want.view(np.uint16))
    np.testing.assert_array_equal(host(q2).view(np.uint16), host(want_q).view(np.uint16))
    np.testing.assert_array_equal(host(k2).view(np.uint16), want_k.view(np.uint16))


def test_helpers_refusals():
    import torch
    rng = np.random.default_rng(34)
    b = ref.Batch(rng, [1, 2], [20, 30], 2, 64, 16, INT8)
    cache, seqs = b.on_gpu()
    f16 = dict(dtype=torch.float16, device="cuda")
    q, k = torch.zeros((3, 4, 64), **f16), torch.zeros((3, 2, 64), **f16)
    rot = tri.Rotary(cuda(table_of(40, 64)))
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [
        lambda: tri.cache_attend(cache, seqs, q.float()), lambda: tri.cache_attend(cache, seqs, q.cpu()),
        lambda: tri.cache_attend(cache, seqs, q[..., :32]), lambda: tri.cache_attend(cache, seqs, q.transpose(0, 1)),
        lambda: tri.cache_attend(cache, seqs, q[0]), lambda: tri.cache_attend(cache, seqs, q, out=k),
        lambda: tri.cache_attend(cache, seqs, q, out=q[:2].clone()), lambda: tri.cache_attend(cache, seqs, q, workspace=q),
        lambda: tri.cache_append(cache, seqs, k, k[:2]), lambda: tri.cache_append(cache, seqs, q, q),
        lambda: tri.cache_append(cache, seqs, k, k, Q=q), lambda: tri.cache_append(cache, seqs, k, k, rotary=rot, out=q),
        lambda: tri.cache_append(cache, seqs, k, k, rotary=rot, Q=q[:2]),
        lambda: tri.heads_rotate((q, k[:2]), rot, pos), lambda: tri.heads_rotate((q,), rot, pos[:2]),
        lambda: tri.heads_rotate((q,), rot, pos.long()), lambda: tri.heads_rotate((), rot, pos),
        lambda: tri.heads_rotate((q,) * 5, rot, pos), lambda: tri.heads_rotate((q, k), rot, pos, out=(q,)),
        lambda: tri.heads_rotate((q, k), tri.Rotary(None, gains=(None,)), pos),
        lambda: tri.heads_rotate((q,), tri.Rotary(None, gains=(q[0, 0, :32],)), pos),
        lambda: tri.KVCache(cache.K, cache.K, cache.K_scale, cache.V_scale, INT8),
        lambda: tri.KVCache(cache.K, cache.V, cache.K_scale, cache.V_scale, 7),
        lambda: tri.KVCache(cache.K, cache.V, cache.K_scale.half(), cache.V_scale, INT8),
        lambda: tri.KVCache(cache.K[:, :, :8].contiguous(), cache.V, cache.K_scale, cache.V_scale, INT8),
        lambda: tri.Sequences(seqs.offsets[:2], seqs.lens, seqs.table, 1), lambda: tri.Sequences(seqs.offsets, seqs.lens, seqs.table, 0),
        lambda: tri.Sequences(seqs.offsets.long(), seqs.lens, seqs.table, 1),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    with pytest.raises(tri.TriError):            # five query heads for two of the cache
        tri.cache_attend(cache, seqs, torch.zeros((3, 5, 64), **f16), workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tri.cache_attend_workspace_bytes(cache, seqs, 3, 5)


def test_sequences_that_caches_of_other_pages_share():
    """One Sequences without max_len for two caches: each call is sized by its own cache's pages, whichever came last."""
    import torch
    rng = np.random.default_rng(35)
    D, width = 64, 40
    K = rng.standard_normal((1, 2, D)).astype(np.float16)
    q = cuda(rng.standard_normal((1, 8, D)).astype(np.float16))
    seqs = tri.Sequences(cuda(np.array([0, 1], np.int32)), cuda(np.array([width * 16], np.int32)),
                         cuda(rng.permutation(width).astype(np.int32)[None]), 1)
    caches = [tri.KVCache.empty(width, 2, D, page, INT8) for page in (16, 128)]
    need = [tri.cache_attend_workspace_bytes(c, seqs, 1, 8) for c in caches]
    assert [tri.cache_attend_workspace_bytes(c, seqs, 1, 8) for c in caches[::-1]] == need[::-1] and need[0] < need[1]
    for c in caches:                             # (scales of 1, large enough for the new token: all values are 3)
        c.K.copy_(torch.randint(0, 256, c.K.shape, device="cuda"))
        c.V.fill_(3)
        tri.cache_append(c, seqs, cuda(K), cuda(np.full_like(K, 3)))
    for c, n in list(zip(caches, need)) * 2:
        o = tri.cache_attend(c, seqs, q, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"))
        assert np.abs(host(o).astype(np.float64) - 3).max() <= 3 * 2.0 ** -11    # (one rounding to fp16)
