"""Experts on the GPU: routing, ragged ternary products and their combination, against their definitions in float64.

Tolerance of a product.  The stored digits t + 1 are exact, sum_k t x is sum_k (t+1) x - sum_k x (at most 3 sum |x| in
magnitude); a term passes at most 32 additions inside a matrix instruction, one per later instruction on the same
accumulator (K/16 at most) and 48 of partial sums, each off by at most 2^-23 (a truncating adder); one rounding to fp16:
    d = (80 + K/16) 2^-23 3 |scale| sum_k |x|,   |Y - Y_ref| <= d + 2^-11 |Y_ref| + 2^-25.
The gated pair: silu'(z) <= 1.1, exp and the division within 2^-18:
    1.1 d_g |u| + |silu(g)| d_u + 1.1 d_g d_u + (2^-18 + 2^-11) |Y_ref| + 2^-25.
Combination: topk + 1 additions of fp32 products, each within 2^-24 of the terms' magnitudes, and one rounding.
"""
import numpy as np
import pytest

import oracle
import bit_mixed_precision_tri_amd as tri
from bit_mixed_precision_tri_amd import synth
from tests.gpu_helpers import say, cuda, host

pytestmark = pytest.mark.gpu
F2, F16 = tri.TRI_FMT_2BIT, tri.TRI_FMT_1P6BIT
INF = np.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------- routing

def route_ref(x, topk, renorm):
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -INF, x)
    T, E = x.shape
    order = np.argsort(-x, axis=1, kind="stable")[:, :topk]
    top = np.take_along_axis(x, order, 1)
    ids = np.where(top > -INF, order, -1)
    mx = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        mass = lambda v: np.where(v == -INF, 0.0, np.where(v == mx, 1.0, np.exp(v - mx)))
        den = (mass(top) if renorm else mass(x)).sum(1, keepdims=True)
        weights = np.where(ids >= 0, mass(top) / np.where(den > 0, den, 1.0), 0.0)
    flat = np.where(ids >= 0, ids, E).reshape(-1)
    by = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[by], np.arange(E + 1))
    rows = np.where(flat[by] < E, by // topk, -1)
    pos = np.empty(T * topk, dtype=np.int64)
    pos[by] = np.arange(T * topk)
    return ids, weights, offsets, rows, np.where(ids >= 0, pos.reshape(T, topk), -1)


def check_route(x, topk, renorm):
    import torch
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = tri.Routing(torch.full((T, topk), 77, **i32), torch.full((T, topk), 7.0, device="cuda"),
                      torch.full((E + 1,), 77, **i32), torch.full((T * topk,), 77, **i32), torch.full((T, topk), 77, **i32))
    got = tri.experts_route(cuda(x), topk, renorm=renorm, out=out)
    assert got is out
    ids, weights, offsets, rows, pos = (host(t) for t in got)
    rids, rweights, roffsets, rrows, rpos = route_ref(x, topk, renorm)
    np.testing.assert_array_equal(ids, rids)
    np.testing.assert_array_equal(offsets, roffsets)
    np.testing.assert_array_equal(rows, rrows)
    np.testing.assert_array_equal(pos, rpos)
    # x - max exact to 2^-24 of its size (<= 120 where exp does not vanish), exp to a few steps, E additions, a division
    assert np.all(np.abs(weights - rweights) <= (E + 140) * 2.0 ** -23 * rweights + 1e-38)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 100, 129, 700])
@pytest.mark.parametrize("E,topk", [(1, 1), (4, 2), (8, 8), (64, 6), (65, 3), (100, 16), (256, 8), (256, 16)])
def test_route(T, E, topk):
    rng = np.random.default_rng([51, T, E, topk])
    x = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    say("route T=%d E=%d k=%d" % (T, E, topk))
    for renorm in (True, False):
        check_route(x, topk, renorm)
        check_route((np.round(2 * x) / 2).astype(np.float16), topk, renorm)   # many equal logits


def test_route_long():
    """More workgroups than one adds up by itself; all tokens at one expert; a padded end."""
    rng = np.random.default_rng(52)
    x = rng.standard_normal((9001, 5)).astype(np.float32)
    check_route(x, 2, True)
    check_route(rng.standard_normal((20011, 256)).astype(np.float16), 3, False)
    x[:] = [0, 0, 9, 0, 0]
    check_route(x, 1, True)
    x[8000:] = -INF
    check_route(x, 2, False)


def test_route_masks_and_extremes():
    rng = np.random.default_rng(53)
    x = rng.standard_normal((40, 8)).astype(np.float32)
    x[0] = -INF                                  # a row without an expert
    x[1, :7] = -INF                              # fewer experts than topk
    x[2, 3] = np.nan
    x[3] = np.nan
    x[4, 5] = INF
    x[5, [1, 6]] = INF                           # two infinities share the weight
    x[6] = np.finfo(np.float32).min              # the lowest finite value is a logit like others
    x[7] = -INF
    x[7, 2] = np.finfo(np.float32).min
    x[8] = 0.0
    x[8, ::2] = -0.0                             # zeros of both signs are equal
    x[9, 4] = np.finfo(np.float32).max
    x[10] = [88, -88, 0, 1, 2, 3, 4, 5]
    x[39] = -INF
    for topk in (1, 2, 3, 8):
        for renorm in (True, False):
            check_route(x, topk, renorm)
    check_route(np.full((70, 8), -INF, dtype=np.float32), 2, True)   # padding only: no pair at all
    check_route(np.full((200, 8), -INF, dtype=np.float16), 4, False)


# ---------------------------------------------------------------- products

def places(sizes, first=0):
    return (first + np.concatenate([[0], np.cumsum(sizes)])).astype(np.int32)


def sum_bound(K, scale, X):
    return (80 + K / 16) * 2.0 ** -23 * 3.0 * abs(float(scale)) * np.abs(X).sum(1, keepdims=True)


def check_experts(rng, T, E, N, K, fmt, sizes, gather, pair, R=None, first=0, rows=None, what=""):
    import torch
    off = places(sizes, first)
    R = int(off[-1]) if R is None else R
    X = rng.standard_normal((T, K)).astype(np.float16)
    if gather and rows is None:
        rows = rng.integers(0, T, R).astype(np.int32)
    Ws = [synth.trits(rng, E * N, K).reshape(E, N, K) for _ in range(2 if pair else 1)]
    # scales of products around 1, so that a gate's exponential is exercised
    ss = [(rng.uniform(0.5, 1.5, E) / np.sqrt(0.6 * K)).astype(np.float32) for _ in Ws]
    mats = [(tri.pack(cuda(W.reshape(E * N, K)), fmt).view(E, N, -1), cuda(s)) for W, s in zip(Ws, ss)]
    Y = torch.full((R + 3, N), 7.0, dtype=torch.float16, device="cuda")
    say("experts %s T=%d E=%d N=%d K=%d fmt=%d R=%d gather=%d pair=%d" % (what, T, E, N, K, fmt, R, gather, pair))
    rd = cuda(rows) if gather else None
    Xd, od = cuda(X), cuda(off)
    if pair:
        tri.tri_experts_pair(Xd, T, od, rd, R, *mats[0], *mats[1], E, N, K, fmt, Y)
    else:
        tri.tri_experts_linear(Xd, T, od, rd, R, *mats[0], E, N, K, fmt, Y)
    got, X = host(Y).astype(np.float64), X.astype(np.float64)
    seen = np.zeros(R + 3, dtype=bool)
    for e in range(E):
        a, b = min(int(off[e]), R), min(int(off[e + 1]), R)
        r = np.arange(a, b)
        src = rows[a:b] if gather else r
        live = (src >= 0) & (src < T)
        r, x = r[live], X[src[live]]
        if not len(r):
            continue
        seen[r] = True
        ys = [float(s[e]) * (x @ W[e].astype(np.float64).T) for W, s in zip(Ws, ss)]
        ds = [sum_bound(K, s[e], x) for s in ss]
        if pair:
            sil = ys[0] / (1 + np.exp(-ys[0]))
            ref = sil * ys[1]
            tol = 1.1 * ds[0] * np.abs(ys[1]) + np.abs(sil) * ds[1] + 1.1 * ds[0] * ds[1] + 2.0 ** -18 * np.abs(ref)
        else:
            ref, tol = ys[0], ds[0]
        tol = tol + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
        err = np.abs(got[r] - ref)
        assert np.all(err <= tol), "%s expert %d: worst %.3g of the tolerance" % (what, e, np.max(err / tol))
    assert np.all(got[~seen] == 7.0), "a row that no expert owns was written"


RAGGED = {"one": [1], "few": [1, 0, 2, 1], "hole": [0, 0, 5, 0], "mixed": [3, 17, 0, 1, 16, 64, 33, 5],
          "single": [0, 130, 0], "many": [2, 0, 1, 3, 0, 0, 4, 1] * 8, "long": [200, 0, 70, 129], "empty": [0, 0]}


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("name", list(RAGGED))
def test_products_of_ragged_experts(name, pair, fmt):
    rng = np.random.default_rng([54, list(RAGGED).index(name), pair, fmt])
    sizes = RAGGED[name]
    for (N, K) in [(48, 256), (100, 648), (513, 1000), (130, 333)]:
        if len(sizes) > 32 and N > 200:
            continue
        for gather in (False, True):
            R = max(1, sum(sizes))
            check_experts(rng, R + 2 if not gather else 9, len(sizes), N, K, fmt, sizes, gather, pair, R=R, what=name)


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 16, 40])
@pytest.mark.parametrize("K", [4096, 11008, 28672])
def test_products_of_long_rows(K, M, fmt):
    """One expert of M rows, and two that share them unevenly."""
    rng = np.random.default_rng([55, M, fmt, K])
    N = 40 if K > 4096 else 80
    check_experts(rng, M, 1, N, K, fmt, [M], False, False)
    check_experts(rng, 7, 3, N, K, fmt, [M // 3, 0, M - M // 3], True, K < 28672)


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("K", [72, 520, 4096, 6000, 11008])
def test_products_of_one_token(K, fmt):
    """A token's experts, one place each, and rows that share one although few experts have any; every length of row whose
    operands stay in registers, with outputs for several turns of a workgroup and a part of a block."""
    rng = np.random.default_rng([64, fmt, K])
    for sizes in ([0, 1, 0, 0, 0, 1, 0, 0], [0, 0, 0, 3, 0, 0, 0, 0, 0], [2, 0, 0, 9, 0, 0, 0, 0, 0, 1]):
        R = sum(sizes)
        check_experts(rng, 1, len(sizes), 100, K, fmt, sizes, True, True, rows=np.zeros(R, dtype=np.int32))
        check_experts(rng, R, len(sizes), 100, K, fmt, sizes, False, False)
    check_experts(rng, 1, 4, 13000 if K < 4096 else 2000, K, fmt, [0, 1, 0, 1], True, True, rows=np.zeros(2, dtype=np.int32))


@pytest.mark.parametrize("fmt", [F2, F16])
def test_more_experts_than_lanes(fmt):
    """Tiles of more than 64 experts are listed four to a lane."""
    rng = np.random.default_rng([65, fmt])
    for E in (65, 200, 256):
        for each in (0.1, 2, 5, 40):
            sizes = rng.poisson(each, E)
            sizes[E - 1] = 3
            check_experts(rng, int(sizes.sum()), E, 20, 256, fmt, sizes, False, each == 2)


@pytest.mark.parametrize("fmt", [F2, F16])
def test_products_of_whole_tiles(fmt):
    """Sizes at the edges of the large tiles, in rows and in columns."""
    rng = np.random.default_rng([56, fmt])
    for pair in (False, True):
        check_experts(rng, 640, 2, 1024, 512, fmt, [128, 512], False, pair)
        check_experts(rng, 300, 3, 511, 520, fmt, [127, 129, 1], True, pair)


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("big", [False, True])
def test_places_that_no_expert_owns(fmt, big):
    """Places before the first offset and behind the last, and rows that name no row of X."""
    rng = np.random.default_rng([57, fmt, big])
    sizes = [150, 0, 200, 33] if big else [2, 0, 3, 1]
    n = sum(sizes)
    for pair in (False, True):
        check_experts(rng, n + 20, 4, 96, 264, fmt, sizes, False, pair, R=n + 15, first=6)
        rows = rng.integers(0, 11, n + 15).astype(np.int32)
        rows[[0, 7, n + 3]] = [-1, 11, -(1 << 31)]
        rows[8] = (1 << 31) - 1
        check_experts(rng, 11, 4, 96, 264, fmt, sizes, True, pair, R=n + 15, first=6, rows=rows)


@pytest.mark.parametrize("fmt", [F2, F16])
def test_offsets_past_the_places_are_clamped(fmt):
    rng = np.random.default_rng([58, fmt])
    for R in (5, 100):
        check_experts(rng, R, 3, 64, 256, fmt, [2, R, 40], False, False, R=R)


@pytest.mark.parametrize("fmt", [F2, F16])
def test_offsets_that_decrease_stay_inside(fmt):
    """Offsets against the contract: what is written is unspecified, but only places 0 .. R - 1 are, and the call ends."""
    import torch
    E, N, K = 16, 48, 256
    W = torch.zeros((E, N, tri.tri_row_bytes(K, fmt)), dtype=torch.uint8, device="cuda")
    s = torch.ones(E, device="cuda")
    for R in (1, 7, 100, 1000):
        X = torch.zeros((R, K), dtype=torch.float16, device="cuda")
        for off in ([0, R] * 8 + [0], [R] * 17, [-5, 1 << 30] * 8 + [-(1 << 31)], list(range(16, -1, -1))):
            o = torch.tensor(off, dtype=torch.int32, device="cuda")
            Y = torch.full((R + 64, N), 7.0, dtype=torch.float16, device="cuda")
            say("decreasing offsets R=%d fmt=%d" % (R, fmt))
            tri.tri_experts_linear(X, R, o, None, R, W, s, E, N, K, fmt, Y)
            tri.tri_experts_pair(X, R, o, None, R, W, s, W, s, E, N, K, fmt, Y)
            assert np.all(host(Y)[R:] == 7.0)


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("name", ["one", "few", "hole", "mixed", "single", "many", "long"])
@pytest.mark.parametrize("K", [640, 328, 5632, 129])
def test_rows_that_are_not_finite_spoil_no_other(name, pair, fmt, K):
    """Tokens of NaN and infinities (padding that was routed all the same): other tokens' results keep every bit."""
    import torch
    rng = np.random.default_rng([70, K, fmt, pair])
    sizes, T, N = RAGGED[name], 9, 100
    E, R = len(sizes), sum(sizes)
    rows = rng.integers(0, T, R).astype(np.int32)
    mats = [(tri.pack(cuda(synth.trits(rng, E * N, K)), fmt).view(E, N, -1), torch.full((E,), 0.05, device="cuda"))
            for _ in range(2 if pair else 1)]
    X = rng.standard_normal((T, K)).astype(np.float16)
    off, rd = cuda(places(sizes)), cuda(rows)
    args = [a for m in mats for a in m]
    run = tri.experts_pair if pair else tri.experts_linear
    want = host(run(cuda(X), off, rd, *args, K, fmt))
    X[[1, 4]] = rng.choice(np.array([np.nan, np.inf, -np.inf], dtype=np.float16), (2, K))
    got = host(run(cuda(X), off, rd, *args, K, fmt))
    bad = (rows == 1) | (rows == 4)
    np.testing.assert_array_equal(got[~bad].view(np.uint16), want[~bad].view(np.uint16))
    if not pair:
        assert not np.any(np.isfinite(got[bad]))


def test_experts_of_a_slice():
    """A rank that holds some of the experts: offsets from its first expert on, its own weights, the places of the others
    untouched; the slices together give what one call gives."""
    import torch
    rng = np.random.default_rng(71)
    for T in (3, 40, 300):
        E, topk, K, N = 8, 2, 256, 200
        r = tri.experts_route(cuda(rng.standard_normal((T, E)).astype(np.float32)), topk)
        W = tri.pack(cuda(synth.trits(rng, E * N, K)), F2).view(E, N, -1)
        s = cuda(rng.uniform(0.02, 0.05, E).astype(np.float32))
        X = cuda(rng.standard_normal((T, K)).astype(np.float16))
        parts = torch.full((T * topk, N), float("nan"), dtype=torch.float16, device="cuda")
        off = host(r.offsets)
        for a, b in ((0, 3), (3, 4), (4, 8)):
            before = host(parts)
            tri.experts_linear(X, r.offsets[a:b + 1], r.rows, W[a:b], s[a:b], K, F2, out=parts)
            after, own = host(parts), np.zeros(T * topk, dtype=bool)
            own[off[a]:off[b]] = True
            np.testing.assert_array_equal(after[~own].view(np.uint16), before[~own].view(np.uint16))
        want = host(tri.experts_linear(X, r.offsets, r.rows, W, s, K, F2)).astype(np.float64)
        # two kernels' results: twice the bound of one
        d = sum_bound(K, float(s.max()), host(X)[host(r.rows)].astype(np.float64))
        assert np.all(np.abs(host(parts) - want) <= 2 * (d + 2.0 ** -11 * np.abs(want) + 2.0 ** -25))


@pytest.mark.parametrize("K", [8, 5])
def test_the_most_places_that_one_expert_may_own(K):
    """2^31 - 1 places of one expert out of three: the last tile's bounds stay below 2^31, nothing is lost (small integers:
    every sum is exact)."""
    import torch
    rng = np.random.default_rng([69, K])
    R, T, E, N = (1 << 31) - 1, 5, 3, 1
    W = rng.integers(-1, 2, (E * N, K)).astype(np.int8)
    X = rng.integers(-4, 5, (T, K)).astype(np.float16)
    want = cuda((X.astype(np.float64) @ W[1].astype(np.float64)).astype(np.float16))
    rows = torch.empty(R, dtype=torch.int32, device="cuda")
    step = 1 << 28
    for r in range(0, R, step):
        rows[r:r + step] = torch.arange(r, min(r + step, R), device="cuda") % T
    offsets = torch.tensor([0, 0, R, R], dtype=torch.int32, device="cuda")
    Y = torch.full((R, N), float("nan"), dtype=torch.float16, device="cuda")
    tri.experts_linear(cuda(X), offsets, rows, tri.pack(cuda(W), F2).view(E, N, -1), torch.ones(E, device="cuda"), K,
                       F2, out=Y)
    for r in range(0, R, step):
        assert torch.equal(Y[r:r + step, 0], want[rows[r:r + step].long()]), r


@pytest.mark.parametrize("places", [3, 200])
def test_gathered_rows_near_the_end_of_four_gigabytes(places):
    """X of almost 4 GiB, its rows gathered from both ends, by the kernels of few and of many places."""
    import torch
    rng = np.random.default_rng([66, places])
    K, N = 4096, 40
    T = ((1 << 31) - 8) // K
    X = torch.zeros((T, K), dtype=torch.float16, device="cuda")
    rows = np.concatenate([rng.integers(0, 50, places // 2), T - 1 - rng.integers(0, 50, places - places // 2),
                           [T // 2 - 1, T // 2]]).astype(np.int32)
    x = rng.standard_normal((len(rows), K)).astype(np.float16)
    X[cuda(rows).long()] = cuda(x)               # (of a row named twice, one copy stays)
    W = synth.trits(rng, N, K)
    Wp = tri.pack(cuda(W), F2).view(1, N, -1)
    off = cuda(np.array([0, len(rows)], dtype=np.int32))
    Y = host(tri.experts_linear(X, off, cuda(rows), Wp, torch.full((1,), 0.02, device="cuda"), K, F2)).astype(np.float64)
    x = host(X[cuda(rows).long()]).astype(np.float64)
    ref = float(np.float32(0.02)) * (x @ W.astype(np.float64).T)
    assert np.all(np.abs(Y - ref) <= sum_bound(K, 0.02, x) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)


@pytest.mark.parametrize("M", [1, 3, 40])
def test_weights_past_four_gigabytes(M):
    """The last expert of a stack of more than 4 GiB gives what it gives alone."""
    import torch
    rng = np.random.default_rng([67, M])
    E, N, K = 9, 65536, 32768
    Wp = torch.zeros((E, N, tri.tri_row_bytes(K, F2)), dtype=torch.uint8, device="cuda").fill_(0x55)
    assert Wp.numel() > 1 << 32
    Wp[-1, -100:] = tri.pack(cuda(synth.trits(rng, 100, K)), F2)
    X = cuda(rng.standard_normal((M, K)).astype(np.float16))
    s = torch.full((E,), 0.01, device="cuda")
    all_ = tri.experts_linear(X, cuda(np.array([0] * E + [M], dtype=np.int32)), None, Wp, s, K, F2)
    one = tri.experts_linear(X, cuda(np.array([0, M], dtype=np.int32)), None, Wp[-1:, -100:].contiguous(), s[:1], K, F2)
    a, b = host(all_).astype(np.float64), host(one).astype(np.float64)
    x = host(X).astype(np.float64)
    assert np.all(np.abs(a[:, :-100]) <= sum_bound(K, 0.01, x) + 2.0 ** -25)   # zero trits
    assert np.all(np.abs(a[:, -100:] - b) <= 2 * sum_bound(K, 0.01, x) + 2.0 ** -10 * np.abs(b) + 2.0 ** -24)


def test_one_expert_equals_the_layer():
    """Against tri_linear on the same matrix, within both tolerances, and the packed rows of one tri_pack2 call for all
    experts are those of one call each."""
    import torch
    rng = np.random.default_rng(59)
    W = synth.trits(rng, 96, 512)
    X = rng.standard_normal((20, 512)).astype(np.float16)
    for fmt in (F2, F16):
        whole = tri.pack(cuda(W), fmt)
        each = torch.cat([tri.pack(cuda(W[48 * e:48 * e + 48]), fmt) for e in range(2)])
        assert torch.equal(whole, each)
        s = torch.full((1,), 0.05, device="cuda")
        Y = tri.experts_linear(cuda(X), cuda(places([20])), None, whole.view(1, 96, -1), s, 512, fmt)
        L = host(tri.linear(cuda(X), whole, float(s[0]), 512, fmt)).astype(np.float64)
        ref = oracle.linear_f64(X, W, float(np.float32(0.05)))
        assert np.all(np.abs(host(Y) - L) <= 2 * oracle.tolerance(X, 0.05, ref))


# ---------------------------------------------------------------- combination

def check_combine(Y, Z, pos, weights, residual):
    Z = Z.astype(np.float64)
    ok = (pos >= 0) & (pos < len(Z))
    terms = np.where(ok[..., None], weights.astype(np.float64)[..., None] * Z[np.where(ok, pos, 0)], 0.0)
    ref, mag = terms.sum(1), np.abs(terms).sum(1)
    if residual is not None:
        ref, mag = ref + residual.astype(np.float64), mag + np.abs(residual.astype(np.float64))
    tol = (pos.shape[1] + 2) * 2.0 ** -24 * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    assert np.all(np.abs(Y.astype(np.float64) - ref) <= tol)


@pytest.mark.parametrize("T,topk,N", [(1, 1, 8), (1, 2, 4096), (3, 5, 100), (17, 8, 257), (300, 6, 1024), (5, 16, 33),
                                      (2, 3, 1)])
def test_combine(T, topk, N):
    rng = np.random.default_rng([60, T, topk, N])
    R = T * topk
    Z = rng.standard_normal((R, N)).astype(np.float16)
    w = rng.uniform(-1, 1, (T, topk)).astype(np.float32)
    pos = rng.permutation(R).reshape(T, topk).astype(np.int32)
    res = rng.standard_normal((T, N)).astype(np.float16)
    for r in (None, res):
        check_combine(host(tri.experts_combine(cuda(Z), cuda(pos), cuda(w), residual=None if r is None else cuda(r))), Z,
                      pos, w, r)
    # left out: places outside Z, with whatever lies at their weights; the rows that nobody names may hold anything
    bad = pos.copy()
    bad[0, 0], bad[-1, -1] = -1, R
    bad[0, topk // 2] = -(1 << 31)
    Z[pos[bad != pos]] = np.nan
    w[bad != pos] = np.nan
    Rd = cuda(res)
    out = tri.experts_combine(cuda(Z), cuda(bad), cuda(w), residual=Rd, out=Rd)   # in place
    w[bad != pos] = 0.0
    check_combine(host(out), np.nan_to_num(Z), bad, w, res)


# ---------------------------------------------------------------- together

def mixed_block(rng, T, E, topk, hidden, inner, fmt):
    """A 4-bit layer that gives the router's logits, and an MLP of ternary experts."""
    Wr = tri.int4_quantize(cuda((0.05 * rng.standard_normal((E, hidden))).astype(np.float32)), 64)
    mats = []
    for (n, k) in ((inner, hidden), (inner, hidden), (hidden, inner)):
        W, s = [], []
        for _ in range(E):                       # experts from latent weights, the scales as the quantiser leaves them
            p, sc = tri.quantize(cuda(synth.latent_weights(rng, n, k)), fmt)
            W.append(p)
            s.append(sc)
        import torch
        mats.append((torch.stack(W), torch.cat(s)))
    return Wr, mats


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("T,E,topk,hidden,inner", [(1, 8, 2, 512, 768), (9, 4, 2, 256, 344), (150, 16, 4, 256, 200)])
def test_a_block_of_experts(T, E, topk, hidden, inner, fmt):
    """All four operators as a block uses them; each step is checked on what the step before gave."""
    rng = np.random.default_rng([61, T, E, fmt])
    Wr, (gate, up, down) = mixed_block(rng, T, E, topk, hidden, inner, fmt)
    X = rng.standard_normal((T, hidden)).astype(np.float16)
    Xd = cuda(X)
    logits = tri.int4_linear(Xd, Wr, E, 64)
    Y = tri.experts_mlp(Xd, logits, topk, gate, up, down, fmt, residual=Xd)
    r = tri.experts_route(logits, topk)
    H = tri.experts_pair(Xd, r.offsets, r.rows, *gate, *up, hidden, fmt)
    Z = tri.experts_linear(H, r.offsets, None, *down, inner, fmt)
    assert np.array_equal(host(tri.experts_combine(Z, r.pos, r.weights, residual=Xd)).view(np.uint16),
                          host(Y).view(np.uint16))
    ids, weights, offsets, rows, pos = route_ref(host(logits), topk, True)
    np.testing.assert_array_equal(host(r.ids), ids)
    np.testing.assert_array_equal(host(r.pos), pos)
    dense = [[oracle.unpack(host(W[e]), k, fmt).astype(np.float64) * float(s[e]) for e in range(E)]
             for (W, s), k in zip((gate, up, down), (hidden, hidden, inner))]
    H, Z = host(H).astype(np.float64), host(Z).astype(np.float64)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        x = X[rows[a:b]].astype(np.float64)
        g, u = x @ dense[0][e].T, x @ dense[1][e].T
        h = g / (1 + np.exp(-g)) * u
        dg, du = (sum_bound(hidden, float(m[1][e]), x) for m in (gate, up))
        tol = 1.1 * dg * np.abs(u) + np.abs(g) * du + 1.1 * dg * du + (2.0 ** -18 + 2.0 ** -11) * np.abs(h) + 2.0 ** -25
        assert np.all(np.abs(H[a:b] - h) <= tol)
        z = H[a:b] @ dense[2][e].T
        assert np.all(np.abs(Z[a:b] - z) <= sum_bound(inner, float(down[1][e]), H[a:b]) + 2.0 ** -11 * np.abs(z) + 2.0 ** -25)
    check_combine(host(Y), Z, pos, host(r.weights), X)


def test_graph_replays_equal_eager_calls():
    """The block captured once and replayed on new inputs, with eager work between the replays."""
    import torch
    rng = np.random.default_rng(62)
    T, E, topk, hidden, inner = 100, 8, 2, 256, 384
    Wr, (gate, up, down) = mixed_block(rng, T, E, topk, hidden, inner, F2)
    X = torch.empty((T, hidden), dtype=torch.float16, device="cuda")
    ws = torch.empty(tri.tri_experts_route_workspace_bytes(T, E, topk), dtype=torch.uint8, device="cuda")
    mk = lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")
    logits, H, Z, Y = mk(T, E), mk(T * topk, inner), mk(T * topk, hidden), mk(T, hidden)
    r = tri.Routing(mk(T, topk, d=torch.int32), mk(T, topk, d=torch.float32), mk(E + 1, d=torch.int32),
                    mk(T * topk, d=torch.int32), mk(T, topk, d=torch.int32))

    def step():
        tri.int4_linear(X, Wr, E, 64, out=logits)
        tri.experts_route(logits, topk, workspace=ws, out=r)
        tri.experts_pair(X, r.offsets, r.rows, *gate, *up, hidden, F2, out=H)
        tri.experts_linear(H, r.offsets, None, *down, inner, F2, out=Z)
        tri.experts_combine(Z, r.pos, r.weights, residual=X, out=Y)

    def inputs(seed):
        X.copy_(torch.randn(X.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).half())

    inputs(0)
    step()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    outs = lambda: [t.clone() for t in (logits, H, Z, Y) + tuple(r)]
    for seed in (1, 2, 3):
        inputs(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = outs()
        step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, outs())):
            assert torch.equal(a, b), "replay %d, output %d" % (seed, i)
    del graph


def test_two_streams_at_once():
    """Two blocks on two streams, with the workspaces and intermediate results that the helpers allocate."""
    import torch
    rng = np.random.default_rng(63)
    T, E, topk, hidden, inner = 200, 8, 2, 256, 384
    Wr, (gate, up, down) = mixed_block(rng, T, E, topk, hidden, inner, F16)
    Xs = [cuda(rng.standard_normal((T, hidden)).astype(np.float16)) for _ in range(2)]

    def step(X, stream=None):
        return tri.experts_mlp(X, tri.int4_linear(X, Wr, E, 64, stream=stream), topk, gate, up, down, F16, stream=stream)

    want = [step(X).clone() for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [step(X, s) for X, s in zip(Xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_results_of_a_named_stream_outlive_their_tensors():
    """Helpers that allocate and run on a stream that is not the current one: memory that the caller lets go while that
    stream is still at work is not handed to the current stream's next allocation."""
    import torch
    rng = np.random.default_rng(68)
    T, E, topk, hidden, inner = 300, 8, 2, 256, 384
    Wr, (gate, up, down) = mixed_block(rng, T, E, topk, hidden, inner, F2)
    X = cuda(rng.standard_normal((T, hidden)).astype(np.float16))
    want = tri.experts_mlp(X, tri.int4_linear(X, Wr, E, 64), topk, gate, up, down, F2).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        Y = tri.experts_mlp(X, tri.int4_linear(X, Wr, E, 64, stream=s), topk, gate, up, down, F2, stream=s)
        for n in (T * topk * inner, T * topk * hidden, T * hidden, T * E):   # sizes of what was let go
            torch.full((n,), float("nan"), dtype=torch.float16, device="cuda")
        got.append(Y)
    torch.cuda.synchronize()
    for Y in got:
        assert torch.equal(Y, want)


def test_refusals_of_the_helpers():
    import torch
    h, i, u, f = (dict(dtype=d, device="cuda") for d in (torch.float16, torch.int32, torch.uint8, torch.float32))
    x, off, rows, s = torch.zeros((4, 64), **h), torch.zeros(3, **i), torch.zeros(5, **i), torch.zeros(2, **f)
    W = torch.zeros((2, 16, 16), **u)
    tri.experts_linear(x, off, rows, W, s, 64, F2)
    for bad in [lambda: tri.experts_linear(x, off.long(), rows, W, s, 64, F2),
                lambda: tri.experts_linear(x, off[:2], rows, W, s, 64, F2),
                lambda: tri.experts_linear(x, off, rows.long(), W, s, 64, F2),
                lambda: tri.experts_linear(x, off, rows, W, s.double(), 64, F2),
                lambda: tri.experts_linear(x, off, rows, W, s[:1], 64, F2),
                lambda: tri.experts_linear(x, off, rows, W, s, 128, F2),
                lambda: tri.experts_linear(x, off, rows, W, s, 64, F2, out=torch.zeros((4, 16), **h)),
                lambda: tri.experts_linear(x, off, rows, W.view(32, 16), s, 64, F2),
                lambda: tri.experts_pair(x, off, rows, W, s, torch.zeros((2, 17, 16), **u), s, 64, F2),
                lambda: tri.experts_route(x, 0), lambda: tri.experts_route(x, 17), lambda: tri.experts_route(x.double(), 2),
                lambda: tri.experts_route(x.t(), 2), lambda: tri.experts_route(torch.zeros((4, 300), **h), 2),
                lambda: tri.experts_combine(x, rows.view(1, 5), torch.zeros((1, 4), **f)),
                lambda: tri.experts_combine(x, rows.view(1, 5), torch.zeros((1, 5), **h)),
                lambda: tri.experts_combine(x, rows.view(1, 5), torch.zeros((1, 5), **f), out=torch.zeros((2, 64), **h))]:
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("T", [3, 5])
def test_a_block_refuses_logits_of_other_tokens(T):
    import torch
    rng = np.random.default_rng(72)
    _, mats = mixed_block(rng, 4, 8, 2, 256, 384, F2)
    X = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        tri.experts_mlp(X, torch.zeros((T, 8), device="cuda"), 2, *mats, F2)


SUMS = {"one place": [0, 1, 0, 0, 0, 0, 1, 0, 0], "three places": [2, 1], "eight places": [3, 5], "seventy places": [30, 40],
        "many places": [200]}


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("name", list(SUMS))
@pytest.mark.parametrize("K", [256, 1001, 4096, 11008, 28672])
def test_sums_are_those_of_fp32(K, name, fmt):
    """How far the sums are off before they are rounded, over all outputs at once (the bound of single outputs above lets
    every rounding fall the same way).  A sum that is off by d moves a result to a neighbouring fp16 value with probability
    d / step, so the mean distance from the correctly rounded results, in steps, is the mean of d / step.  d by the model of
    independent roundings: 80 + K/16 additions, each off by at most 2^-23 of a partial sum of digits t + 1, whose size is the
    root of sum_k (t+1)^2 x^2; twice its root mean square, 2 sqrt(80 + K/16) 2^-23 of that.  Results below 1/16 of their root
    mean square (6%) are left out, their steps are too fine; 1/200 is added for chance, four deviations of 8000 results'
    share at 1%."""
    rng = np.random.default_rng([73, K, fmt, list(SUMS).index(name)])
    sizes, N = SUMS[name], 4000
    E, R = len(sizes), sum(sizes)
    X = rng.standard_normal((R, K)).astype(np.float16)
    W = synth.trits(rng, N, K)
    mats = tri.pack(cuda(W), fmt).expand(E, N, -1).contiguous()
    say("sums K=%d fmt=%d %s" % (K, fmt, name))
    Y = host(tri.experts_linear(cuda(X), cuda(places(sizes)), None, mats, cuda(np.full(E, 1 / 64, np.float32)), K, fmt))
    x = X.astype(np.float64)
    ref = x @ W.astype(np.float64).T / 64
    size = np.sqrt((x * x) @ ((W + 1.0) ** 2).T) / 64
    near = ref.astype(np.float16)
    step = np.spacing(np.abs(near)).astype(np.float64)
    live = np.abs(ref) > np.sqrt(np.mean(ref * ref)) / 16
    off = np.abs(Y.astype(np.float64) - near.astype(np.float64)) / step
    d = 2 * np.sqrt(80 + K / 16) * 2.0 ** -23 * size
    say("  mean distance %.5f steps, %.5f allowed" % (off[live].mean(), (d / step)[live].mean() + 0.005))
    assert off[live].mean() <= (d / step)[live].mean() + 0.005


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("K", [5, 8])
def test_the_most_outputs_of_a_product(K, fmt):
    """2^27 - 16 outputs, the last that are taken, by the kernel of a workgroup per 16 outputs (K = 5) and the resident grid
    (K = 8): rows that repeat, small integers, so that every result is exact."""
    import torch
    rng = np.random.default_rng([74, K, fmt])
    N, n = (1 << 27) - 16, 1 << 12
    W = rng.integers(-1, 2, (n, K)).astype(np.int8)
    X = rng.integers(-4, 5, (1, K)).astype(np.float16)
    Wp = tri.pack(cuda(W), fmt).repeat(N // n + 1, 1)[:N].view(1, N, -1)
    want = cuda((X.astype(np.float64) @ W.T.astype(np.float64)).astype(np.float16)[0])
    say("outputs N=%d K=%d fmt=%d" % (N, K, fmt))
    Y = torch.full((1, N), float("nan"), dtype=torch.float16, device="cuda")
    tri.experts_linear(cuda(X), cuda(places([1])), None, Wp, torch.ones(1, device="cuda"), K, fmt, out=Y)
    assert torch.equal(Y[0], want.repeat(N // n + 1)[:N])
