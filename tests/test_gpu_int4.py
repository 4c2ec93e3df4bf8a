"""4-bit layers with group scales on the GPU, against the definition in float64.

Tolerance of a product.  Codes minus zero points are exact, products of two fp16 values are exact in fp32, and a sum's
term passes at most 32 additions inside a matrix instruction, one per later instruction on the same accumulator (K/32 at
most), its scaling and 48 additions of partial sums; each is off by at most 2^-23 relative to the terms' magnitudes (a
truncating adder).  The result is rounded to fp16 once: half a step, 2^-11 relative, or 2^-25 among subnormals.
    |Y - Y_ref| <= (81 + K/32) 2^-23 (sum_k |W X| + |residual|) + 2^-11 |Y_ref| + 2^-25
"""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests.gpu_helpers import say, cuda, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


def matrix(rng, N, K, group, zeros):
    G = -(-K // group)
    Q = rng.integers(0, 16, (N, K), dtype=np.uint8)
    S = (rng.uniform(0.5, 1.5, (N, G)) * 0.01 * rng.choice([-1.0, 1.0], (N, G))).astype(np.float16)
    S[rng.random((N, G)) < 0.02] = 0
    Z = rng.integers(0, 16, (N, G), dtype=np.uint8) if zeros else None
    return Q, S, Z


def dense(Q, S, Z, group):
    K = Q.shape[1]
    rep = lambda v: np.repeat(v.astype(np.float64), group, axis=1)[:, :K]
    return rep(S) * (Q.astype(np.float64) - (8.0 if Z is None else rep(Z)))


def check(Y, X, W, residual=None, what=""):
    X, K = X.astype(np.float64), X.shape[1]
    ref, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    if residual is not None:
        ref, mag = ref + residual.astype(np.float64), mag + np.abs(residual.astype(np.float64))
    tol = (81 + K / 32) * 2.0 ** -23 * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    err = np.abs(Y.astype(np.float64) - ref)
    assert np.all(err <= tol), "%s: worst %.3g of the tolerance at %s" % (
        what, np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))


def stored(Q, S, Z, group):
    """The layout of include/tri.h, written out value by value."""
    N, K = Q.shape
    nb, ks, gps = -(-N // 16), -(-K // 128), 128 // group
    codes = np.zeros(nb * ks * 256, dtype=np.uint32)
    scales = np.zeros(nb * ks * 16 * gps, dtype=np.float16)
    zeros = np.full(nb * ks * 16 * gps, 8, dtype=np.uint8)
    for n in range(nb * 16):
        for k in range(ks * 128):
            b, j, s, p, g, i = n // 16, n % 16, k // 128, k % 128 // 32, k % 32 // 8, k % 8
            q = int(Q[n, k]) if n < N and k < K else 8
            codes[((b * ks + s) * 64 + 16 * g + j) * 4 + p] |= np.uint32(q << (4 * (i // 2) + 16 * (i % 2)))
    for n in range(N):
        for i in range(S.shape[1]):
            at = ((n // 16 * ks + i // gps) * 16 + n % 16) * gps + i % gps
            scales[at] = S[n, i]
            if Z is not None:
                zeros[at] = Z[n, i]
    parts = [codes.view(np.uint8), scales.view(np.uint8)] + ([zeros] if Z is not None else [])
    return np.concatenate(parts)


@pytest.mark.parametrize("N,K", [(16, 128), (1, 1), (17, 129), (33, 300), (5, 1000)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_layout_and_its_inverse(N, K, group, zeros):
    rng = np.random.default_rng([41, N, K, group, zeros])
    Q, S, Z = matrix(rng, N, K, group, zeros)
    Wp = tri.int4_pack(cuda(Q | (rng.integers(0, 16, Q.shape, dtype=np.uint8) << 4)), cuda(S), group,
                       None if Z is None else cuda(Z))
    np.testing.assert_array_equal(host(Wp), stored(Q, S, Z, group))
    q, s, z = tri.int4_unpack(Wp, N, K, group, zeros)
    np.testing.assert_array_equal(host(q), Q)
    np.testing.assert_array_equal(host(s).view(np.uint16), S.view(np.uint16))
    assert (z is None) == (Z is None)
    if zeros:
        np.testing.assert_array_equal(host(z), Z)


@pytest.mark.parametrize("N,K", [(16, 128), (3, 1), (40, 333), (64, 2048)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize(N, K, group, zeros):
    """Bit for bit the rule of include/tri.h, evaluated in float32."""
    rng = np.random.default_rng([42, N, K, group, zeros])
    W = (0.02 * rng.standard_normal((N, K))).astype(np.float32)
    if N > 16:
        W[0, :] = 0.0                            # groups of zeros
        W[1, :] = 1e-9                           # a scale that rounds to zero
        W[2, :] = 1e6                            # one that fp16 does not hold
        W[3, :] = np.abs(W[3, :])                # one sign only
        W[4, :] = -np.abs(W[4, :])
    G = -(-K // group)
    f = np.float32
    pad = np.zeros((N, G * group), dtype=f)
    pad[:, :K] = W
    g = pad.reshape(N, G, group)
    lo, hi = np.minimum(g.min(2), f(0)), np.maximum(g.max(2), f(0))
    top = (hi - lo) / f(15) if zeros else np.abs(g).max(2) / f(7)
    S = np.minimum(top, f(65504)).astype(np.float16)
    sf = S.astype(f)
    with np.errstate(divide="ignore", invalid="ignore"):
        Z = np.where(sf > 0, np.clip(np.rint(-lo / sf), 0, 15), 8) if zeros else np.full((N, G), 8)
        r = np.rint(g / sf[..., None])
    Q = np.clip(r + Z[..., None], 0, 15)
    Q = np.where(sf[..., None] > 0, Q, 8).reshape(N, -1)[:, :K].astype(np.uint8)
    q, s, z = tri.int4_unpack(tri.int4_quantize(cuda(W), group, zeros), N, K, group, zeros)
    np.testing.assert_array_equal(host(s).view(np.uint16), S.view(np.uint16))
    if zeros:
        np.testing.assert_array_equal(host(z), Z.astype(np.uint8))
    np.testing.assert_array_equal(host(q), Q)


SHAPES = [(16, 128), (256, 512), (1, 1), (7, 33), (100, 1000), (333, 640), (50, 1001), (2000, 4096), (48, 11008),
          (24, 28672)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 130])
def test_product(M, N, K):
    """Every group size and both kinds of zero points at every number of rows and shape."""
    rng = np.random.default_rng([43, M, N, K])
    X = rng.standard_normal((M, K)).astype(np.float16)
    Xd = cuda(X)
    for group in (32, 64, 128):
        for zeros in (False, True):
            Q, S, Z = matrix(rng, N, K, group, zeros)
            Wp = tri.int4_pack(cuda(Q), cuda(S), group, None if Z is None else cuda(Z))
            say("int4 M=%d N=%d K=%d group=%d zeros=%d" % (M, N, K, group, zeros))
            Y = tri.int4_linear(Xd, Wp, N, group, zeros)
            check(host(Y), X, dense(Q, S, Z, group), what="M=%d N=%d K=%d group=%d zeros=%d" % (M, N, K, group, zeros))


@pytest.mark.parametrize("M,N", [(20, 20500), (33, 20500), (100, 6500), (130, 20490), (600, 2100)])
@pytest.mark.parametrize("K", [128, 264, 1024, 1160])
def test_product_of_many_tiles(M, N, K):
    """Enough row and column tiles for the kernel whose waves share their activations: both of its tile heights, rows and
    columns that end inside a tile, rows of one step, of whole steps and of a part."""
    rng = np.random.default_rng([47, M, N, K])
    X = rng.standard_normal((M, K)).astype(np.float16)
    R = rng.standard_normal((M, N)).astype(np.float16)
    Xd, Rd = cuda(X), cuda(R)
    for group, zeros in ((32, True), (64, False), (128, True), (32, False), (64, True), (128, False)):
        Q, S, Z = matrix(rng, N, K, group, zeros)
        Wp = tri.int4_pack(cuda(Q), cuda(S), group, None if Z is None else cuda(Z))
        say("int4 M=%d N=%d K=%d group=%d zeros=%d" % (M, N, K, group, zeros))
        res = zeros and group == 64
        Y = tri.int4_linear(Xd, Wp, N, group, zeros, residual=Rd if res else None)
        check(host(Y), X, dense(Q, S, Z, group), R if res else None, what="M=%d N=%d K=%d group=%d zeros=%d" % (M, N, K, group, zeros))


@pytest.mark.parametrize("M,N", [(1, 300), (6, 300), (16, 300), (40, 300), (70, 20500)])
def test_residual_and_in_place(M, N):
    rng = np.random.default_rng([44, M])
    K, group = 768, 64
    Q, S, Z = matrix(rng, N, K, group, True)
    X, R = rng.standard_normal((M, K)).astype(np.float16), rng.standard_normal((M, N)).astype(np.float16)
    Wp, Xd, Rd = tri.int4_pack(cuda(Q), cuda(S), group, cuda(Z)), cuda(X), cuda(R)
    Y = tri.int4_linear(Xd, Wp, N, group, True, residual=Rd)
    check(host(Y), X, dense(Q, S, Z, group), R)
    tri.int4_linear(Xd, Wp, N, group, True, residual=Rd, out=Rd)
    np.testing.assert_array_equal(host(Rd).view(np.uint16), host(Y).view(np.uint16))


@pytest.mark.parametrize("M", [1, 5, 16, 70])
def test_extreme_values(M):
    """Activations up to fp16's largest, subnormal scales, results past fp16 (which become infinities)."""
    rng = np.random.default_rng([45, M])
    N, K, group = 64, 256, 32
    Q, S, Z = matrix(rng, N, K, group, True)
    S[:16] = np.float16(6e-8)                    # the smallest subnormal
    S[16:32] = np.float16(60000.0)
    X = rng.standard_normal((M, K)).astype(np.float16)
    X[:, :7] = np.float16(65504.0)
    X[0, :] *= np.float16(2.0 ** -20)            # subnormal activations
    Y = host(tri.int4_linear(cuda(X), tri.int4_pack(cuda(Q), cuda(S), group, cuda(Z)), N, group, True))
    W = dense(Q, S, Z, group)
    ref, mag = X.astype(np.float64) @ W.T, np.abs(X.astype(np.float64)) @ np.abs(W).T
    tol = (81 + K / 32) * 2.0 ** -23 * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    big = np.abs(ref) - tol > 65520.0            # rounds to an infinity whatever the error
    assert np.all(np.isinf(Y[big])) and np.all(np.sign(Y[big]) == np.sign(ref[big]))
    fits = np.abs(ref) + tol < 65504.0
    assert np.all(np.abs(Y[fits].astype(np.float64) - ref[fits]) <= tol[fits])


@pytest.mark.parametrize("M,N", [(2, 300), (4, 300), (7, 300), (16, 300), (40, 300), (40, 20500), (70, 20500)])
@pytest.mark.parametrize("K", [256, 264, 129])
def test_rows_that_are_not_finite_spoil_no_other(M, N, K):
    """A padded batch whose padding holds NaN and infinities: the other rows' results keep every bit."""
    rng = np.random.default_rng([50, M, N, K])
    Q, S, Z = matrix(rng, N, K, 64, True)
    Wp = tri.int4_pack(cuda(Q), cuda(S), 64, cuda(Z))
    X = rng.standard_normal((M, K)).astype(np.float16)
    want = host(tri.int4_linear(cuda(X), Wp, N, 64, True))
    bad = np.arange(M) % 3 == 1
    X[bad] = rng.choice(np.array([np.nan, np.inf, -np.inf], dtype=np.float16), (int(bad.sum()), K))
    got = host(tri.int4_linear(cuda(X), Wp, N, 64, True))
    np.testing.assert_array_equal(got[~bad].view(np.uint16), want[~bad].view(np.uint16))
    assert not np.any(np.isfinite(got[bad]))


@pytest.mark.parametrize("M", [1, 7, 40])
def test_weights_past_four_gigabytes(M):
    """The last blocks of the largest matrix, whose scales lie past 4 GiB, give what they give alone."""
    import torch
    rng = np.random.default_rng([48, M])
    N, K, group = (1 << 20) - 16, 8192, 128
    assert tri.tri_int4_bytes(N + 16, K, group, False) == -1
    nb, ks = N // 16, K // 128
    Wp = torch.zeros(tri.tri_int4_bytes(N, K, group, False), dtype=torch.uint8, device="cuda")
    n = 64
    Q, S, _ = matrix(rng, n, K, group, False)
    small = tri.int4_pack(cuda(Q), cuda(S), group)
    codes, scales = n // 16 * ks * 1024, n // 16 * ks * 32
    assert Wp.numel() > 1 << 32 and small.numel() == codes + scales
    Wp[nb * ks * 1024 - codes:nb * ks * 1024] = small[:codes]
    Wp[Wp.numel() - scales:] = small[codes:]
    X = rng.standard_normal((M, K)).astype(np.float16)
    Y = host(tri.int4_linear(cuda(X), Wp, N, group))
    check(Y[:, -n:], X, dense(Q, S, None, group))
    assert np.all(Y[:, :-n] == 0.0)


def test_more_rows_than_one_launch_takes():
    """An output of more than 2^22 tiles of 32 x 128 (34 GB) is made by several launches: rows at their seam and the last."""
    import torch
    rng = np.random.default_rng(49)
    N, K, group = 1 << 16, 128, 128
    seam = (1 << 22) // (N // 128) * 32
    M = seam + 40
    Q, S, _ = matrix(rng, N, K, group, False)
    X = rng.standard_normal((M, K)).astype(np.float16)
    out = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    tri.int4_linear(cuda(X), tri.int4_pack(cuda(Q), cuda(S), group), N, group, out=out)
    for m0 in range(0, M, 1 << 14):
        assert not bool(out[m0:m0 + (1 << 14)].isnan().any())
    rows = np.r_[0:3, seam - 20:seam, seam:M]
    check(host(out[torch.from_numpy(rows).cuda()]), X[rows], dense(Q, S, None, group))


def test_rows_behind_the_output_are_untouched():
    """Only M x N values are written, and only the codes of N rows count."""
    import torch
    rng = np.random.default_rng(46)
    for (M, N, K) in [(1, 37, 200), (5, 37, 200), (20, 37, 200)]:
        Q, S, Z = matrix(rng, N, K, 128, False)
        X = rng.standard_normal((M, K)).astype(np.float16)
        buf = torch.full((M * N + 64,), 7.0, dtype=torch.float16, device="cuda")
        tri.tri_int4_linear(cuda(X), tri.int4_pack(cuda(Q), cuda(S), 128), M, N, K, 128, False, None, buf)
        got = host(buf)
        assert np.all(got[M * N:] == 7.0)
        check(got[:M * N].reshape(M, N), X, dense(Q, S, Z, 128))


def test_refusals_of_the_helpers():
    import torch
    h, u = dict(dtype=torch.float16, device="cuda"), dict(dtype=torch.uint8, device="cuda")
    X, Wp = torch.zeros((2, 64), **h), torch.zeros(tri.tri_int4_bytes(16, 64, 32, False), **u)
    tri.int4_linear(X, Wp, 16, 32)
    for bad in [lambda: tri.int4_linear(X.float(), Wp, 16, 32), lambda: tri.int4_linear(X, Wp[:-1], 16, 32),
                lambda: tri.int4_linear(X, Wp, 16, 32, zeros=True), lambda: tri.int4_linear(X, Wp, 17, 32),
                lambda: tri.int4_linear(X, Wp, 16, 48), lambda: tri.int4_linear(torch.zeros((2, 200), **h), Wp, 16, 32),
                lambda: tri.int4_linear(torch.zeros((64, 2), **h).t(), Wp, 16, 32),
                lambda: tri.int4_linear(X, Wp, 16, 32, out=torch.zeros((2, 17), **h)),
                lambda: tri.int4_linear(X, Wp, 16, 32, residual=torch.zeros((1, 16), **h)),
                lambda: tri.int4_linear(torch.zeros((0, 64), **h), Wp, 16, 32),
                lambda: tri.int4_pack(torch.zeros((4, 64), **u), torch.zeros((4, 1), **h), 32),
                lambda: tri.int4_pack(torch.zeros((4, 64), **u), torch.zeros((4, 2), **h), 32, torch.zeros((4, 3), **u)),
                lambda: tri.int4_quantize(torch.zeros((4, 64), **h), 32),
                lambda: tri.int4_unpack(Wp, 16, 640, 32)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tri.TriError):            # the second row of a one-column tensor: not 16-byte aligned
        tri.int4_linear(torch.zeros((3, 1), **h)[1:], torch.zeros(tri.tri_int4_bytes(16, 1, 32, False), **u), 16, 32)
