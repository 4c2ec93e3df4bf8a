"""The 4-bit and experts' products on small integers: every partial sum is an integer below 2^24, exact in fp32 in any order,
and a result is that integer rounded once.  So results are compared bit for bit, and one weight or activation left out, read
twice or put in another column shows, however long the row.

Only the gated pair has a tolerance: its gate and up sums are exact, exp, the division and two products are within 2^-18,
and the result is rounded to fp16 once, half a step: (2^-18 + 2^-11) |Y_ref| + 2^-25."""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu
F2, F16 = tri.TRI_FMT_2BIT, tri.TRI_FMT_1P6BIT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


def integers(seed, lo, hi, shape, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, device="cuda", generator=g, dtype=torch.int8).to(dtype)


def products(X, Ws, sizes, N):
    """float64 sums (R, N) of every matrix: the rows of X in order, sizes[e] of them with W[e][:N]."""
    import torch
    out = [torch.zeros((X.shape[0], N), dtype=torch.float64, device="cuda") for _ in Ws]
    r = 0
    for e, n in enumerate(sizes):
        if n:
            for o, W in zip(out, Ws):
                o[r:r + n] = X[r:r + n].float() @ W[e, :N].float().t()   # (integers below 2^24)
        r += n
    return out


def check(X, Ws, sums, sizes, N, K, fmt, gather, what):
    """One product (or pair) over the first N outputs of every expert."""
    import torch
    E, R = len(sizes), X.shape[0]
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    Wp = [tri.pack(W[:, :N].reshape(E * N, K).contiguous(), fmt).view(E, N, -1) for W in Ws]
    if gather:                                   # the rows of X in another order
        order = torch.randperm(R, device="cuda", generator=torch.Generator(device="cuda").manual_seed(R))
        Xg, rows = torch.empty_like(X), order.to(torch.int32)
        Xg[order] = X
        X = Xg
    else:
        rows = None
    Y = torch.full((R + 2, N), 7.0, dtype=torch.float16, device="cuda")
    say("exact", what, "N=%d K=%d fmt=%d R=%d of %d, %d matrices" % (N, K, fmt, R, E, len(Ws)))
    if len(Ws) == 1:
        tri.experts_linear(X, off, rows, Wp[0], torch.ones(E, device="cuda"), K, fmt, out=Y)
        assert torch.equal(Y[:R], sums[0][:, :N].half()), what
    else:
        s = torch.full((E,), 1 / 64, device="cuda")
        tri.experts_pair(X, off, rows, Wp[0], s, Wp[1], s, K, fmt, out=Y)
        g, u = sums[0][:, :N] / 64, sums[1][:, :N] / 64
        ref = g / (1 + torch.exp(-g)) * u
        assert bool(((Y[:R].double() - ref).abs() <= (2.0 ** -18 + 2.0 ** -11) * ref.abs() + 2.0 ** -25).all()), what
    assert bool((Y[R:] == 7.0).all())


# 64 tiles of each height: with one, two or three workgroups per CU a tile has 4, 8 or 12 of them, so a workgroup takes from
# 15 to 17 of these blocks somewhere among each four (results are written 15 or 16 at a time), and up to 128.
BLOCKS = [57, 60, 61, 64, 65, 68, 69, 113, 120, 121, 124, 128, 129, 136, 137, 169, 180, 181, 192, 193, 204, 205, 257]
HEIGHTS = {1: [1, 0] * 64, 8: [2] * 64, 16: [4] * 64}


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("height", list(HEIGHTS))
@pytest.mark.parametrize("K,most", [(264, 513), (2568, 257), (5000, 137), (10248, 69)])
def test_many_blocks_per_workgroup(K, most, height, pair, fmt):
    sizes = HEIGHTS[height]
    E, R, N = len(sizes), sum(sizes), 16 * most
    import torch
    X = integers(K + height, -2, 2, (R, K), torch.float16)
    Ws = [integers(7 * K + q, -1, 1, (E, N, K), torch.int8) for q in range(2 if pair else 1)]
    sums = products(X, Ws, sizes, N)
    for nb in [b for b in BLOCKS + [513] if b <= most]:
        for n in (16 * nb, 16 * nb - 7):
            check(X, Ws, sums, sizes, n, K, fmt, nb % 2 == 0, "blocks=%d" % nb)


LONG = [1001, 2048, 2049, 4096, 4104, 6144, 8192, 8200, 10240, 10248, 11005, 11008, 12288, 12296, 12800, 12808, 14336, 28672]
SIZES = {"one place each": [1, 0, 0, 1, 0, 0], "few": [3, 0, 1], "some": [7, 5], "sixteen": [16, 15], "forty": [40, 33],
         "many": [150]}


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("K", LONG)
def test_every_weight_counts(K, name, fmt):
    """Rows at the edges of every number of steps that a wave may take, and between them."""
    sizes, N = SIZES[name], 130
    import torch
    X = integers(K + len(name), -2, 2, (sum(sizes), K), torch.float16)
    Ws = [integers(K + 50 + q, -1, 1, (len(sizes), N, K), torch.int8) for q in range(2)]
    sums = products(X, Ws, sizes, N)
    check(X, Ws[:1], sums[:1], sizes, N, K, fmt, False, name)
    check(X, Ws[:1], sums[:1], sizes, N, K, fmt, True, name)
    check(X, Ws, sums, sizes, N, K, fmt, True, name)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 16, 33, 70])
def test_every_code_counts(M, group, zeros):
    """4-bit layers, scales of one: rows of one step and of many, whole and not, in few and in many blocks."""
    import torch
    for (N, K) in [(130, 128), (130, 129), (300, 1000), (20500, 264), (130, 4099), (4100, 4096), (130, 11008), (130, 28672)]:
        X = integers(K + M, -2, 2, (M, K), torch.float16)
        Q = integers(K + 1, 0, 15, (N, K), torch.uint8)
        G = -(-K // group)
        Z = integers(K + 2, 0, 15, (N, G), torch.uint8) if zeros else None
        S = torch.ones((N, G), dtype=torch.float16, device="cuda")
        W = Q.float() - (8.0 if Z is None else Z.float().repeat_interleave(group, 1)[:, :K])
        say("exact int4 M=%d N=%d K=%d group=%d zeros=%d" % (M, N, K, group, zeros))
        Y = tri.int4_linear(X, tri.int4_pack(Q, S, group, Z), N, group, zeros)
        assert torch.equal(Y, (X.float() @ W.t()).half()), (N, K)   # (integers below 2^24; past 65504: infinities)


@pytest.mark.parametrize("fmt", [F2, F16])
@pytest.mark.parametrize("K", [520, 129])
@pytest.mark.parametrize("name", ["one place each", "few", "sixteen", "many"])
def test_gates_of_any_size(name, K, fmt):
    """Gates up to thousands of either sign: exp of the negative ones passes fp32, and their results are zeros.  (exp's
    argument is off by 2^-24 of the gate, which weighs where the gate's result is not yet nothing: up to 2^-18 at 64; past
    -64 the result is below 2^-80.)"""
    import torch
    sizes, N = SIZES[name], 100
    E, R = len(sizes), sum(sizes)
    X = integers(K + R, -2, 2, (R, K), torch.float16)
    Ws = [integers(K + 70 + q, -1, 1, (E, N, K), torch.int8) for q in range(2)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    Wp = [tri.pack(W.reshape(E * N, K), fmt).view(E, N, -1) for W in Ws]
    sums = products(X, Ws, sizes, N)
    for gate in (1 / 4, 4.0, 64.0):
        say("gates", name, K, fmt, gate)
        Y = tri.experts_pair(X, off, None, Wp[0], torch.full((E,), gate, device="cuda"), Wp[1],
                             torch.full((E,), 1 / 256, device="cuda"), K, fmt)
        g, u = sums[0] * gate, sums[1] / 256
        ref = g / (1 + torch.exp(-g)) * u
        assert bool(((Y.double() - ref).abs() <= (2.0 ** -17 + 2.0 ** -11) * ref.abs() + 2.0 ** -25).all())
