"""Host-side refusals of the heads' and the cache's entry points: bad arguments are rejected before anything is launched (no
GPU needed; the addresses are fake and must not be touched)."""
import ctypes

import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from tests import cache_ref as ref

A, B, C, D, ODD = 4096, 8192, 12288, 16384, 4097
BIG = 1 << 31
EINVAL, EALIGN = tri.TRI_EINVAL, tri.TRI_EALIGN
NAN = float("nan")


def raw(name, *args):
    return getattr(tri.lib(), name)(*args)


def heads(**kw):
    v = dict(X=A, Y=B, gain=None, x_stride=512, y_stride=512, heads=4, **{})
    return tri.TriHeads(**{**v, **kw})


def rotary(**kw):
    return tri.TriRotary(**{**dict(table=C, rows=100, dims=128, interleaved=0, norm=1, eps=1e-5), **kw})


def cache(**kw):
    return tri.TriCache(**{**dict(K=A, V=B, K_scale=C, V_scale=D, pages=10, heads=4, dim=128, page=64, fmt=0), **kw})


def seqs(**kw):
    return tri.TriSequences(**{**dict(offsets=A, lens=B, table=C, B=3, width=5, max_new=1, max_len=300), **kw})


def at(s):
    return None if s is None else ctypes.addressof(s)


BAD_HEADS = [dict(X=None), dict(Y=None), dict(heads=0), dict(heads=65536, x_stride=1 << 24, y_stride=1 << 24),
             dict(x_stride=504), dict(y_stride=504), dict(x_stride=516), dict(y_stride=513), dict(x_stride=-512)]
ODD_HEADS = [dict(X=ODD), dict(Y=B + 8), dict(gain=ODD)]
BAD_ROTARY = [dict(dims=-16), dict(dims=144), dict(dims=24), dict(table=None), dict(rows=0), dict(rows=BIG), dict(eps=-1.0),
              dict(eps=NAN), dict(eps=float("inf"))]


def test_rotate_refusals():
    def call(h=(), r=None, T=5, dim=128, G=None, positions=D, hs="made"):
        made = (tri.TriHeads * max(len(h), 1))(*h)
        return raw("tri_heads_rotate", None if hs is None else ctypes.addressof(made), len(h) if G is None else G, T, dim,
                   at(r), positions, None)

    ok = heads()
    for kw in BAD_HEADS:
        assert call([heads(**kw)], rotary()) == EINVAL, kw
        assert call([ok, heads(**kw)], rotary()) == EINVAL, kw
    for kw in ODD_HEADS:
        assert call([ok, heads(**kw)], rotary()) == EALIGN, kw
    for kw in BAD_ROTARY:
        assert call([ok], rotary(**kw)) == EINVAL, kw
    assert call([ok], rotary(table=ODD)) == EALIGN
    assert call([ok], rotary(table=C + 8)) == EALIGN
    assert call([ok], None) == EINVAL and call([ok], rotary(), positions=None) == EINVAL
    assert call([ok], rotary(), positions=D + 2) == EALIGN
    assert call([ok], rotary(), hs=None) == EINVAL
    for kw in [dict(T=0), dict(T=BIG), dict(T=1 << 29), dict(dim=32), dict(dim=96), dict(dim=512), dict(G=0), dict(G=5)]:
        assert call([ok], rotary(), **kw) == EINVAL, kw


BAD_CACHE = [dict(K=None), dict(V=None), dict(K_scale=None), dict(V_scale=None), dict(pages=0), dict(pages=BIG), dict(heads=0),
             dict(heads=65536), dict(dim=96), dict(dim=0), dict(page=8), dict(page=48), dict(page=256), dict(fmt=2), dict(fmt=-1)]
ODD_CACHE = [dict(K=ODD), dict(V=B + 8), dict(K_scale=C + 2), dict(V_scale=D + 1)]
BAD_SEQS = [dict(offsets=None), dict(lens=None), dict(table=None), dict(B=0), dict(B=65536), dict(width=0), dict(width=BIG - 128),
            dict(max_new=0), dict(max_new=BIG), dict(max_len=0), dict(max_len=BIG)]
ODD_SEQS = [dict(offsets=A + 2), dict(lens=B + 1), dict(table=C + 2)]


def test_append_refusals():
    def call(c=cache(), q=seqs(), T=3, K=A, ks=512, V=B, vs=512, rot=None, gain=None, queries=None):
        return raw("tri_cache_append", at(c), at(q), T, K, ks, V, vs, at(rot), gain, at(queries), None)

    for kw in BAD_CACHE:
        assert call(c=cache(**kw)) == EINVAL, kw
    for kw in ODD_CACHE:
        assert call(c=cache(**kw)) == EALIGN, kw
    for kw in BAD_SEQS:
        assert call(q=seqs(**kw)) == EINVAL, kw
    for kw in ODD_SEQS:
        assert call(q=seqs(**kw)) == EALIGN, kw
    assert call(c=None) == EINVAL and call(q=None) == EINVAL
    for kw in [dict(T=0), dict(T=BIG), dict(T=1 << 29), dict(K=None), dict(V=None), dict(ks=504), dict(vs=504), dict(ks=517)]:
        assert call(**kw) == EINVAL, kw
    for kw in [dict(K=ODD), dict(V=B + 8), dict(gain=ODD)]:
        assert call(rot=rotary(), **kw) == EALIGN, kw
    for kw in BAD_ROTARY:
        assert call(rot=rotary(**kw)) == EINVAL, kw
    assert call(rot=rotary(table=ODD)) == EALIGN
    assert call(queries=heads()) == EINVAL       # queries go through the rotation
    for kw in BAD_HEADS:
        assert call(rot=rotary(), queries=heads(**kw)) == EINVAL, kw
    for kw in ODD_HEADS:
        assert call(rot=rotary(), queries=heads(**kw)) == EALIGN, kw


def test_attend_refusals_and_workspace():
    long = seqs(max_len=100000, width=2000)
    need = tri.tri_cache_attend_workspace_bytes(cache(), long, 3, 8)
    assert need > 0 and need % 16 == 0           # one sequence's row is split
    assert tri.tri_cache_attend_workspace_bytes(cache(), seqs(), 3, 8) >= 0

    def call(c=cache(), q=long, T=3, Q=A, qs=1024, H=8, scale=0.1, window=0, sinks=0, O=B, os=1024, ws=C, nbytes=need):
        return raw("tri_cache_attend", at(c), at(q), T, Q, qs, H, scale, window, sinks, O, os, ws, nbytes, None)

    for kw in BAD_CACHE:
        assert call(c=cache(**kw)) == EINVAL, kw
        assert tri.tri_cache_attend_workspace_bytes(cache(**kw), long, 3, 8) == -1
    for kw in ODD_CACHE:
        assert call(c=cache(**kw)) == EALIGN, kw
    for kw in BAD_SEQS:
        assert call(q=seqs(**kw)) == EINVAL, kw
    for kw in ODD_SEQS:
        assert call(q=seqs(**kw)) == EALIGN, kw
    for kw in [dict(T=0), dict(T=BIG), dict(T=1 << 28), dict(H=0), dict(H=6), dict(H=65540, qs=1 << 24, os=1 << 24), dict(window=-1),
               dict(window=BIG), dict(sinks=-1), dict(sinks=BIG)]:
        assert call(**kw) == EINVAL, kw
        kw = {k: v for k, v in kw.items() if k in ("T", "H", "window", "sinks")}
        assert tri.tri_cache_attend_workspace_bytes(cache(), long, kw.get("T", 3), kw.get("H", 8), kw.get("window", 0),
                                                    kw.get("sinks", 0)) == -1
    for kw in [dict(Q=None), dict(O=None), dict(qs=1016), dict(os=1016), dict(qs=1028), dict(scale=NAN), dict(scale=float("inf")),
               dict(ws=None), dict(nbytes=need - 16)]:
        assert call(**kw) == EINVAL, kw
    for kw in [dict(Q=ODD), dict(O=B + 8), dict(ws=C + 8)]:
        assert call(**kw) == EALIGN, kw


def test_results_over_their_inputs_are_refused():
    """Rows that would overlap others' inputs: attention in place, rotation in place with another stride."""
    def rotate(h):
        return raw("tri_heads_rotate", ctypes.addressof(h), 1, 5, 128, at(rotary()), ODD, None)

    assert rotate(heads(Y=A, y_stride=520)) == EINVAL and rotate(heads(Y=A, x_stride=1024)) == EINVAL
    assert rotate(heads(Y=A)) == EALIGN          # (in place with the same stride: refused for the positions' address only)
    queries = heads(Y=A, y_stride=520)
    assert raw("tri_cache_append", at(cache()), at(seqs()), 3, A, 512, B, 512, at(rotary()), None, at(queries), None) == EINVAL
    assert raw("tri_cache_attend", at(cache()), at(seqs()), 3, A, 512, 4, 0.1, 0, 0, A, 512, None, 0, None) == EINVAL


def test_binding_raises_on_error_status():
    with pytest.raises(tri.TriError):
        tri.tri_heads_rotate([heads(heads=0)], 1, 128, rotary(), D, stream=0)
    with pytest.raises(tri.TriError):
        tri.tri_cache_append(cache(page=17), seqs(), 1, A, 512, B, 512, stream=0)
    with pytest.raises(tri.TriError):
        tri.tri_cache_attend(cache(), seqs(), 1, A, 512, 5, 1.0, 0, 0, B, 512, None, 0, stream=0)


def test_helpers_refuse_tensors_off_the_gpu():
    import torch
    x, i = torch.zeros((1, 1, 64), dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    k = torch.zeros((1, 1, 64, 64), dtype=torch.uint8)
    s = torch.ones((1, 1))
    for call in [lambda: tri.heads_rotate((x,), tri.Rotary(None), i), lambda: tri.KVCache(k, k, s, s, 0),
                 lambda: tri.Sequences(i, i, i.view(1, 1), 1), lambda: tri.Rotary(torch.zeros((4, 32, 2))),
                 lambda: tri.Rotary(None, gains=(x[0, 0],))]:
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the definitions that the GPU tests go by

def test_code_values():
    v = ref.values_of(ref.E4M3)
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1 and v[0x7E] == 448 and v[0xFE] == -448
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fine = ~np.isnan(t)
    assert fine.sum() == 254 and np.array_equal(t[fine], v[fine])
    assert ref.values_of(ref.INT8)[[0, 1, 127, 129, 255]].tolist() == [0, 1, 127, -127, -1]


def test_codes_are_nearest_ties_even():
    import torch
    x = np.concatenate([np.random.default_rng(5).standard_normal(4000) * 60, [0.0, -0.0, 448, -448, 2.0 ** -10, 3 * 2.0 ** -10, 17, 19, 0.5, 1.5]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.codes_of(x.astype(np.float64), ref.E4M3), want)
    assert ref.codes_of(np.array([0.5, 1.5, -0.5, -126.5, 127.0]), ref.INT8).view(np.int8).tolist() == [0, 2, 0, -126, 127]


def test_scales_are_the_least_powers_of_two():
    for fmt, top in ref.TOP.items():
        m = np.array([0.0, top, np.nextafter(top, 1e9), top / 2, 65504.0, 2.0 ** -24])
        s = ref.need_scale(m, fmt)
        assert s[0] == 2.0 ** -30 and s[1] == 1 and s[2] == 2 and s[3] == 0.5
        assert np.all(m <= top * s) and np.all((m > top * s / 2) | (s == 2.0 ** -30))


def test_reference_attention_closed_forms():
    """One visible token gives its value; equal scores give the mean; a window of one gives the token's own value."""
    rng = np.random.default_rng(3)
    b = ref.Batch(rng, [3, 1], [3, 40], 2, 64, 16, ref.INT8)
    Q = np.zeros((4, 4, 64), dtype=np.float16)
    out, tol, live = b.attend(Q, 1.0)
    v = ref.values_of(ref.INT8)
    pg, vs = b.table, b.vs.astype(np.float64)
    first = v[b.V[pg[0, 0], 0, :, 0]] * vs[pg[0, 0], 0]
    assert live.all() and np.allclose(out[0, 0], first)
    mean = np.mean([v[b.V[pg[1, j // 16], 1, :, j % 16]] * vs[pg[1, j // 16], 1] for j in range(40)], 0)
    assert np.allclose(out[3, 3], mean)
    own, _, _ = b.attend(Q, 1.0, window=1)
    assert np.allclose(own[2, 1], v[b.V[pg[0, 0], 0, :, 2]] * vs[pg[0, 0], 0])
    both, _, _ = b.attend(Q, 1.0, window=1, sinks=1)
    assert np.allclose(both[2, 1], (own[2, 1] + first) / 2)


def test_reference_append_grows_and_keeps_scales():
    rng = np.random.default_rng(4)
    b = ref.Batch(rng, [1], [5], 1, 64, 16, ref.INT8)
    page = b.table[0, 0]
    b.ks[page], b.vs[page] = 1.0, 1.0
    before = b.K[page, 0].view(np.int8).copy()
    K, V = np.full((1, 1, 64), 300.0, dtype=np.float16), np.full((1, 1, 64), 5.0, dtype=np.float16)
    b.append(K, V)
    assert b.ks[page, 0] == 4 and b.vs[page, 0] == 1
    now = b.K[page, 0].view(np.int8)
    assert np.array_equal(now[:4], np.rint(before[:4] / 4)) and np.all(now[4] == 75) and np.array_equal(now[5:], before[5:])
    assert np.all(b.V[page, 0, :, 4] == 5)


def test_rotation_of_the_reference():
    """A quarter turn, norms, and both pairings."""
    x = np.random.default_rng(6).standard_normal((1, 1, 64))
    quarter = np.zeros((1, 32, 2))
    quarter[..., 1] = 1
    y, _ = ref.rotate(x, np.array([0]), quarter, norm=False)
    assert np.allclose(y[..., :32], -x[..., 32:]) and np.allclose(y[..., 32:], x[..., :32])
    y, _ = ref.rotate(x, np.array([0]), quarter, interleaved=True, norm=False)
    assert np.allclose(y[..., 0::2], -x[..., 1::2]) and np.allclose(y[..., 1::2], x[..., 0::2])
    y, _ = ref.rotate(1000 * x, np.array([0]), quarter, eps=0.0)
    assert np.isclose((y * y).mean(), 1)
