"""Host-side refusals of the 4-bit and experts' entry points: bad arguments are rejected before anything is launched (no
GPU needed; the addresses are fake and must not be touched)."""
import pytest

import bit_mixed_precision_tri_amd as tri

A, B, C, D, ODD = 4096, 8192, 12288, 16384, 4097
BIG = 1 << 31
OK, EINVAL, EALIGN = tri.TRI_OK, tri.TRI_EINVAL, tri.TRI_EALIGN


def raw(name, *args):
    return getattr(tri.lib(), name)(*args)


def test_int4_bytes():
    # tiles of 16 x 128: 1 KB of codes, 16 * 128/group scales of 2 bytes (and zero points of 1)
    assert tri.tri_int4_bytes(16, 128, 128, False) == 1024 + 32
    assert tri.tri_int4_bytes(16, 128, 32, False) == 1024 + 128
    assert tri.tri_int4_bytes(16, 128, 32, True) == 1024 + 192
    assert tri.tri_int4_bytes(17, 129, 64, True) == 4 * (1024 + 96)
    assert tri.tri_int4_bytes(4096, 11008, 128, False) == 256 * 86 * (1024 + 32)
    for bad in [(0, 1, 32), (1, 0, 32), (1, 1, 16), (1, 1, 256), (1, 1, 0), (BIG, 1, 32), (1, BIG, 32)]:
        assert tri.tri_int4_bytes(*bad, False) == -1
    assert tri.tri_int4_bytes(1 << 26, 1, 32, False) == -1          # 2^22 tiles
    assert tri.tri_int4_bytes((1 << 26) - 16, 1, 32, False) > 0


def test_int4_layout_refusals():
    for args in [(None, B, None, 4, 64, 32, C), (A, None, None, 4, 64, 32, C), (A, B, None, 4, 64, 32, None),
                 (A, B, None, 0, 64, 32, C), (A, B, None, 4, 0, 32, C), (A, B, None, 4, 64, 48, C),
                 (A, B, None, BIG, 64, 32, C), (A, B, None, 4, BIG, 32, C)]:
        assert raw("tri_int4_pack", *args, None) == EINVAL
    assert raw("tri_int4_pack", A, B, None, 4, 64, 32, ODD, None) == EALIGN
    assert raw("tri_int4_pack", A, ODD, None, 4, 64, 32, C, None) == EALIGN
    for args in [(None, 4, 64, 32, 0, A, B, None), (C, 4, 64, 32, 0, None, B, None), (C, 4, 64, 32, 0, A, None, None),
                 (C, 4, 64, 32, 1, A, B, None), (C, 4, 64, 31, 0, A, B, None), (C, 0, 64, 32, 0, A, B, None)]:
        assert raw("tri_int4_unpack", *args, None) == EINVAL
    assert raw("tri_int4_unpack", ODD, 4, 64, 32, 0, A, B, None, None) == EALIGN
    for args in [(None, 4, 64, 32, 0, C), (A, 4, 64, 32, 0, None), (A, 0, 64, 32, 0, C), (A, 4, 64, 33, 0, C)]:
        assert raw("tri_int4_quantize", *args, None) == EINVAL
    assert raw("tri_int4_quantize", A, 4, 64, 32, 0, ODD, None) == EALIGN
    assert raw("tri_int4_quantize", A + 2, 4, 64, 32, 0, C, None) == EALIGN


def test_int4_linear_refusals():
    for args in [(None, B, 1, 4, 64, 32, 0, None, C), (A, None, 1, 4, 64, 32, 0, None, C),
                 (A, B, 1, 4, 64, 32, 0, None, None), (A, B, 0, 4, 64, 32, 0, None, C), (A, B, 1, 0, 64, 32, 0, None, C),
                 (A, B, 1, 4, 0, 32, 0, None, C), (A, B, 1, 4, 64, 40, 0, None, C), (A, B, BIG, 4, 64, 32, 0, None, C),
                 (A, B, 1, BIG, 64, 32, 0, None, C), (A, B, 1, 4, BIG, 32, 0, None, C)]:
        assert raw("tri_int4_linear", *args, None) == EINVAL
    for args in [(ODD, B, 1, 4, 64, 32, 0, None, C), (A, ODD, 1, 4, 64, 32, 0, None, C),
                 (A, B, 1, 4, 64, 32, 0, ODD, C), (A, B, 1, 4, 64, 32, 0, None, ODD)]:
        assert raw("tri_int4_linear", *args, None) == EALIGN


def test_route_workspace_and_refusals():
    assert tri.tri_experts_route_workspace_bytes(1, 8, 2) == 0      # one workgroup needs none
    need = tri.tri_experts_route_workspace_bytes(4096, 64, 8)
    assert need > 0 and need % 16 == 0
    for bad in [(0, 8, 2), (1, 0, 1), (1, 257, 2), (1, 8, 0), (1, 8, 9), (1, 64, 17), (BIG, 8, 2), (1 << 27, 16, 16)]:
        assert tri.tri_experts_route_workspace_bytes(*bad) == -1
    ok = dict(logits=A, dtype=0, T=4096, E=64, topk=8, renorm=1, ids=A, weights=A, offsets=A, rows=A, pos=A, ws=B,
              ws_bytes=need)

    def call(**kw):
        return raw("tri_experts_route", *{**ok, **kw}.values(), None)

    for kw in [dict(logits=None), dict(ids=None), dict(weights=None), dict(offsets=None), dict(rows=None), dict(pos=None),
               dict(ws=None), dict(ws_bytes=need - 16), dict(dtype=2), dict(T=0), dict(E=0), dict(E=257), dict(topk=0),
               dict(topk=65), dict(topk=17)]:
        assert call(**kw) == EINVAL, kw
    for kw in [dict(logits=ODD), dict(logits=A + 2, dtype=1), dict(ids=A + 2), dict(weights=A + 2), dict(offsets=A + 2),
               dict(rows=A + 2), dict(pos=A + 2), dict(ws=B + 8)]:
        assert call(**kw) == EALIGN, kw


def test_experts_products_refusals():
    ok = dict(X=A, T=16, offsets=B, rows=B, R=32, Wp=C, scale=D, E=8, N=64, K=128, fmt=0, Y=A)

    def linear(**kw):
        return raw("tri_experts_linear", *{**ok, **kw}.values(), None)

    def pair(Wp_up=C, scale_up=D, **kw):
        v = {**ok, **kw}
        return raw("tri_experts_pair", *[v[n] for n in ("X", "T", "offsets", "rows", "R", "Wp", "scale")], Wp_up,
                   scale_up, *[v[n] for n in ("E", "N", "K", "fmt", "Y")], None)

    for call in (linear, pair):
        for kw in [dict(X=None), dict(offsets=None), dict(Wp=None), dict(scale=None), dict(Y=None), dict(T=0), dict(R=0),
                   dict(E=0), dict(E=257), dict(N=0), dict(K=0), dict(fmt=2), dict(T=BIG), dict(R=BIG), dict(N=BIG),
                   dict(K=BIG), dict(rows=None), dict(T=1 << 20, K=4096)]:   # (X in order: T >= R; gathered: 4 GiB)
            assert call(**kw) == EINVAL, kw
        for kw in [dict(X=ODD), dict(Wp=ODD), dict(Y=ODD), dict(offsets=B + 2), dict(rows=B + 2), dict(scale=D + 2)]:
            assert call(**kw) == EALIGN, kw
    assert pair(Wp_up=None) == EINVAL and pair(scale_up=None) == EINVAL
    assert pair(Wp_up=ODD) == EALIGN and pair(scale_up=D + 2) == EALIGN


def test_combine_refusals():
    ok = dict(Z=A, R=32, pos=B, weights=C, residual=None, T=16, topk=2, N=64, Y=D)

    def call(**kw):
        return raw("tri_experts_combine", *{**ok, **kw}.values(), None)

    for kw in [dict(Z=None), dict(pos=None), dict(weights=None), dict(Y=None), dict(R=0), dict(T=0), dict(topk=0),
               dict(topk=17), dict(N=0), dict(R=BIG), dict(T=BIG), dict(N=BIG)]:
        assert call(**kw) == EINVAL, kw
    for kw in [dict(Z=ODD), dict(Y=ODD), dict(residual=ODD), dict(pos=B + 2), dict(weights=C + 2)]:
        assert call(**kw) == EALIGN, kw


def test_binding_raises_on_error_status():
    with pytest.raises(tri.TriError):
        tri.tri_int4_linear(A, B, 0, 4, 64, 32, False, None, C, stream=0)
    with pytest.raises(tri.TriError):
        tri.tri_experts_combine(A, 0, B, C, None, 1, 1, 64, D, stream=0)


def test_helpers_refuse_tensors_off_the_gpu():
    import torch
    x, w = torch.zeros((1, 64), dtype=torch.float16), torch.zeros(1, dtype=torch.uint8)
    i = torch.zeros((1, 1), dtype=torch.int32)
    for call in [lambda: tri.int4_linear(x, w, 16, 32), lambda: tri.int4_pack(w.view(1, 1), x, 32),
                 lambda: tri.int4_unpack(w, 1, 1, 32), lambda: tri.int4_quantize(x.float(), 32),
                 lambda: tri.experts_route(x, 2), lambda: tri.experts_combine(x, i, x),
                 lambda: tri.experts_linear(x, i, i, w, x, 64, 0)]:
        with pytest.raises(ValueError):
            call()


def test_experts_products_refuse_more_outputs_than_a_grid_takes():
    """2^27 - 15 outputs would be 2^23 workgroups of 512 threads, one thread more than a grid's row may have."""
    for N in ((1 << 27) - 15, (1 << 27) - 1, 1 << 27):
        for K, fmt in ((5, 0), (8, 1)):
            assert raw("tri_experts_linear", A, 16, B, B, 32, C, D, 8, N, K, fmt, A, None) == EINVAL
            assert raw("tri_experts_pair", A, 16, B, B, 32, C, D, C, D, 8, N, K, fmt, A, None) == EINVAL
