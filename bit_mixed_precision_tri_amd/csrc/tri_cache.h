// tri_cache.h -- batches of sequences and the 8-bit cache, as the kernels see them (contract: include/tri.h).
#pragma once
#include "tri_device.h"
#include "tri_internal.h"

namespace tri {

// One sequence's new tokens: rows r0 .. r0 + n - 1 of the call, at positions p0 .. p0 + n - 1 (p0 may be negative).
struct Span {
    int r0, n, p0;
};
__device__ __forceinline__ Span span_of(const tri_sequences &sq, int T, int b)
{
    const int lo = min(max(sq.offsets[b], 0), T), hi = min(max(sq.offsets[b + 1], 0), T);
    const int n = max(hi - lo, 0);
    return Span{lo, min(n, (int)sq.max_new), min(max(sq.lens[b], 0), 0x7fffff00) - n};
}

// The sequence that owns row t: the last b with offsets[b] <= t; the wave's lanes probe 64 of them at a time.
__device__ __forceinline__ int owner(const tri_sequences &sq, int t)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, n = (int)sq.B;                   // candidates lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 63) / 64, k = lane * step;
        const bool before = k < n && sq.offsets[lo + k] <= t;
        const int last = max(__popcll(__ballot(before)) - 1, 0);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The page of place `i` of a sequence's row of the table; -1: none.
__device__ __forceinline__ int page_at(const tri_sequences &sq, const tri_cache &c, int b, int64_t i)
{
    if (i < 0 || i >= sq.width) return -1;
    const int id = sq.table[(int64_t)b * sq.width + i];
    return id >= 0 && id < (int)c.pages ? id : -1;
}

// One launch's part of a call: seqs sequences from seq0 on, tiles pieces (row tiles, page slots) of each from tile0 on.
struct Grid {
    int seq0, seqs, tile0, tiles;
};

// A grid has fewer than 2^32 threads: as many launches as that takes (one, but for bounds of millions of pieces), each of at
// most 2^21 workgroups of up to 1024 threads; `one` workgroups (far fewer than that) are for one piece of a sequence.
template <typename Launch>
void for_grids(int64_t B, int64_t pieces, int64_t one, Launch launch)
{
    const int64_t most = 1 << 21;
    int64_t tiles = most / one, seqs;
    tiles = tiles < 1 ? 1 : tiles < pieces ? tiles : pieces;
    seqs = most / (tiles * one);
    seqs = seqs < 1 ? 1 : seqs < B ? seqs : B;
    for (int64_t b = 0; b < B; b += seqs)
        for (int64_t t = 0; t < pieces; t += tiles) {
            const Grid gd = {(int)b, (int)(seqs < B - b ? seqs : B - b), (int)t, (int)(tiles < pieces - t ? tiles : pieces - t)};
            launch(gd, (uint32_t)(gd.seqs * (int64_t)gd.tiles * one));
        }
}

// Largest code's value, as the exponent e and the fraction f (of 2^23) of f 2^e: 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8.
template <int FMT> constexpr int kTopExp = FMT == TRI_KV_INT8 ? 6 : 8;
template <int FMT> constexpr uint32_t kTopFrac = FMT == TRI_KV_INT8 ? 0x7E0000u : 0x600000u;

// The exponent of the least power of two, 2^-30 or more, at which fp16 bits `amax` (no sign, finite) are within the codes.
template <int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t amax)
{
    const uint32_t f = __float_as_uint(h2f((uint16_t)amax));     // 0 or normal: fp32 holds every fp16 as a normal number
    const int e = (int)(f >> 23) - 127 - kTopExp<FMT> + ((f & 0x7FFFFFu) > kTopFrac<FMT> ? 1 : 0);
    return max(e, -30);                                          // (0 gives -133)
}

// |x| of an fp16 as bits, NaN as 0 and infinity as 65504; and x itself under the same rules.
__device__ __forceinline__ uint32_t magnitude(uint32_t h)
{
    const uint32_t m = h & 0x7FFFu;
    return m > 0x7C00u ? 0u : min(m, 0x7BFFu);
}
__device__ __forceinline__ float plain_value(uint32_t h) { return h2f((uint16_t)((h & 0x8000u) | magnitude(h))); }

// Four values times inv, rounded to nearest even, as four codes.  int8: adding 1.5 * 2^23 leaves the rounded integer in
// the low bits of the sum (one rounding: fma).  The caller's scale keeps them within the codes.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    if constexpr (FMT == TRI_KV_INT8) {
        constexpr float kMagic = 12582912.f;
        const uint32_t ia = __float_as_uint(fmaf(a, inv, kMagic)), ib = __float_as_uint(fmaf(b, inv, kMagic));
        const uint32_t ic = __float_as_uint(fmaf(c, inv, kMagic)), id = __float_as_uint(fmaf(d, inv, kMagic));
        return perm(perm(id, ic, 0x0C0C0400u), perm(ib, ia, 0x0C0C0400u), 0x05040100u);
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, lo, true);
    }
}

// Four codes (bytes of w) as fp16 pairs (0, 1) and (2, 3), exactly.  int8: the byte with its sign bit flipped under the
// fp16 exponent of 1024 reads 1024 + 128 + code.  e4m3: its bits one place lower in an fp16 are its value times 2^-8
// (both keep subnormals); the factor kCodeUnit goes into the scale.
template <int FMT> constexpr float kCodeUnit = FMT == TRI_KV_INT8 ? 1.f : 256.f;
template <int FMT>
__device__ __forceinline__ uint2 decode4(uint32_t w)
{
    if constexpr (FMT == TRI_KV_INT8) {
        const half2_t off = {(_Float16)1152.f, (_Float16)1152.f};
        const uint32_t u = w ^ 0x80808080u;
        return make_uint2(__builtin_bit_cast(uint32_t, (half2_t)(as_h2(perm(0x64646464u, u, 0x04010400u)) - off)),
                          __builtin_bit_cast(uint32_t, (half2_t)(as_h2(perm(0x64646464u, u, 0x04030402u)) - off)));
    } else {
        typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
        const i16x2 a = __builtin_bit_cast(i16x2, perm(0u, w, 0x010C000Cu)) >> (int16_t)1;    // sign, sign, exponent, fraction
        const i16x2 b = __builtin_bit_cast(i16x2, perm(0u, w, 0x030C020Cu)) >> (int16_t)1;
        return make_uint2(__builtin_bit_cast(uint32_t, a) & 0xBF80BF80u, __builtin_bit_cast(uint32_t, b) & 0xBF80BF80u);
    }
}
// Eight codes, an operand of a product.
template <int FMT>
__device__ __forceinline__ half8_t decode8(uint32_t w0, uint32_t w1)
{
    const uint2 a = decode4<FMT>(w0), b = decode4<FMT>(w1);
    return __builtin_bit_cast(half8_t, u32x4{a.x, a.y, b.x, b.y});
}

// The value of one code, for the rounding of earlier codes to a larger scale.
template <int FMT>
__device__ __forceinline__ float code_value(uint32_t byte)
{
    if constexpr (FMT == TRI_KV_INT8) return (float)(int8_t)byte;
    return 256.f * h2f((uint16_t)decode4<FMT>(byte).x);
}

}  // namespace tri
