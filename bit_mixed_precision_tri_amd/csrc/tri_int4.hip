// tri_int4.hip -- 4-bit layers with group scales: layout, quantiser and product.
//
//   W[n][k] = S[n][k / group] * (Q[n][k] - Z[n][k / group]),   Y[m][n] = sum_k W[n][k] X[m][k]
// with Q and Z in 0..15 (Z = 8 for a matrix without zero points).  The stored layout is described
// in include/tri.h: tiles of 16 rows x 128 values, 1 KB of codes each.
#include "tri_device.h"
#include "tri_internal.h"

namespace tri {

namespace {

// Where a packed matrix's regions begin and how many words, scales they hold.
struct Int4Map {
    int64_t NB, KS;                              // 16-row blocks, 128-value steps
    int gps;                                     // groups per step
    int64_t tiles() const { return NB * KS; }
    int64_t scales() const { return tiles() * 16 * gps; }
};

// Tiles of a matrix, at most (2^33 weights): keeps every launch's thread count below 2^32.
constexpr int64_t kInt4MaxTiles = (int64_t)1 << 22;
// Longest row: 32-bit buffer offsets over 16 activation rows and over four blocks of a row's tiles.
constexpr int64_t kInt4MaxK = (int64_t)1 << 25;

Int4Map int4_map(int64_t N, int64_t K, int group) { return {(N + 15) / 16, (K + 127) / 128, 128 / group}; }

// bit position of value i of a word
__device__ __forceinline__ int nibble_at(int i) { return 4 * (i / 2) + 16 * (i % 2); }

// The layout kernels move each byte once.  One workgroup per tile (block b, step s): thread (j, q) packs piece q (8 values) of row j.  Threads
// q < gps also write a scale and a zero point.
__global__ __launch_bounds__(256) void k_int4_pack(const uint8_t *__restrict__ Q, const uint16_t *__restrict__ S,
                                                   const uint8_t *__restrict__ Z, int N, int K, int KS, int gps,
                                                   uint32_t *__restrict__ codes, uint16_t *__restrict__ scales,
                                                   uint8_t *__restrict__ zeros)
{
    const int64_t tile = blockIdx.x;
    const int b = (int)(tile / KS), s = (int)(tile % KS);
    const int j = threadIdx.x >> 4, q = threadIdx.x & 15;
    const int64_t n = 16 * (int64_t)b + j, k0 = 128 * (int64_t)s + 8 * q;
    uint32_t w = 0x88888888u;
    if (n < N) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w |= (uint32_t)(k0 + i < K ? Q[n * K + k0 + i] & 15 : 8) << nibble_at(i);
    }
    codes[tile * 256 + (16 * (q & 3) + j) * 4 + (q >> 2)] = w;
    if (q < gps) {
        const int group = 128 / gps;
        const int64_t G = ((int64_t)K + group - 1) / group, gi = (int64_t)s * gps + q;
        const bool in = n < N && gi < G;
        const int64_t o = (tile * 16 + j) * gps + q;
        scales[o] = in ? S[n * G + gi] : (uint16_t)0;
        if (zeros) zeros[o] = in ? Z[n * G + gi] & 15 : 8;
    }
}

__global__ __launch_bounds__(256) void k_int4_unpack(const uint32_t *__restrict__ codes,
                                                     const uint16_t *__restrict__ scales,
                                                     const uint8_t *__restrict__ zeros, int N, int K, int KS, int gps,
                                                     uint8_t *__restrict__ Q, uint16_t *__restrict__ S,
                                                     uint8_t *__restrict__ Z)
{
    const int64_t tile = blockIdx.x;
    const int b = (int)(tile / KS), s = (int)(tile % KS);
    const int j = threadIdx.x >> 4, q = threadIdx.x & 15;
    const int64_t n = 16 * (int64_t)b + j, k0 = 128 * (int64_t)s + 8 * q;
    if (n >= N) return;
    const uint32_t w = codes[tile * 256 + (16 * (q & 3) + j) * 4 + (q >> 2)];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k0 + i < K) Q[n * K + k0 + i] = (uint8_t)((w >> nibble_at(i)) & 15u);
    if (q < gps) {
        const int group = 128 / gps;
        const int64_t G = ((int64_t)K + group - 1) / group, gi = (int64_t)s * gps + q;
        if (gi < G) {
            const int64_t o = (tile * 16 + j) * gps + q;
            S[n * G + gi] = scales[o];
            if (zeros) Z[n * G + gi] = zeros[o];
        }
    }
}

// One workgroup per tile; the 16/gps threads of a group are neighbours in a 16-lane row.
__global__ __launch_bounds__(256) void k_int4_quantize(const float *__restrict__ W, int N, int K, int KS, int gps,
                                                       uint32_t *__restrict__ codes, uint16_t *__restrict__ scales,
                                                       uint8_t *__restrict__ zeros)
{
    const int64_t tile = blockIdx.x;
    const int b = (int)(tile / KS), s = (int)(tile % KS);
    const int j = threadIdx.x >> 4, q = threadIdx.x & 15;
    const int64_t n = 16 * (int64_t)b + j, k0 = 128 * (int64_t)s + 8 * q;
    float v[8], lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = (n < N && k0 + i < K) ? W[n * K + k0 + i] : 0.f;
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    const int width = 16 / gps;                  // threads per group
    for (int m = 1; m < width; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m, 16));
        hi = fmaxf(hi, __shfl_xor(hi, m, 16));
    }
    const float top = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
    const _Float16 sh = (_Float16)fminf(top, 65504.f);
    const float sc = (float)sh;
    int z = 8;
    if (zeros && sc > 0.f) z = (int)fminf(fmaxf(rintf(-lo / sc), 0.f), 15.f);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int c = 8;                               // rows past N, values past K, groups of scale 0
        if (n < N && k0 + i < K && sc > 0.f) {
            const float r = rintf(v[i] / sc);
            c = zeros ? (int)fminf(fmaxf(r + (float)z, 0.f), 15.f) : (int)fminf(fmaxf(r, -8.f), 7.f) + 8;
        }
        w |= (uint32_t)c << nibble_at(i);
    }
    codes[tile * 256 + (16 * (q & 3) + j) * 4 + (q >> 2)] = w;
    if (q % width == 0) {
        const int64_t o = (tile * 16 + j) * gps + q / width;
        scales[o] = __builtin_bit_cast(uint16_t, sh);
        if (zeros) zeros[o] = (uint8_t)z;
    }
}

// ---------------------------------------------------------------- product, up to 16 rows per pass

constexpr uint32_t kRsrcWord3 = 0x00020000u;     // raw buffer resource, gfx9 family
constexpr uint32_t kOob = 0x80000000u;           // an offset past every buffer here: reads zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, (int)kRsrcWord3);
}

__device__ __forceinline__ float4_t mfma(const u32x4 a, const u32x4 b, float4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                  0, 0);
}

// Eight codes of a word as fp16 code - zero, exactly.  Codes at bits 0-3 of a half, OR-ed into 1024.0 (mantissa
// step 1), read 1024 + q; at bits 4-7, OR-ed into 64.0 (step 1/16), 64 + q; one packed add takes 1024 + z or
// 64 + z away.  lo, hi: the two fp16 pairs -(1024 + z) and -(64 + z); b10, b6: 1024.0 and 64.0 pairs held in
// registers (an instruction takes one scalar operand: the mask).
__device__ __forceinline__ u32x4 decode(uint32_t w, uint32_t b10, uint32_t b6, uint32_t lo, uint32_t hi)
{
    const uint32_t v = w >> 8;
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, as_h2((w & 0x000F000Fu) | b10) + as_h2(lo));
    r[1] = __builtin_bit_cast(uint32_t, as_h2((w & 0x00F000F0u) | b6) + as_h2(hi));
    r[2] = __builtin_bit_cast(uint32_t, as_h2((v & 0x000F000Fu) | b10) + as_h2(lo));
    r[3] = __builtin_bit_cast(uint32_t, as_h2((v & 0x00F000F0u) | b6) + as_h2(hi));
    return r;
}

// MA (1, 2, 4, 8, 16) activation rows times RB blocks of 16 weight rows per workgroup of NW waves.
//
// v_mfma_f32_16x16x32_f16 takes 16 A rows.  With fewer activation rows than that, the A rows that one product does
// not need carry the activations of the next ones: A row i = MA c + a holds activation row a at the c-th of
// 16/MA consecutive pieces of 32 values.  One 16-byte load per lane then fetches the A operand of 16/MA products
// (for one activation row, of four whole steps), with nothing to permute or stage; of product c's result only
// the rows MA c .. MA c + MA-1 are taken.  B operands are whole words of the layout, lane for lane.
//
// A unit is U steps (the span of one A load, at least one step); wave w takes units w, w + NW, ..., the loads of two
// units in flight.  Each step's partial sums are scaled in fp32 by their group's scale where they lie: lane (g, j)
// of the result holds row j's products of step tl(g), so it loads the scales of that row and step.  Zero points
// shift the codes as they are decoded (U == 1), or are taken off by sum_k x, formed by one more product with
// ones per A load (U > 1, where a lane decodes other steps than it scales).
//
// One row is bound by the weight stream: 4096 -> 11008 (23.3 MB, group 128) takes 6.6 us, a plain read of as many bytes
// 4.7 us, an empty launch 1.9 us; 8192 -> 28672 (121 MB) 24.6 us against 19.4.  From about eight rows on the activations
// that every workgroup reads weigh as much (16 rows: 7.9 us, and 12.7 us on 11008 -> 4096).  Twelve or sixteen waves, or
// three to six units in flight, changed a few shapes by 5% either way and are not used.
template <int MA, int RB, int GPS, bool ZP, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW) void k_int4_mv(const uint16_t *__restrict__ X, const uint8_t *__restrict__ codes,
                                                     const uint16_t *__restrict__ scales,
                                                     const uint8_t *__restrict__ zeros, int M, int N, int K, int KS,
                                                     const uint16_t *R, uint16_t *Y)
{
    constexpr int CL = 16 / MA;                  // pieces of 32 values per A load
    constexpr int U = CL > 4 ? CL / 4 : 1;       // steps per unit
    constexpr int AL = CL < 4 ? 4 / CL : 1;      // A loads per unit
    constexpr bool ZSUM = ZP && U > 1, ZDEC = ZP && U == 1;
    constexpr int TE = MA < 4 ? MA : 4;          // results per lane and block
    __shared__ float red[NW][MA][16 * RB];

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    const int m0 = MA * (int)blockIdx.y;
    const int64_t b0 = (int64_t)blockIdx.x * RB; // first block of 16 weight rows
    const int nb = min(RB, (N + 15) / 16 - (int)b0);

    const __amdgpu_buffer_rsrc_t wr = rsrc(codes + b0 * KS * 1024, __builtin_amdgcn_readfirstlane((uint32_t)nb * KS * 1024u));
    const __amdgpu_buffer_rsrc_t sr =
        rsrc(scales + b0 * KS * (16 * GPS), __builtin_amdgcn_readfirstlane((uint32_t)nb * KS * (32u * GPS)));
    const __amdgpu_buffer_rsrc_t zr =
        rsrc(ZP ? zeros + b0 * KS * (16 * GPS) : nullptr, __builtin_amdgcn_readfirstlane(ZP ? (uint32_t)nb * KS * (16u * GPS) : 0u));
    const int mm = min(MA, M - m0);
    const __amdgpu_buffer_rsrc_t xr =
        rsrc(X + (int64_t)m0 * K, __builtin_amdgcn_readfirstlane((uint32_t)mm * (uint32_t)K * 2u));

    const int ac = j / MA, aa = j % MA;          // this lane's A row: piece ac of the load, activation row aa
    const uint32_t xrow = aa < mm ? (uint32_t)aa * (uint32_t)K * 2u : kOob;
    const uint16_t *const xlane = X + ((int64_t)m0 + aa) * K;
    const int tl = U == 4 ? g : U == 2 ? g >> 1 : 0;   // the step of a unit that this lane scales

    struct Unit {
        u32x4 w[RB][U];
        u32x4 a[AL];
        uint32_t s[RB][GPS == 4 ? 2 : 1];        // GPS scales
        uint32_t z[RB];                          // GPS zero points
    };
    auto load = [&](int u, Unit &t) __attribute__((always_inline)) {
        const int s0 = u * U;
#pragma unroll
        for (int q = 0; q < AL; ++q) {
            const int k = 128 * s0 + 32 * (CL * q + ac) + 8 * g;
            if constexpr (VEC) {
                t.a[q] = __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(k < K ? xrow + 2u * (uint32_t)k : kOob), 0, 0);
            } else {                             // rows that are no whole pieces
                t.a[q] = u32x4{0u, 0u, 0u, 0u};
                if (aa < mm && k < K) t.a[q] = k + 8 <= K ? ld16_any(xlane + k) : ld16_part(xlane + k, K - k);
            }
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int st = s0 + tl;
            const uint32_t so = st < KS ? ((uint32_t)(r * KS + st) * 16u + (uint32_t)j) * GPS : kOob >> 1;
            if constexpr (GPS == 4) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(sr, (int)(so * 2u), 0, 0);
                t.s[r][0] = v[0];
                t.s[r][1] = v[1];
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b32(zr, (int)so, 0, 0);
            } else if constexpr (GPS == 2) {
                t.s[r][0] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)(so * 2u), 0, 0);
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b16(zr, (int)so, 0, 0);
            } else {
                t.s[r][0] = __builtin_amdgcn_raw_buffer_load_b16(sr, (int)(so * 2u), 0, 0);
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b8(zr, (int)so, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint32_t o = s0 + i < KS ? (uint32_t)(r * KS + s0 + i) * 1024u + 16u * (uint32_t)lane : kOob;
                t.w[r][i] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)o, 0, 0);
            }
        }
    };
    uint32_t b10, b6;
    asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(b10));
    asm volatile("v_mov_b32 %0, 0x54005400" : "=v"(b6));
    const float4_t zero4 = {0.f, 0.f, 0.f, 0.f};
    float tot[RB][TE];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int e = 0; e < TE; ++e) tot[r][e] = 0.f;

    auto scale_of = [](const Unit &t, int r, int i) {
        return h2f((uint16_t)(t.s[r][GPS == 4 ? i / 2 : 0] >> (GPS == 1 ? 0 : 16 * (i % 2))));
    };
    auto run = [&](const Unit &t) __attribute__((always_inline)) {
        float4_t xs = zero4;                     // ZSUM: sums of the A rows
        if constexpr (ZSUM) {
            const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
            xs = mfma(t.a[0], ones, zero4);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            float sc[GPS];
#pragma unroll
            for (int i = 0; i < GPS; ++i) sc[i] = scale_of(t, r, i);
            if constexpr (U > 1) {
                // products of step i, piece p: A row 4 i + p (MA = 1), 2 (4 i + p) + a (MA = 2)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    float4_t d[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) d[p] = mfma(t.a[0], decode(t.w[r][i][p], b10, b6, 0xE408E408u, 0xD480D480u), zero4);
                    if constexpr (MA == 1) {     // lane group i, element p
                        float v = 0.f;
                        if constexpr (ZP) {
#pragma unroll
                            for (int p = 0; p < 4; ++p)
                                d[p][p] = fmaf(xs[p], 8.f - (float)((t.z[r] >> (8 * (p * GPS / 4))) & 15u), d[p][p]);
                        }
                        if constexpr (GPS == 4) v = (d[0][0] * sc[0] + d[1][1] * sc[1]) + (d[2][2] * sc[2] + d[3][3] * sc[3]);
                        if constexpr (GPS == 2) v = (d[0][0] + d[1][1]) * sc[0] + (d[2][2] + d[3][3]) * sc[1];
                        if constexpr (GPS == 1) v = ((d[0][0] + d[1][1]) + (d[2][2] + d[3][3])) * sc[0];
                        tot[r][0] += g == i ? v : 0.f;
                    } else {                     // lane group 2 i + p / 2, elements 2 (p % 2) + a
                        const bool odd = g & 1;
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            float v0 = odd ? d[2][a] : d[0][a], v1 = odd ? d[3][2 + a] : d[1][2 + a];
                            if constexpr (ZP) {
                                const uint32_t zz = GPS == 4 ? (odd ? t.z[r] >> 16 : t.z[r])
                                                             : GPS == 2 ? (odd ? t.z[r] >> 8 : t.z[r]) : t.z[r];
                                v0 = fmaf(xs[a], 8.f - (float)(zz & 15u), v0);
                                v1 = fmaf(xs[2 + a], 8.f - (float)((GPS == 4 ? zz >> 8 : zz) & 15u), v1);
                            }
                            float v;
                            if constexpr (GPS == 4) v = v0 * (odd ? sc[2] : sc[0]) + v1 * (odd ? sc[3] : sc[1]);
                            else v = (v0 + v1) * (GPS == 2 && odd ? sc[GPS - 1] : sc[0]);
                            tot[r][a] += (g >> 1) == i ? v : 0.f;
                        }
                    }
                }
            } else {
                u32x4 bop[4];
                uint32_t lo = 0xE408E408u, hi = 0xD480D480u;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if constexpr (ZDEC) {
                        if (p % (4 / GPS) == 0) {
                            const uint32_t z = (t.z[r] >> (8 * (p * GPS / 4))) & 15u, zz = z | z << 16;
                            lo = 0xE400E400u + zz;
                            hi = 0xD400D400u + (zz << 4);
                        }
                    }
                    bop[p] = decode(t.w[r][0][p], b10, b6, lo, hi);
                }
                if constexpr (MA == 4) {         // piece p in lane group p, elements the rows
                    float4_t d[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) d[p] = mfma(t.a[0], bop[p], zero4);
                    const float s01 = g & 1 ? sc[1 * GPS / 4] : sc[0], s23 = g & 1 ? sc[3 * GPS / 4] : sc[2 * GPS / 4];
                    const float sg = g & 2 ? s23 : s01;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v01 = g & 1 ? d[1][e] : d[0][e], v23 = g & 1 ? d[3][e] : d[2][e];
                        tot[r][e] = fmaf(g & 2 ? v23 : v01, sg, tot[r][e]);
                    }
                } else if constexpr (MA == 8) {  // pieces 2 q + c, c = g / 2
                    const bool up = g & 2;
                    float4_t d0 = zero4, d1 = zero4;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        d0 = mfma(t.a[q], bop[2 * q], GPS == 1 && q ? d0 : zero4);
                        d1 = mfma(t.a[q], bop[2 * q + 1], GPS == 1 && q ? d1 : zero4);
                        if (GPS == 1 && q == 0) continue;
                        const float sq = GPS == 4 ? (up ? sc[GPS == 4 ? 2 * q + 1 : 0] : sc[GPS == 4 ? 2 * q : 0])
                                                  : sc[GPS == 2 ? q : 0];
#pragma unroll
                        for (int e = 0; e < 4; ++e) tot[r][e] = fmaf(up ? d1[e] : d0[e], sq, tot[r][e]);
                    }
                } else {                         // every lane its four rows
                    float4_t d = zero4;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        d = mfma(t.a[p], bop[p], p % (4 / GPS) ? d : zero4);
                        if ((p + 1) % (4 / GPS) == 0) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) tot[r][e] = fmaf(d[e], sc[p * GPS / 4], tot[r][e]);
                        }
                    }
                }
            }
        }
    };

    // units u < nu are this wave's (wave-uniform)
    const int nu = (KS + U - 1) / U;
    Unit t0, t1;
    int u = wv;
    if (u < nu) load(u, t0);
    for (; u < nu; u += 2 * NW) {
        if (u + NW < nu) load(u + NW, t1);
        run(t0);
        if (u + 2 * NW < nu) load(u + 2 * NW, t0);
        if (u + NW < nu) run(t1);
    }

    // sum over the lane groups that hold the same activation row, then over the waves in a fixed order
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int e = 0; e < TE; ++e) {
            float v = tot[r][e];
            if constexpr (MA <= 4) {
                v = sum_over_rows(v);
                if (g == 0) red[wv][e][16 * r + j] = v;
            } else if constexpr (MA == 8) {
                float a = v, b = v;
                swap32(a, b);
                v = a + b;
                if (g < 2) red[wv][4 * g + e][16 * r + j] = v;
            } else {
                red[wv][4 * g + e][16 * r + j] = v;
            }
        }
    __syncthreads();
    for (int o = threadIdx.x; o < MA * 16 * RB; o += 64 * NW) {
        const int m = o / (16 * RB), c = o % (16 * RB);
        const int64_t n = 16 * b0 + c;
        if (m < mm && n < N) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) y += red[w][m][c];
            const int64_t at = (int64_t)(m0 + m) * N + n;
            if (R) y += h2f(R[at]);
            Y[at] = __builtin_bit_cast(uint16_t, (_Float16)y);
        }
    }
}

// ---------------------------------------------------------------- product, 17 rows and more

typedef __attribute__((address_space(3))) char *lds_ptr_t;

// s_waitcnt vmcnt(N): at most N vector memory loads of this wave still outstanding (they retire in issue order)
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (((N >> 4) & 3) << 14));
}

// A barrier that waits for nothing itself: what it has to order (loads to LDS of this wave, and its LDS reads, whose values
// every product before it has used) is waited for explicitly.  __syncthreads() would wait for every load to LDS that is
// still in flight.
__device__ __forceinline__ void group_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// A workgroup computes 16 MT rows (MT = 2 or 4) x 128 outputs: four waves of two 16-output blocks side by side, and two
// such groups, each over every other step of the row, whose sums are added in LDS at the end.
//
// With more than 16 rows the activations, not the weights, are what is read most, so the four waves of a group share them:
// each step's 16 MT x 128 values are written into one of four LDS buffers by loads to LDS, up to three steps ahead, and a
// decoded B operand serves MT products.  In a buffer, piece q (8 values) of row r lies at position q ^ (r % 16) of its row,
// so that the 16 rows which one read touches at one piece fall in 16 distinct bank groups; a load instruction fills four
// rows, 256 consecutive bytes each.  Weights and scales go to registers, as far ahead.  The order of issue, a step's weights
// and then its activations, is what the waits count on.
//
// Measured at 64 rows, 8192 -> 28672, group 64: 50 us, of which the loads alone take 38 (the weights alone 28) and the
// products and decoding alone 36: the two overlap by half.  More outputs per wave, one group or four, two or three buffers
// were no faster (54 - 99 us).
constexpr int kMmWaves = 8;                      // waves of a workgroup: two groups of four

template <int MT, int GPS, bool ZP, bool TAIL>
__global__ __launch_bounds__(64 * kMmWaves) void k_int4_mm(const uint16_t *__restrict__ X, const uint8_t *__restrict__ codes,
                                                      const uint16_t *__restrict__ scales,
                                                      const uint8_t *__restrict__ zeros, int M, int N, int K, int KS,
                                                      const uint16_t *R, uint16_t *Y)
{
    constexpr int NB = 2, NW = 4, KG = 2, D = 4; // blocks per wave, waves per group, groups, buffers
    constexpr int NI = 4 * MT / NW;              // load instructions per wave and step: 16 MT rows, four each
    constexpr int NWL = NB * (ZP ? 3 : 2);       // loads of weights, scales and zero points per wave and step
    constexpr int kCols = NW * 16 * NB;           // outputs per workgroup
    constexpr int kBuf = MT * 16 * 16;           // 16-byte pieces of a group's step
    // (separate arrays, not one indexed by a variable: loads to LDS are waited for before LDS reads that the compiler
    // cannot prove disjoint from them, and it proves it for distinct arrays)
    __shared__ u32x4 buf0[KG * kBuf], buf1[KG * kBuf], buf2[KG * kBuf], buf3[KG * kBuf];
    auto buf_of = [&](int i) -> u32x4 * { return i == 0 ? buf0 : i == 1 ? buf1 : i == 2 ? buf2 : buf3; };

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % NW, kg = wave / NW;
    const int g = lane >> 4, j = lane & 15;
    // consecutive workgroups of an XCD (every eighth) take the row tiles of the same outputs
    const int tiles_m = (M + 16 * MT - 1) / (16 * MT);
    int wg = (int)blockIdx.x;
    if ((gridDim.x & 7) == 0) wg = (wg & 7) * ((int)gridDim.x >> 3) + (wg >> 3);
    const int m0 = wg % tiles_m * 16 * MT;
    const int64_t n0 = (int64_t)(wg / tiles_m) * kCols;
    const int64_t b0 = n0 / 16 + NB * wn;        // this wave's first block
    const int64_t blocks = ((int64_t)N + 15) / 16;
    const int nb = (int)(blocks - b0 < NB ? (blocks - b0 > 0 ? blocks - b0 : 0) : NB);
    const int64_t bs = b0 < blocks ? b0 : 0;     // (waves past the last block read nothing: empty resources)
    const int mm = min(16 * MT, M - m0);

    // Resources begin at the step that is read, so that a lane's offsets never change: a step costs scalar work only.
    const uint8_t *const cbase = codes + bs * KS * 1024;
    const uint16_t *const sbase = scales + bs * KS * (16 * GPS);
    const uint8_t *const zbase = ZP ? zeros + bs * KS * (16 * GPS) : nullptr;
    const uint16_t *const xbase = X + (int64_t)m0 * K;
    const uint32_t xbytes = __builtin_amdgcn_readfirstlane((uint32_t)mm * (uint32_t)K * 2u);

    // load instruction i of this wave: rows 4 (wn NI + i) + lane / 16, position lane % 16
    uint32_t xoff[NI];
    int klim[NI];                                // the piece's values exist in steps that begin below
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int row = 4 * (wn * NI + i) + g, q = j ^ (row & 15);
        xoff[i] = row < mm ? ((uint32_t)row * (uint32_t)K + 8u * (uint32_t)q) * 2u : kOob;
        klim[i] = K - 8 * q;
    }
    auto load_a = [&](int s, int buf) __attribute__((always_inline)) {
        const lds_ptr_t dst = (lds_ptr_t)(buf_of(buf) + kg * kBuf + wn * NI * 64);
        const bool in = s < KS;                  // (past the row's end: an empty resource)
        const __amdgpu_buffer_rsrc_t xr = rsrc(xbase + 128 * (int64_t)(in ? s : 0), in ? xbytes - 256u * (uint32_t)s : 0u);
#pragma unroll
        for (int i = 0; i < NI; ++i)             // (TAIL: pieces past K read zeros)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                xr, dst + 1024 * i, 16, (int)(!TAIL || 128 * s < klim[i] ? xoff[i] : kOob), 0, 0, 0);
    };
    struct Step {
        u32x4 w[NB];
        uint32_t s[NB][GPS == 4 ? 2 : 1];
        uint32_t z[NB];
    };
    auto load_w = [&](int s, Step &t) __attribute__((always_inline)) {
        const int si = s < KS ? s : 0;
        const uint32_t left = s < KS && nb > 0 ? (uint32_t)(nb * KS - s) : 0u;   // tiles from this step on (none past the end)
        const __amdgpu_buffer_rsrc_t wr = rsrc(cbase + 1024 * (int64_t)si, left * 1024u);
        const __amdgpu_buffer_rsrc_t sr = rsrc(sbase + 16 * GPS * (int64_t)si, left * (32u * GPS));
        const __amdgpu_buffer_rsrc_t zr = rsrc(ZP ? zbase + 16 * GPS * (int64_t)si : nullptr, ZP ? left * (16u * GPS) : 0u);
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            const uint32_t wo = (uint32_t)(r * KS) * 1024u + 16u * (uint32_t)lane, so = ((uint32_t)(r * KS) * 16u + (uint32_t)j) * GPS;
            t.w[r] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)wo, 0, 0);
            if constexpr (GPS == 4) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(sr, (int)(so * 2u), 0, 0);
                t.s[r][0] = v[0];
                t.s[r][1] = v[1];
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b32(zr, (int)so, 0, 0);
            } else if constexpr (GPS == 2) {
                t.s[r][0] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)(so * 2u), 0, 0);
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b16(zr, (int)so, 0, 0);
            } else {
                t.s[r][0] = __builtin_amdgcn_raw_buffer_load_b16(sr, (int)(so * 2u), 0, 0);
                if constexpr (ZP) t.z[r] = __builtin_amdgcn_raw_buffer_load_b8(zr, (int)so, 0, 0);
            }
        }
    };
    uint32_t b10, b6;
    asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(b10));
    asm volatile("v_mov_b32 %0, 0x54005400" : "=v"(b6));
    const float4_t zero4 = {0.f, 0.f, 0.f, 0.f};
    float4_t tot[MT][NB];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < NB; ++r) tot[m][r] = zero4;
    auto run = [&](const Step &t, int buf) __attribute__((always_inline)) {
        const u32x4 *const as = buf_of(buf) + kg * kBuf;
        float4_t d[MT][NB];
        u32x4 a[2][MT], b[2][NB];                // operands of two pieces in turn
        auto operands = [&](int p) __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < MT; ++m) a[p % 2][m] = as[(16 * m + j) * 16 + ((4 * p + g) ^ j)];
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                uint32_t lo = 0xE408E408u, hi = 0xD480D480u;
                if constexpr (ZP) {
                    const uint32_t z = (t.z[r] >> (8 * (p * GPS / 4))) & 15u, zz = z | z << 16;
                    lo = 0xE400E400u + zz;
                    hi = 0xD400D400u + (zz << 4);
                }
                b[p % 2][r] = decode(t.w[r][p], b10, b6, lo, hi);
            }
        };
        operands(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p < 3) operands(p + 1);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < NB; ++r) d[m][r] = mfma(a[p % 2][m], b[p % 2][r], p % (4 / GPS) ? d[m][r] : zero4);
            // the next piece's reads and decoding between the products
#pragma unroll
            for (int i = 0; i < MT * NB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // 1 MFMA
                if (i % NB == 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // 1 LDS read
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // 4 VALU
            }
            __builtin_amdgcn_sched_barrier(0);
            if ((p + 1) % (4 / GPS) == 0) {
                constexpr int kPer = GPS == 4 ? 2 : 1;
#pragma unroll
                for (int r = 0; r < NB; ++r) {
                    const int i = p * GPS / 4;
                    const float sc = h2f((uint16_t)(t.s[r][kPer == 2 ? i / 2 : 0] >> (GPS == 1 ? 0 : 16 * (i % 2))));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) tot[m][r][e] = fmaf(d[m][r][e], sc, tot[m][r][e]);
                }
            }
        }
    };

    // step i of this group is step kg + KG i of the row; steps past the end read zeros
    const int turns = ((KS + KG - 1) / KG + D - 1) / D * D;
    Step t[D];
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        load_w(kg + KG * i, t[i]);
        __builtin_amdgcn_sched_barrier(0);
        load_a(kg + KG * i, i);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int i = 0; i < turns; i += D) {
#pragma unroll
        for (int h = 0; h < D; ++h) {
            // this wave's share of the step's activations is in (younger: the D - 2 steps after it); behind the barrier
            // everybody's is, and everybody is done with the step before, whose buffer and registers are free
            wait_vm<(D - 2) * (NWL + NI)>();
            group_barrier();
            const int s = kg + KG * (i + h + D - 1), f = (h + D - 1) % D;
            __builtin_amdgcn_sched_barrier(0);
            load_w(s, t[f]);
            __builtin_amdgcn_sched_barrier(0);
            load_a(s, f);
            __builtin_amdgcn_sched_barrier(0);
            run(t[h], h);
        }
    }
    wait_vm<0>();                                // (the last loads to LDS, past the end, are in)
    __syncthreads();

    // the second group leaves its sums in a buffer, lane for lane, and the first adds them
    static_assert(KG == 2 && MT * NB * 64 * NW <= KG * kBuf, "a group's sums in one buffer");
    const int at = (int)threadIdx.x % (64 * NW);
    if (kg == 1) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < NB; ++r) buf0[(m * NB + r) * 64 * NW + at] = __builtin_bit_cast(u32x4, tot[m][r]);
    }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < NB; ++r) tot[m][r] += __builtin_bit_cast(float4_t, buf0[(m * NB + r) * 64 * NW + at]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 16 * m + 4 * g + e;
            if (row >= mm) continue;
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int64_t n = 16 * (b0 + r) + j, o = (int64_t)(m0 + row) * N + n;
                if (n >= N) continue;
                float y = tot[m][r][e];
                if (R) y += h2f(R[o]);
                Y[o] = __builtin_bit_cast(uint16_t, (_Float16)y);
            }
        }
}

uint16_t *scales_of(uint8_t *Wp, const Int4Map &m) { return reinterpret_cast<uint16_t *>(Wp + m.tiles() * 1024); }
uint8_t *zeros_of(uint8_t *Wp, const Int4Map &m) { return Wp + m.tiles() * 1024 + m.scales() * 2; }

int launched() { return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP; }

}  // namespace

int64_t int4_bytes(int64_t N, int64_t K, int group, bool zeros)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles || K >= kInt4MaxK) return -1;
    return m.tiles() * 1024 + m.scales() * (zeros ? 3 : 2);
}

int launch_int4_pack(const uint8_t *Q, const uint16_t *S, const uint8_t *Z, int N, int K, int group, uint8_t *Wp,
                     hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles || K >= kInt4MaxK) return TRI_EINVAL;
    hipLaunchKernelGGL(k_int4_pack, dim3((unsigned)m.tiles()), dim3(256), 0, s, Q, S, Z, N, K, (int)m.KS, m.gps,
                       reinterpret_cast<uint32_t *>(Wp), scales_of(Wp, m), Z ? zeros_of(Wp, m) : nullptr);
    return launched();
}

int launch_int4_unpack(const uint8_t *Wp, int N, int K, int group, bool zeros, uint8_t *Q, uint16_t *S, uint8_t *Z,
                       hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles || K >= kInt4MaxK) return TRI_EINVAL;
    uint8_t *p = const_cast<uint8_t *>(Wp);      // (read only)
    hipLaunchKernelGGL(k_int4_unpack, dim3((unsigned)m.tiles()), dim3(256), 0, s, reinterpret_cast<const uint32_t *>(Wp),
                       scales_of(p, m), zeros ? zeros_of(p, m) : nullptr, N, K, (int)m.KS, m.gps, Q, S, Z);
    return launched();
}

int launch_int4_quantize(const float *W, int N, int K, int group, bool zeros, uint8_t *Wp, hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles || K >= kInt4MaxK) return TRI_EINVAL;
    hipLaunchKernelGGL(k_int4_quantize, dim3((unsigned)m.tiles()), dim3(256), 0, s, W, N, K, (int)m.KS, m.gps,
                       reinterpret_cast<uint32_t *>(Wp), scales_of(Wp, m), zeros ? zeros_of(Wp, m) : nullptr);
    return launched();
}

namespace {

struct Int4Args {
    const uint16_t *X;
    const uint8_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    int M, N, K, KS;
    const uint16_t *R;
    uint16_t *Y;
};

template <int MA, int RB, int GPS, bool ZP, bool VEC>
void mv_go(const Int4Args &a, hipStream_t s)
{
    constexpr int NW = 8;
    const int blocks = (a.N + 15) / 16;
    hipLaunchKernelGGL((k_int4_mv<MA, RB, GPS, ZP, NW, VEC>), dim3((blocks + RB - 1) / RB, (a.M + MA - 1) / MA),
                       dim3(64 * NW), 0, s, a.X, a.codes, a.scales, a.zeros, a.M, a.N, a.K, a.KS, a.R, a.Y);
}

template <int MA, int RB, bool VEC>
void mv_fmt(const Int4Args &a, int gps, hipStream_t s)
{
    if (a.zeros) {
        if (gps == 1) mv_go<MA, RB, 1, true, VEC>(a, s);
        else if (gps == 2) mv_go<MA, RB, 2, true, VEC>(a, s);
        else mv_go<MA, RB, 4, true, VEC>(a, s);
    } else {
        if (gps == 1) mv_go<MA, RB, 1, false, VEC>(a, s);
        else if (gps == 2) mv_go<MA, RB, 2, false, VEC>(a, s);
        else mv_go<MA, RB, 4, false, VEC>(a, s);
    }
}

// Blocks per workgroup: the busiest CU's rounds times (1 + RB), a workgroup costing about one block's work on top of
// its blocks (the activations it loads), at most four; the larger on a tie.  Measured at 8 rows, group 128: 688 blocks
// (4096 -> 11008) 9.0 / 8.5 / 7.4 / 7.9 us with RB = 1 .. 4 (3 taken), 256 blocks (11008 -> 4096) 8.4 / 10.0 / 12.3 /
// 14.3 (1), 1792 blocks (8192 -> 28672) 38.4 / 29.5 / 29.3 / 29.1 (4); 64 rows in four slices 43 / 25 / - / 17.8 on 256
// blocks (4).
int blocks_per_workgroup(int64_t blocks, int64_t slices)
{
    const int64_t cus = cu_count();
    int best = 1;
    int64_t least = -1;
    for (int rb = 4; rb >= 1; --rb) {
        const int64_t cost = ((blocks + rb - 1) / rb * slices + cus - 1) / cus * (1 + rb);
        if (least < 0 || cost < least) {
            best = rb;
            least = cost;
        }
    }
    return best;
}

template <int MA, bool VEC>
void mv_rb(const Int4Args &a, int gps, hipStream_t s)
{
    switch (blocks_per_workgroup((a.N + 15) / 16, (a.M + MA - 1) / MA)) {
    case 1: mv_fmt<MA, 1, VEC>(a, gps, s); break;
    case 2: mv_fmt<MA, 2, VEC>(a, gps, s); break;
    case 3: mv_fmt<MA, 3, VEC>(a, gps, s); break;
    default: mv_fmt<MA, 4, VEC>(a, gps, s); break;
    }
}

constexpr int kMmMaxK = 1 << 24;                 // 32-bit offsets over 64 activation rows

template <int MT, int GPS, bool ZP>
void mm_go(const Int4Args &a, hipStream_t s)
{
    const int64_t wgs = (int64_t)((a.M + 16 * MT - 1) / (16 * MT)) * (((int64_t)a.N + 127) / 128);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(64 * kMmWaves), 0, s, a.X, a.codes, a.scales, a.zeros, a.M, a.N, a.K, a.KS,
                           a.R, a.Y);
    };
    if (a.K % 128) go(k_int4_mm<MT, GPS, ZP, true>);
    else go(k_int4_mm<MT, GPS, ZP, false>);
}

template <int MT>
void mm_fmt(const Int4Args &a, int gps, hipStream_t s)
{
    if (a.zeros) {
        if (gps == 1) mm_go<MT, 1, true>(a, s);
        else if (gps == 2) mm_go<MT, 2, true>(a, s);
        else mm_go<MT, 4, true>(a, s);
    } else {
        if (gps == 1) mm_go<MT, 1, false>(a, s);
        else if (gps == 2) mm_go<MT, 2, false>(a, s);
        else mm_go<MT, 4, false>(a, s);
    }
}

void mv_rows(const Int4Args &a, int gps, hipStream_t s)
{
    if (a.K % 8) {
        if (a.M <= 4) mv_fmt<4, 1, false>(a, gps, s);
        else mv_rb<16, false>(a, gps, s);
        return;
    }
    // The shared-activation kernel from five eighths of a round of its smaller tiles on (32 x 128), with the larger ones (64
    // rows) where those still make as many.  64 rows: 8192 -> 28672 94 -> 47 us (group 128), 4096 -> 11008 23.4 -> 15.2 us;
    // with 64 tiles (11008 -> 4096) it would lose, 17.6 against 31 us.
    if (a.M > 16 && a.K < kMmMaxK) {
        const int64_t cols = ((int64_t)a.N + 127) / 128, enough = 5 * (int64_t)cu_count() / 8;
        if ((a.M + 63) / 64 * cols >= enough && a.M > 32) return mm_fmt<4>(a, gps, s);
        if ((a.M + 31) / 32 * cols >= enough) return mm_fmt<2>(a, gps, s);
    }
    // up to four rows one block per workgroup: the activations are few (more blocks lost 10 - 90% at 256 and 688 blocks,
    // and at most 5% was won at 1792)
    if (a.M <= 1) mv_fmt<1, 1, true>(a, gps, s);
    else if (a.M <= 2) mv_fmt<2, 1, true>(a, gps, s);
    else if (a.M <= 4) mv_fmt<4, 1, true>(a, gps, s);
    else if (a.M <= 8) mv_rb<8, true>(a, gps, s);
    else mv_rb<16, true>(a, gps, s);
}

}  // namespace

int launch_int4_linear(const uint16_t *X, const uint8_t *Wp, int M, int N, int K, int group, bool zeros,
                       const uint16_t *R, uint16_t *Y, hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles || K >= kInt4MaxK) return TRI_EINVAL;
    uint8_t *p = const_cast<uint8_t *>(Wp);      // (read only)
    // Rows per launch: at most 65535 16-row slices (the second grid dimension) and 2^22 tiles of 32 x 128 (a grid has
    // fewer than 2^32 threads), a multiple of 64.
    const int64_t cols = ((int64_t)N + 127) / 128, tiles = ((int64_t)1 << 22) / cols * 32 / 64 * 64;
    const int64_t most = tiles < 64 ? 64 : tiles < 16 * 65535 ? tiles : 16 * 65535;
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        const int rows = (int)(M - m0 < most ? M - m0 : most);
        const Int4Args a{X + m0 * K, Wp, scales_of(p, m), zeros ? zeros_of(p, m) : nullptr, rows, N, K, (int)m.KS,
                         R ? R + m0 * N : nullptr, Y + m0 * N};
        mv_rows(a, m.gps, s);
    }
    return launched();
}

}  // namespace tri
