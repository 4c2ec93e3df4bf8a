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

Int4Map int4_map(int64_t N, int64_t K, int group) { return {(N + 15) / 16, (K + 127) / 128, 128 / group}; }

// bit position of value i of a word
__device__ __forceinline__ int nibble_at(int i) { return 4 * (i / 2) + 16 * (i % 2); }

// One workgroup per tile (block b, step s): thread (j, q) packs piece q (8 values) of row j.  Threads
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

// The product, one wave per weight row and eight activation rows: lanes own pieces of eight values.
__global__ __launch_bounds__(256) void k_int4_rows(const uint16_t *__restrict__ X, const uint32_t *__restrict__ codes,
                                                   const uint16_t *__restrict__ scales,
                                                   const uint8_t *__restrict__ zeros, int M, int N, int K, int KS,
                                                   int gps, const uint16_t *R, uint16_t *Y)
{
    const int lane = threadIdx.x & 63;
    const int64_t n = 4 * (int64_t)blockIdx.x + (threadIdx.x >> 6);
    if (n >= N) return;
    const int64_t b = n / 16, j = n % 16;
    for (int64_t m0 = 8 * (int64_t)blockIdx.y; m0 < M; m0 += 8 * (int64_t)gridDim.y) {
        float acc[8] = {};
        for (int64_t q = lane; q < 16 * (int64_t)KS; q += 64) {
            const int64_t tile = b * KS + q / 16;
            const int qq = (int)(q % 16);
            const uint32_t w = codes[tile * 256 + (16 * (qq & 3) + j) * 4 + (qq >> 2)];
            const int64_t o = (tile * 16 + j) * gps + qq * gps / 16;
            const float sc = h2f(scales[o]);
            const int z = zeros ? zeros[o] : 8;
            for (int i = 0; i < 8; ++i) {
                const int64_t k = 8 * q + i;
                if (k >= K) break;
                const float wv = sc * (float)((int)((w >> nibble_at(i)) & 15u) - z);
                for (int r = 0; r < 8; ++r)
                    if (m0 + r < M) acc[r] += wv * h2f(X[(m0 + r) * K + k]);
            }
        }
        const float t = wave_reduce_rows<8>(acc, lane);
        const int64_t m = m0 + (lane >> 3);
        if ((lane & 7) == 0 && m < M) {
            float y = t;
            if (R) y += h2f(R[m * N + n]);
            Y[m * N + n] = __builtin_bit_cast(uint16_t, (_Float16)y);
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
    if (m.tiles() >= kInt4MaxTiles) return -1;
    return m.tiles() * 1024 + m.scales() * (zeros ? 3 : 2);
}

int launch_int4_pack(const uint8_t *Q, const uint16_t *S, const uint8_t *Z, int N, int K, int group, uint8_t *Wp,
                     hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles) return TRI_EINVAL;
    hipLaunchKernelGGL(k_int4_pack, dim3((unsigned)m.tiles()), dim3(256), 0, s, Q, S, Z, N, K, (int)m.KS, m.gps,
                       reinterpret_cast<uint32_t *>(Wp), scales_of(Wp, m), Z ? zeros_of(Wp, m) : nullptr);
    return launched();
}

int launch_int4_unpack(const uint8_t *Wp, int N, int K, int group, bool zeros, uint8_t *Q, uint16_t *S, uint8_t *Z,
                       hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles) return TRI_EINVAL;
    uint8_t *p = const_cast<uint8_t *>(Wp);      // (read only)
    hipLaunchKernelGGL(k_int4_unpack, dim3((unsigned)m.tiles()), dim3(256), 0, s, reinterpret_cast<const uint32_t *>(Wp),
                       scales_of(p, m), zeros ? zeros_of(p, m) : nullptr, N, K, (int)m.KS, m.gps, Q, S, Z);
    return launched();
}

int launch_int4_quantize(const float *W, int N, int K, int group, bool zeros, uint8_t *Wp, hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles) return TRI_EINVAL;
    hipLaunchKernelGGL(k_int4_quantize, dim3((unsigned)m.tiles()), dim3(256), 0, s, W, N, K, (int)m.KS, m.gps,
                       reinterpret_cast<uint32_t *>(Wp), scales_of(Wp, m), zeros ? zeros_of(Wp, m) : nullptr);
    return launched();
}

int launch_int4_linear(const uint16_t *X, const uint8_t *Wp, int M, int N, int K, int group, bool zeros,
                       const uint16_t *R, uint16_t *Y, hipStream_t s)
{
    const Int4Map m = int4_map(N, K, group);
    if (m.tiles() >= kInt4MaxTiles) return TRI_EINVAL;
    uint8_t *p = const_cast<uint8_t *>(Wp);      // (read only)
    const int64_t rows = ((int64_t)M + 7) / 8;
    hipLaunchKernelGGL(k_int4_rows, dim3((unsigned)((N + 3) / 4), (unsigned)(rows < 32768 ? rows : 32768)), dim3(256), 0,
                       s, X, reinterpret_cast<const uint32_t *>(Wp), scales_of(p, m), zeros ? zeros_of(p, m) : nullptr, M,
                       N, K, (int)m.KS, m.gps, R, Y);
    return launched();
}

}  // namespace tri
