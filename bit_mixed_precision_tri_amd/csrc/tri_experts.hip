// tri_experts.hip -- experts: routing, ragged ternary products, combination (include/tri.h).
//
//   route    top-k of every token's logits and the stable order of the (token, expert) pairs by expert
//   product  Y[r] = scale[e] X[rows[r]] W_e^T for the places r of expert e, one matrix or a gated pair
//   combine  Y[t] = residual[t] + sum_j weights[t][j] Z[pos[t][j]]
#include "tri_device.h"
#include "tri_internal.h"

namespace tri {

namespace {

int launched() { return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP; }

// ---------------------------------------------------------------- routing

constexpr int kRouteThreads = 512;               // eight waves; one (token, expert) pair per thread
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = 32;                 // tokens per workgroup where there are several (32 * 16 pairs at most)
constexpr int kMaxCols = TRI_MAX_EXPERTS + 1;    // the last bucket holds the pairs that take no expert

__device__ __forceinline__ float wave_max(float v)
{
    float a = v, b = v;
    swap32(a, b);
    v = fmaxf(a, b);
    a = b = v;
    swap16(a, b);
    v = fmaxf(a, b);
    v = fmaxf(v, dpp<0x140>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    return fmaxf(v, dpp<0xB1>(v));
}

__device__ __forceinline__ float wave_sum(float v)
{
    float a[1] = {v};
    return wave_reduce_rows<1>(a, 0);
}

// Exclusive prefix sums of total[0 .. cols-1] into first[] (first wave; cols <= 64 * 5).
__device__ __forceinline__ void scan_cols(const int *total, int *first, int cols, int lane)
{
    int v[5], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        v[i] = 5 * lane + i < cols ? total[5 * lane + i] : 0;
        sum += v[i];
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d, 64);
        if (lane >= d) run += o;
    }
    run -= sum;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        if (5 * lane + i < cols) first[5 * lane + i] = run;
        run += v[i];
    }
}

// One workgroup per TB tokens.  A wave takes one token at a time: lane l holds logits EP l .. EP l + EP-1, so
// the lowest lane among equals holds the lowest expert.  Then thread i ranks pair i of the workgroup among the
// pairs before it with the same expert: lanes that agree in all nine bits of the bucket number (ballots), and
// counts of the waves before.  With one workgroup (hist null) that finishes the order; otherwise the counts go
// to hist[block][bucket], the ranks to pos, and k_route_place finishes.
template <bool HALF, int EP>
__global__ __launch_bounds__(kRouteThreads) void k_route(const void *__restrict__ logits, int T, int E, int topk,
                                                         int renorm, int TB, int32_t *__restrict__ ids,
                                                         float *__restrict__ weights, int32_t *__restrict__ offsets,
                                                         int32_t *__restrict__ rows, int32_t *__restrict__ pos,
                                                         int32_t *__restrict__ hist)
{
    __shared__ int bucket[kRouteThreads];
    __shared__ int count[kRouteWaves][kMaxCols];
    __shared__ int total[kMaxCols], first[kMaxCols];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t0 = blockIdx.x * TB, nt = min(TB, T - t0), cols = E + 1;
    for (int i = threadIdx.x; i < kRouteWaves * kMaxCols; i += kRouteThreads) (&count[0][0])[i] = 0;
    const float ninf = -__builtin_inff();
    for (int tt = wv; tt < nt; tt += kRouteWaves) {
        const int64_t t = t0 + tt;
        float v[EP];
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int e = EP * lane + i;
            v[i] = ninf;
            if (e < E) {
                const float x = HALF ? h2f(static_cast<const uint16_t *>(logits)[t * E + e])
                                     : static_cast<const float *>(logits)[t * E + e];
                v[i] = x == x ? x : ninf;
            }
        }
        float top = v[0];
#pragma unroll
        for (int i = 1; i < EP; ++i) top = fmaxf(top, v[i]);
        const float mx = wave_max(top);
        auto mass = [&](float x) { return x == mx ? 1.f : expf(x - mx); };   // (x, mx > -inf; inf against inf: 1)
        float whole = 0.f;
        if (!renorm) {
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (v[i] > ninf) whole += mass(v[i]);
            whole = wave_sum(whole);
        }
        int my_e = -1;
        float my_v = ninf;
        for (int j = 0; j < topk; ++j) {
            float best = v[0];
#pragma unroll
            for (int i = 1; i < EP; ++i) best = fmaxf(best, v[i]);
            const float w = wave_max(best);
            if (!(w > ninf)) break;              // (wave-uniform) nothing left to take
            const int src = __ffsll((unsigned long long)__ballot(best == w)) - 1;
            int li = 0;
#pragma unroll
            for (int i = EP - 1; i >= 0; --i)
                if (v[i] == w) li = i;
            const int e = __builtin_amdgcn_readlane(EP * lane + li, src);
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (EP * lane + i == e) v[i] = ninf;
            if (lane == j) {
                my_e = e;
                my_v = w;
            }
        }
        const float m = my_e >= 0 ? mass(my_v) : 0.f;
        if (renorm) whole = wave_sum(m);
        if (lane < topk) {
            ids[t * topk + lane] = my_e;
            weights[t * topk + lane] = my_e >= 0 ? m / whole : 0.f;
            bucket[tt * topk + lane] = my_e >= 0 ? my_e : E;
        }
    }
    __syncthreads();
    const int n = nt * topk, i = threadIdx.x;
    const int b = i < n ? bucket[i] : kMaxCols;  // (a bucket of its own for threads without a pair)
    unsigned long long same = ~0ull;
#pragma unroll
    for (int bit = 0; bit < 9; ++bit) {
        const unsigned long long has = __ballot((b >> bit) & 1);
        same &= (b >> bit) & 1 ? has : ~has;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    if (i < n && before == 0) count[wv][b] = __popcll(same);
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += kRouteThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) {
            const int x = count[w][c];
            count[w][c] = run;
            run += x;
        }
        total[c] = run;
        if (hist) hist[(int64_t)blockIdx.x * cols + c] = run;
    }
    __syncthreads();
    const int64_t p = (int64_t)t0 * topk + i;
    if (hist) {
        if (i < n) pos[p] = count[wv][b] + before;
        return;
    }
    if (wv == 0) scan_cols(total, first, cols, lane);
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += kRouteThreads) offsets[c] = first[c];
    if (i < n) {
        const int place = first[b] + count[wv][b] + before;
        pos[p] = b < E ? place : -1;
        rows[place] = b < E ? t0 + i / topk : -1;
    }
}

// Many workgroups: workgroup c turns column c of the counts into sums over the workgroups before, and writes the
// column's total behind the last row.
__global__ __launch_bounds__(kRouteThreads) void k_route_scan(int nb, int cols, int32_t *__restrict__ hist)
{
    __shared__ int sums[kRouteWaves];
    const int c = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int carry = 0;
    for (int b0 = 0; b0 < nb; b0 += kRouteThreads) {
        const int b = b0 + threadIdx.x;
        const int x = b < nb ? hist[(int64_t)b * cols + c] : 0;
        int run = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(run, d, 64);
            if (lane >= d) run += o;
        }
        if (lane == 63) sums[wv] = run;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) {
            if (w < wv) run += sums[w];
            all += sums[w];
        }
        if (b < nb) hist[(int64_t)b * cols + c] = carry + run - x;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) hist[(int64_t)nb * cols + c] = carry;
}

// The order's last step: workgroup b takes the sum per bucket of all workgroups and of those before it (added here, or
// by k_route_scan where scanned), and turns the ranks of its pairs into places.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(int T, int E, int topk, int scanned,
                                                               const int32_t *__restrict__ ids,
                                                               const int32_t *__restrict__ hist,
                                                               int32_t *__restrict__ offsets,
                                                               int32_t *__restrict__ rows, int32_t *__restrict__ pos)
{
    __shared__ int part[2][kRouteThreads];
    __shared__ int total[kMaxCols], first[kMaxCols], mine[kMaxCols];
    const int cols = E + 1, nb = gridDim.x, me = blockIdx.x;
    if (scanned) {
        if ((int)threadIdx.x < cols) {
            total[threadIdx.x] = hist[(int64_t)nb * cols + threadIdx.x];
            mine[threadIdx.x] = hist[(int64_t)me * cols + threadIdx.x];
        }
    } else {
        const int slices = kRouteThreads / cols; // >= 1 (cols <= 257)
        const int c = threadIdx.x % cols, s = threadIdx.x / cols;
        int all = 0, prev = 0;
        if (s < slices) {
            for (int b = s; b < nb; b += slices) {
                const int x = hist[(int64_t)b * cols + c];
                all += x;
                prev += b < me ? x : 0;
            }
        }
        part[0][threadIdx.x] = all;
        part[1][threadIdx.x] = prev;
        __syncthreads();
        if ((int)threadIdx.x < cols) {
            for (int q = 1; q < slices; ++q) {
                all += part[0][q * cols + threadIdx.x];
                prev += part[1][q * cols + threadIdx.x];
            }
            total[threadIdx.x] = all;
            mine[threadIdx.x] = prev;
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) scan_cols(total, first, cols, threadIdx.x);
    __syncthreads();
    if (me == 0)
        for (int q = threadIdx.x; q < cols; q += kRouteThreads) offsets[q] = first[q];
    const int64_t t0 = (int64_t)me * kRouteTokens;
    const int n = (int)min((int64_t)kRouteTokens, T - t0) * topk;
    if ((int)threadIdx.x < n) {
        const int64_t p = t0 * topk + threadIdx.x;
        const int e = ids[p], b = e >= 0 ? e : E;
        const int place = first[b] + mine[b] + pos[p];
        pos[p] = e >= 0 ? place : -1;
        rows[place] = e >= 0 ? (int)(t0 + threadIdx.x / topk) : -1;
    }
}

// One workgroup does all of it while its pairs fit its threads and a wave has few tokens.
bool route_single(int T, int topk) { return (int64_t)T * topk <= kRouteThreads && T <= 4 * kRouteTokens; }
int route_blocks(int T) { return (T + kRouteTokens - 1) / kRouteTokens; }
// From here on the counts are scanned by a launch of their own (below, every workgroup adds all of them).
constexpr int kRouteScanBlocks = 256;

// ---------------------------------------------------------------- product

// Simple form: one wave per place and output.
template <int FMT>
__global__ __launch_bounds__(256) void k_experts_rows(const Experts ex, int S)
{
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int r = (int)(w / ex.N), n = (int)(w % ex.N);
    if (r >= ex.R) return;
    int e = -1;
    for (int q = 0; q < ex.E; ++q)
        if (r >= ex.offsets[q] && r < ex.offsets[q + 1]) e = q;
    if (e < 0) return;
    const int x = ex.rows ? ex.rows[r] : r;
    if (x < 0 || x >= ex.T) return;
    constexpr int PER = FMT == TRI_FMT_2BIT ? 4 : 5, BASE = FMT == TRI_FMT_2BIT ? 4 : 3;
    float y[2] = {0.f, 0.f};
    for (int q = 0; q < 2; ++q) {
        if (!ex.Wp[q]) break;
        const uint8_t *row = ex.Wp[q] + ((int64_t)e * ex.N + n) * S;
        float acc[1] = {0.f};
        for (int b = lane; b < S; b += 64) {
            int v = row[b];
            for (int i = 0; i < PER; ++i, v /= BASE)
                if (PER * b + i < ex.K) acc[0] += (float)(v % BASE - 1) * h2f(ex.X[(int64_t)x * ex.K + PER * b + i]);
        }
        y[q] = wave_reduce_rows<1>(acc, lane) * ex.scale[q][e];
    }
    const float o = ex.Wp[1] ? y[0] / (1.f + __expf(-y[0])) * y[1] : y[0];
    if (lane == 0) ex.Y[(int64_t)r * ex.N + n] = __builtin_bit_cast(uint16_t, (_Float16)o);
}

// ---------------------------------------------------------------- combination

// Thread p of the grid's stride loop owns VEC values (one 16-byte piece, or one value where rows are not whole
// pieces) of one token; JT >= topk sources, all requested before the first is added.
template <int JT, int VEC>
__global__ __launch_bounds__(256) void k_combine(const uint16_t *__restrict__ Z, int64_t R,
                                                 const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                                 const uint16_t *res, int T, int topk, int N, uint16_t *Y)
{
    const int64_t per = N / VEC, all = per * T;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < all; p += (int64_t)gridDim.x * 256) {
        const int64_t t = p / per, c = (p - t * per) * VEC;
        float w[JT];
        uint4 z[JT];
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            w[j] = 0.f;
            z[j] = uint4{0, 0, 0, 0};
            if (j < topk) {
                const int r = pos[t * topk + j];
                if (r >= 0 && r < R) {
                    w[j] = weights[t * topk + j];
                    if constexpr (VEC == 8) z[j] = ld16(Z + r * (int64_t)N + c);
                    else z[j].x = Z[r * (int64_t)N + c];
                }
            }
        }
        uint4 old = {0, 0, 0, 0};
        if (res) {
            if constexpr (VEC == 8) old = ld16(res + t * N + c);
            else old.x = res[t * N + c];
        }
        uint32_t out[4];
#pragma unroll
        for (int q = 0; q < (VEC + 1) / 2; ++q) {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                const uint32_t v = (&z[j].x)[q];
                lo = fmaf(w[j], h2f((uint16_t)v), lo);
                hi = fmaf(w[j], h2f((uint16_t)(v >> 16)), hi);
            }
            const uint32_t v = (&old.x)[q];
            lo += h2f((uint16_t)v);
            hi += h2f((uint16_t)(v >> 16));
            out[q] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
                     (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
        }
        if constexpr (VEC == 8) *reinterpret_cast<uint4 *>(Y + t * N + c) = uint4{out[0], out[1], out[2], out[3]};
        else Y[t * N + c] = (uint16_t)out[0];
    }
}

template <int JT>
void combine_jt(const uint16_t *Z, int64_t R, const int32_t *pos, const float *weights, const uint16_t *res, int T,
                int topk, int N, uint16_t *Y, hipStream_t s)
{
    const bool vec = N % 8 == 0;
    const int64_t all = (int64_t)(vec ? N / 8 : N) * T, wgs = (all + 255) / 256;
    const dim3 grid((unsigned)(wgs < 65536 ? wgs : 65536));
    if (vec) hipLaunchKernelGGL((k_combine<JT, 8>), grid, dim3(256), 0, s, Z, R, pos, weights, res, T, topk, N, Y);
    else hipLaunchKernelGGL((k_combine<JT, 1>), grid, dim3(256), 0, s, Z, R, pos, weights, res, T, topk, N, Y);
}

}  // namespace

int64_t route_workspace_bytes(int64_t T, int E, int topk)
{
    if (route_single((int)T, topk)) return 0;
    return ((int64_t)(route_blocks((int)T) + 1) * (E + 1) * 4 + 15) / 16 * 16;
}

int launch_route(const void *logits, bool half, int T, int E, int topk, bool renorm, int32_t *ids, float *weights,
                 int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace, hipStream_t s)
{
    const bool single = route_single(T, topk);
    const int blocks = single ? 1 : route_blocks(T), TB = single ? T : kRouteTokens;
    int32_t *hist = single ? nullptr : static_cast<int32_t *>(workspace);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kRouteThreads), 0, s, logits, T, E, topk, renorm ? 1 : 0, TB, ids,
                           weights, offsets, rows, pos, hist);
    };
    if (half) {
        if (E <= 64) go(k_route<true, 1>);
        else if (E <= 128) go(k_route<true, 2>);
        else go(k_route<true, 4>);
    } else {
        if (E <= 64) go(k_route<false, 1>);
        else if (E <= 128) go(k_route<false, 2>);
        else go(k_route<false, 4>);
    }
    if (!single) {
        const bool scan = blocks > kRouteScanBlocks;
        if (scan) hipLaunchKernelGGL(k_route_scan, dim3(E + 1), dim3(kRouteThreads), 0, s, blocks, E + 1, hist);
        hipLaunchKernelGGL(k_route_place, dim3(blocks), dim3(kRouteThreads), 0, s, T, E, topk, scan ? 1 : 0, ids, hist,
                           offsets, rows, pos);
    }
    return launched();
}

int launch_experts(const Experts &ex, int fmt, hipStream_t s)
{
    const int S = (int)row_bytes(ex.K, fmt);
    const int64_t wgs = ((int64_t)ex.R * ex.N + 3) / 4;
    if (wgs >= ((int64_t)1 << 24)) return TRI_EINVAL;
    if (fmt == TRI_FMT_2BIT) hipLaunchKernelGGL(k_experts_rows<TRI_FMT_2BIT>, dim3((unsigned)wgs), dim3(256), 0, s, ex, S);
    else hipLaunchKernelGGL(k_experts_rows<TRI_FMT_1P6BIT>, dim3((unsigned)wgs), dim3(256), 0, s, ex, S);
    return launched();
}

int launch_combine(const uint16_t *Z, int64_t R, const int32_t *pos, const float *weights, const uint16_t *res, int T,
                   int topk, int N, uint16_t *Y, hipStream_t s)
{
    if (topk <= 1) combine_jt<1>(Z, R, pos, weights, res, T, topk, N, Y, s);
    else if (topk <= 2) combine_jt<2>(Z, R, pos, weights, res, T, topk, N, Y, s);
    else if (topk <= 4) combine_jt<4>(Z, R, pos, weights, res, T, topk, N, Y, s);
    else if (topk <= 8) combine_jt<8>(Z, R, pos, weights, res, T, topk, N, Y, s);
    else combine_jt<16>(Z, R, pos, weights, res, T, topk, N, Y, s);
    return launched();
}

}  // namespace tri
