// tri_experts.hip -- experts: routing, ragged ternary products, combination (include/tri.h).
//
//   route    top-k of every token's logits and the stable order of the (token, expert) pairs by expert
//   product  Y[r] = scale[e] X[rows[r]] W_e^T for the places r of expert e, one matrix or a gated pair
//   combine  Y[t] = residual[t] + sum_j weights[t][j] Z[pos[t][j]]
#include <type_traits>

#include "tri_experts.h"

namespace tri {

namespace {

int launched() { return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP; }

// ---------------------------------------------------------------- routing

constexpr int kRouteThreads = 512;               // eight waves; one (token, expert) pair per thread
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = 32;                 // tokens per workgroup where there are several (32 * 16 pairs at most)
constexpr int kMaxCols = TRI_MAX_EXPERTS + 1;    // the last bucket holds the pairs that take no expert

// Over the 16 lanes of a row, in every one of them.
template <typename F>
__device__ __forceinline__ float row_all(float v, F f)
{
    v = f(v, dpp<0x140>(v));                     // row_mirror: lane ^ 15
    v = f(v, dpp<0x141>(v));                     // row_half_mirror: lane ^ 7
    v = f(v, dpp<0x4E>(v));                      // lane ^ 2
    return f(v, dpp<0xB1>(v));                   // lane ^ 1
}
__device__ __forceinline__ float row_max(float v) { return row_all(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float row_min(float v) { return row_all(v, [](float a, float b) { return fminf(a, b); }); }
__device__ __forceinline__ float row_sum(float v) { return row_all(v, [](float a, float b) { return a + b; }); }

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

// One workgroup per TB tokens.  A row of 16 lanes takes a token, four a wave: lane l holds logits EP l .. EP l + EP-1.
// Each round takes the row's largest value and, among the lanes that hold it, the lowest expert (as an exact small float:
// the row reductions are those of floats).  Then thread i ranks pair i of the workgroup among the pairs before it with
// the same expert: lanes that agree in all nine bits of the bucket number (ballots), and counts of the waves before.  With
// one workgroup (hist null) that finishes the order; otherwise the counts go to hist[block][bucket], the ranks to pos, and
// k_route_place finishes.
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
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane & 15;
    const int t0 = blockIdx.x * TB, nt = min(TB, T - t0), cols = E + 1;
    const float ninf = -__builtin_inff();
    for (int i = threadIdx.x; i < kRouteWaves * kMaxCols; i += kRouteThreads) (&count[0][0])[i] = 0;
    for (int tw = 4 * wv; tw < nt; tw += 4 * kRouteWaves) {   // (wave-uniform)
        const int tt = tw + (lane >> 4);
        const int64_t t = t0 + min(tt, nt - 1);  // (rows past the end repeat the last token and write nothing)
        float v[EP];
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int e = EP * l + i;
            v[i] = ninf;
            if (e < E) {
                const float x = HALF ? h2f(static_cast<const uint16_t *>(logits)[t * E + e])
                                     : static_cast<const float *>(logits)[t * E + e];
                v[i] = x == x ? x : ninf;
            }
        }
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < EP; ++i) mx = fmaxf(mx, v[i]);
        mx = row_max(mx);
        auto mass = [&](float x) { return x == mx ? 1.f : expf(x - mx); };   // (x, mx > -inf; inf against inf: 1)
        float whole = 0.f;
        if (!renorm) {
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (v[i] > ninf) whole += mass(v[i]);
            whole = row_sum(whole);
        }
        int my_e = -1;
        float my_v = ninf;
        for (int j = 0; j < topk; ++j) {
            float best = v[0];
#pragma unroll
            for (int i = 1; i < EP; ++i) best = fmaxf(best, v[i]);
            const float w = row_max(best);
            float at = 1024.f;                   // this lane's lowest expert of that value
#pragma unroll
            for (int i = EP - 1; i >= 0; --i) at = v[i] == w ? (float)(EP * l + i) : at;
            const int e = (int)row_min(at);
#pragma unroll
            for (int i = 0; i < EP; ++i) v[i] = EP * l + i == e ? ninf : v[i];
            if (l == j && w > ninf) {
                my_e = e;
                my_v = w;
            }
        }
        const float m = my_e >= 0 ? mass(my_v) : 0.f;
        if (renorm) whole = row_sum(m);
        if (l < topk && tt < nt) {
            ids[t * topk + l] = my_e;
            weights[t * topk + l] = my_e >= 0 ? m / whole : 0.f;
            bucket[tt * topk + l] = my_e >= 0 ? my_e : E;
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

// Bound by latency, not by its few bytes: 4095 tokens of 64 experts take 9.3 us in two launches (5.4 and 4.8 us under the
// profiler), one token 3.3 us in one, where an empty launch takes 1.9.
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
#pragma unroll 8
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

// One workgroup does all of it while its pairs fit its threads and a row of lanes has few tokens.
bool route_single(int T, int topk) { return (int64_t)T * topk <= kRouteThreads && T <= 4 * kRouteTokens; }
int route_blocks(int T) { return (T + kRouteTokens - 1) / kRouteTokens; }
// From here on the counts are scanned by a launch of their own (below, every workgroup adds all of them).
constexpr int kRouteScanBlocks = 256;

// ---------------------------------------------------------------- product

constexpr uint32_t kRsrcWord3 = 0x00020000u;     // raw buffer resource, gfx9 family
constexpr uint32_t kOob = 0xFFFFFFF0u;           // an offset past every buffer here: reads zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, (int)kRsrcWord3);
}

__device__ __forceinline__ float4_t mfma(const u32x4 a, const u32x4 b, float4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                  0, 0);
}

// A few rows per expert, of any length (tiles of MA = 4 or 16 places): workgroup (x, y) computes 16 outputs of tile y.  It
// serves rows that are no whole 16-byte pieces or too long for the kernel after it.
//
// The eight waves split the row; wave w takes the chunk-steps w, w + 8, ..., where lane (g = lane/16, j = lane%16) reads
// 16-byte chunk 4 s + g of weight row j and decodes it to digits d = t + 1 in place, as exact fp16 values d * 2^-14 (2-bit:
// shifted and masked, d * 2^-16 at even positions of a 16-bit half; 1.6-bit: multiply-shift quotients).  One
// v_mfma_f32_16x16x32_f16 per position p contracts them; sum_k x, from products with ones, is taken off at the end.
//
// A operands.  A product's 8 values per lane are strided over the chunk (2-bit: 16 v + p and 16 v + 8 + p; 1.6-bit:
// 5 q + p and 5 q + 40 + p), so the wave puts the step's activations in LDS, rows as they are, and gathers.  With fewer
// rows than 16, A row MA c + a holds row a in the order of the c-th of 16/MA products: eight 2-byte reads per lane then
// serve 16/MA products, and of product c's result the rows MA c .. MA c + MA-1 are taken.  With 16 rows every lane
// reads its row's pieces whole and pairs the values in registers.
//
// Loads of the next step's activations and of the next kAhead steps' weights are in flight in registers.
template <int FMT, int MA, bool PAIR, bool VEC>
__global__ __launch_bounds__(512) void k_experts_mv(const Experts ex, int C, int slot0)
{
    constexpr int NW = 8;
    constexpr bool TWO = FMT == TRI_FMT_2BIT;
    constexpr int XH = TWO ? 64 : 80;            // values per chunk
    constexpr int NOP = TWO ? 8 : 10;            // products per chunk
    constexpr int CL = 16 / MA;                  // products per gathered A operand
    constexpr int NSET = (NOP + CL - 1) / CL;
    constexpr int NM = PAIR ? 2 : 1;             // matrices
    constexpr int PR = 4 * XH / 8;               // 16-byte pieces of a row per step
    constexpr int NLD = (MA * PR + 63) / 64;
    constexpr int ROW = 4 * XH + 8;              // values of a row's place in LDS (16 bytes more than a step: banks)
    constexpr int kAhead = 2;
    constexpr int NACC = MA == 16 ? 2 : CL;      // accumulators: one per product of an A operand, two at least
    __shared__ __attribute__((aligned(16))) uint16_t xs[NW][MA][ROW];
    __shared__ float red[NW][MA][16 * NM + 1];

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    const ExpertTile et = expert_tile(ex.offsets, ex.E, ex.R, MA, [&](int) { return slot0 + (int)blockIdx.y; });
    if (et.e < 0) return;                        // (the whole workgroup)
    const int K = ex.K, N = ex.N;
    const int64_t S = (int64_t)C * 16;
    const int n0 = (int)blockIdx.x * 16;

    // source rows of the tile, -1 where there is none: lane l holds row l's
    int src = -1;
    if (lane < et.rows) {
        src = ex.rows ? ex.rows[et.r0 + lane] : et.r0 + lane;
        if (src < 0 || src >= ex.T) src = -1;
    }
    const int wrows = min(16, N - n0);
    __amdgpu_buffer_rsrc_t wr[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q)
        wr[q] = rsrc(ex.Wp[q] + ((int64_t)et.e * N + n0) * S, __builtin_amdgcn_readfirstlane((uint32_t)(wrows * S)));
    u32x4 w[kAhead][NM];
    auto load_w = [&](int s, u32x4 (&t)[NM]) __attribute__((always_inline)) {
        const int c = 4 * s + g;
#pragma unroll
        for (int q = 0; q < NM; ++q)
            t[q] = __builtin_amdgcn_raw_buffer_load_b128(wr[q], (int)(c < C ? (uint32_t)(j * S + 16 * c) : kOob), 0, 0);
    };
    const int ns = (C + 3) / 4;                  // steps of the row
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (wv + NW * i < ns) load_w(wv + NW * i, w[i]);

    // activations of a step: piece P = 64 i + lane is piece P % PR of row P / PR
    const uint16_t *xrow[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
        const int P = 64 * i + lane, row = P / PR;
        const int r = row < MA ? __shfl(src, row < MA ? row : 0, 64) : -1;
        xrow[i] = r >= 0 ? ex.X + (int64_t)r * K : nullptr;
    }
    u32x4 xv[NLD];
    auto load_x = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            const int k = 4 * XH * s + 8 * ((64 * i + lane) % PR);
            xv[i] = u32x4{0u, 0u, 0u, 0u};
            if constexpr (VEC) {
                if (xrow[i] && k < K) xv[i] = *reinterpret_cast<const u32x4 *>(xrow[i] + k);
            } else if (xrow[i] && k < K) {       // rows that are no whole pieces
                xv[i] = k + 8 <= K ? ld16_any(xrow[i] + k) : ld16_part(xrow[i] + k, K - k);
            }
        }
    };
    if (wv < ns) load_x(wv);

    const float4_t zero4 = {0.f, 0.f, 0.f, 0.f};
    float4_t acc[NM][NACC], accx = zero4;
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int c = 0; c < NACC; ++c) acc[q][c] = zero4;
    const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};

    // digits of a chunk for product p (and, 1.6-bit, half hh: products 2 p + hh)
    auto contract = [&](const u32x4 (&a)[MA == 16 ? NOP : NSET], const u32x4 v, float4_t (&ac)[NACC]) __attribute__((always_inline)) {
        auto A = [&](int op) -> const u32x4 & { return a[MA == 16 ? op : op / CL]; };
        if constexpr (TWO) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = i ^ 4;             // (positions 4 and 5 need no shift)
                ac[p % NACC] = mfma(A(p), digits_2bit(v, p), ac[p % NACC]);
            }
        } else {
            uint32_t d[8][5];
#pragma unroll
            for (int q = 0; q < 8; ++q) base3_digits_normal(byte_pair(v, q), d[q]);
#pragma unroll
            for (int op = 0; op < 10; ++op) {
                const int p = op / 2, q = 4 * (op % 2), c = op % NACC;
                ac[c] = mfma(A(op), u32x4{d[q][p], d[q + 1][p], d[q + 2][p], d[q + 3][p]}, ac[c]);
            }
        }
    };
    auto step = [&](int s, u32x4 (&wc)[NM]) __attribute__((always_inline)) {
        // this step's activations into LDS, the next step's on the way
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            const int P = 64 * i + lane, row = P / PR;
            if (row < MA) *reinterpret_cast<u32x4 *>(&xs[wv][row][8 * (P % PR)]) = xv[i];
        }
        if (s + NW < ns) load_x(s + NW);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if constexpr (MA == 16) {
            const u32x4 *row = reinterpret_cast<const u32x4 *>(&xs[wv][j][XH * g]);
            uint32_t x32[XH / 2];
#pragma unroll
            for (int q = 0; q < XH / 8; ++q) {
                const u32x4 v = row[q];
                x32[4 * q] = v[0]; x32[4 * q + 1] = v[1]; x32[4 * q + 2] = v[2]; x32[4 * q + 3] = v[3];
            }
            u32x4 a[NOP];
            if constexpr (TWO) {
#pragma unroll
                for (int p = 0; p < 8; ++p)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        a[p][v] = (p & 1) ? pair_halves<1>(x32[8 * v + 4 + p / 2], x32[8 * v + p / 2])
                                          : pair_halves<0>(x32[8 * v + 4 + p / 2], x32[8 * v + p / 2]);
            } else {
#pragma unroll
                for (int op = 0; op < 10; ++op)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = 5 * (4 * (op % 2) + q) + op / 2;   // value; its partner is e + 40
                        a[op][q] = (e & 1) ? pair_halves<1>(x32[(e >> 1) + 20], x32[e >> 1])
                                           : pair_halves<0>(x32[(e >> 1) + 20], x32[e >> 1]);
                    }
            }
#pragma unroll
            for (int p = 0; p < NOP; ++p) accx = mfma(a[p], ones, accx);
#pragma unroll
            for (int q = 0; q < NM; ++q) contract(a, wc[q], acc[q]);
        } else {
            u32x4 a[NSET];
            const int aa = j % MA, c = j / MA;
#pragma unroll
            for (int t = 0; t < NSET; ++t) {
                const int op = min(CL * t + c, NOP - 1);
                const uint16_t *x = &xs[wv][aa][XH * g + (TWO ? op : 5 * 4 * (op & 1) + (op >> 1))];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t lo = x[TWO ? 16 * v : 5 * v], hi = x[TWO ? 16 * v + 8 : 5 * v + 40];
                    a[t][v] = lo | hi << 16;
                }
                if (NOP % CL && t == NSET - 1 && CL * t + c >= NOP) a[t] = u32x4{0u, 0u, 0u, 0u};   // no product left
                accx = mfma(a[t], ones, accx);
            }
#pragma unroll
            for (int q = 0; q < NM; ++q) contract(a, wc[q], acc[q]);
        }
    };
    for (int s = wv; s < ns; s += NW * kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s + NW * i < ns) {
                step(s + NW * i, w[i]);
                if (s + NW * (i + kAhead) < ns) load_w(s + NW * (i + kAhead), w[i]);
            }
        }
    }

    // Merge: product op's rows of result r lie in A rows MA c + a, c = op % CL: lane group (MA c + a) / 4, element
    // (MA c + a) % 4.  Lanes take what is theirs, and the lane groups that hold the same row are added.
    auto unit = [&](int c) { return TWO && c % 2 == 0 ? 4.f : 1.f; };   // (2-bit digits of even positions: 2^-16)
    auto put = [&](int col, float (&v)[4], bool leader) __attribute__((always_inline)) {   // v[e]: this lane's rows
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float t = MA == 16 ? v[e] : sum_over_rows(v[e]);
            if (leader) red[wv][MA == 16 ? 4 * g + e : e][col] = t;
        }
    };
#pragma unroll
    for (int q = 0; q < NM; ++q) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NACC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += MA == 16 || g == c % 4 ? acc[q][c][e] * unit(c) : 0.f;
        put(16 * q + j, v, MA == 16 || g == 0);
    }
    float vx[4] = {accx[0], accx[1], accx[2], accx[3]};   // sum_k x: every product of an A operand counts once
    put(16 * NM, vx, MA == 16 ? j == 0 : lane == 0);
    __syncthreads();
    for (int o = threadIdx.x; o < MA * 16; o += 64 * NW) {
        const int m = o / 16, c = o % 16;
        if (m >= et.rows || n0 + c >= N) continue;
        const int row = ex.rows ? ex.rows[et.r0 + m] : et.r0 + m;
        if (row < 0 || row >= ex.T) continue;
        float sx = 0.f, sd[NM] = {};
#pragma unroll
        for (int q = 0; q < NW; ++q) {
            sx += red[q][m][16 * NM];
#pragma unroll
            for (int p = 0; p < NM; ++p) sd[p] += red[q][m][16 * p + c];
        }
        float y = (sd[0] * 16384.f - sx) * ex.scale[0][et.e];
        if constexpr (PAIR) y = y / (1.f + __expf(-y)) * ((sd[NM - 1] * 16384.f - sx) * ex.scale[1][et.e]);
        ex.Y[(int64_t)(et.r0 + m) * N + n0 + c] = __builtin_bit_cast(uint16_t, (_Float16)y);
    }
}

// The same product with the activations kept: rows short enough that a wave's A operands of all its CST steps stay in
// registers (gathered once, as above; tiles of MA = 1, 8 or 16 places).  The workgroup then runs through blocks of 16
// outputs, blockIdx.x, + gridDim.x, ...: only weights are read, the next block's chunks in flight while one is
// contracted; the waves' partial sums meet in one of two LDS buffers in turn, so a block costs one barrier.
//
// Measured on eight experts, two per token: gate and up 4096 -> 11008 of one token (45 MB of 2-bit weights) 13.6 us, where
// a plain read takes 7.6; of 16 tokens (180 MB) 44 us against 28; down 11008 -> 4096 of 16 tokens, 1.6-bit (72 MB) 37 us
// against 12.  What bounds it is the vector ALU (19 of 44 us at 16 tokens, 22 of 37 with 1.6-bit digits; the matrix cores
// another 10 and 7, hardly overlapped) and the waits around a block's barrier; splitting the waves by outputs instead, with
// all of the row per wave and no barrier, was slower (59 us), as were deeper loads (48 us).  Digits as subnormals d * 2^-24
// would save the 1.6-bit products 4 - 8% (down 34 us) and the 2-bit ones nothing, at the price of ten bits of every sum.
constexpr int kHeld = 16;                        // blocks whose results wait in LDS
// Whether the loop's registers for A operands and for D blocks' chunks leave the rest of its code enough of 128 registers
// (two workgroups per CU) that the compiler spills nothing, or next to nothing; limits as found by compiling.
constexpr bool loop_fits(int fmt, int ma, int cst, bool pair, int d)
{
    // (84 KB of LDS: one workgroup per CU, which may have 256 registers; held to 128 the short rows, where both fit, take
    // as long: pair of 64 tokens, 2048 -> 5632 31.9 us either way)
    if (ma == 16 && fmt == TRI_FMT_1P6BIT) return false;
    const int nop = fmt == TRI_FMT_2BIT ? 8 : 10, cl = ma == 1 ? nop : 16 / ma, na = (nop + cl - 1) / cl;
    return 4 * cst * (na + (pair ? 2 : 1) * d) <= (fmt == TRI_FMT_2BIT ? 80 : ma == 1 ? 40 : 64);
}
// Waves per SIMD to compile for, and blocks in registers: three workgroups per CU with one block each where the registers
// are very few (a pair of two tokens 19.6 us against 20.3 with two of two blocks, of one token 13.2 either way); else two
// per CU where they fit, with the next block's chunks in flight (D = 2) or, failing that, one workgroup's loads under the
// other's products (D = 1); else one.
constexpr bool loop_light(int fmt, int ma, int cst, bool pair) { return ma == 1 && fmt == TRI_FMT_2BIT && pair && cst <= 2; }
constexpr int loop_waves(int fmt, int ma, int cst, bool pair)
{
    return loop_light(fmt, ma, cst, pair) ? 6 : loop_fits(fmt, ma, cst, pair, 1) ? 4 : 2;
}
constexpr int loop_depth(int fmt, int ma, int cst, bool pair)
{
    if (loop_light(fmt, ma, cst, pair)) return 1;
    return loop_fits(fmt, ma, cst, pair, 2) || !loop_fits(fmt, ma, cst, pair, 1) ? 2 : 1;
}

template <int FMT, int MA, int CST, bool PAIR, int D, int EU>
__global__ __launch_bounds__(512, EU) void k_experts_loop(const Experts ex, int C)
{
    constexpr int NW = 8;
    constexpr bool TWO = FMT == TRI_FMT_2BIT;
    constexpr int XH = TWO ? 64 : 80;            // values per chunk
    constexpr int NOP = TWO ? 8 : 10;            // products per chunk
    constexpr int CL = MA == 1 ? NOP : 16 / MA;  // products per gathered A operand
    constexpr int NA = MA == 16 ? NOP : (NOP + CL - 1) / CL;   // A operands per step
    constexpr int NM = PAIR ? 2 : 1;             // matrices
    constexpr int PR = 4 * XH / 8;               // 16-byte pieces of a row per step
    constexpr int NLD = (MA * PR + 63) / 64;
    constexpr int ROW = 4 * XH + 8;              // values of a row's place in LDS (16 bytes more than a step: banks)
    constexpr int NACC = MA == 16 ? 2 : CL;      // accumulators: one per product of an A operand, two at least
    // (the activations' passage and, after it, the partial sums use the same LDS)
    constexpr int XS = NW * MA * ROW * 2, RED = 2 * NW * MA * (16 * NM + 1) * 4;
    __shared__ u32x4 smem[((XS > RED ? XS : RED) + 15) / 16];
    auto xs = reinterpret_cast<uint16_t (*)[MA][ROW]>(smem);
    auto red = reinterpret_cast<float (*)[NW][MA][16 * NM + 1]>(smem);
    __shared__ float sxw[NW][MA], sxt[MA];
    __shared__ uint16_t done[kHeld][MA][16];     // results not yet written
    __shared__ int source[MA];

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    const int K = ex.K, N = ex.N;
    const int64_t S = (int64_t)C * 16;
    const int nblk = (N + 15) / 16;
    // The tiles share the workgroups evenly (there are at least as many): tile t has workgroups t G .. t G + G - 1, of
    // which the q-th takes blocks q, q + G, ...
    int G = 1;
    const ExpertTile et = expert_tile(ex.offsets, ex.E, ex.R, MA, [&](int tiles) {
        G = max(min((int)gridDim.x / max(tiles, 1), nblk), 1);   // (offsets that decrease list more tiles than there may be)
        return (int)blockIdx.x / G;
    });
    if (et.e < 0) return;                        // (the whole workgroup)
    int src = -1;                                // source rows of the tile: lane l holds row l's
    if (lane < et.rows) {
        src = ex.rows ? ex.rows[et.r0 + lane] : et.r0 + lane;
        if (src < 0 || src >= ex.T) src = -1;
    }
    if (wv == 0 && lane < MA) source[lane] = src;

    const uint8_t *W[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q) W[q] = ex.Wp[q] + (int64_t)et.e * N * S;
    auto load_w = [&](int b, u32x4 (&t)[NM][CST]) __attribute__((always_inline)) {
        const int rows = min(16, N - 16 * b);
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            const __amdgpu_buffer_rsrc_t wr =
                rsrc(W[q] + 16 * (int64_t)b * S, __builtin_amdgcn_readfirstlane((uint32_t)(rows * S)));
#pragma unroll
            for (int i = 0; i < CST; ++i) {
                const int c = 4 * (wv + NW * i) + g;
                t[q][i] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)(c < C ? (uint32_t)(j * S + 16 * c) : kOob), 0, 0);
            }
        }
    };
    u32x4 w[D][NM][CST];
    int b = (int)blockIdx.x % G;
#pragma unroll
    for (int i = 0; i < (D > 1 ? D - 1 : 1); ++i)
        if (b + i * G < nblk) load_w(b + i * G, w[i]);

    // activations: piece P = 64 i + lane of a step is piece P % PR of row P / PR
    const float4_t zero4 = {0.f, 0.f, 0.f, 0.f};
    const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    u32x4 a[CST][NA];
    {
        const uint16_t *xrow[NLD];
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            const int row = (64 * i + lane) / PR;
            const int r = row < MA ? __shfl(src, row < MA ? row : 0, 64) : -1;
            xrow[i] = r >= 0 ? ex.X + (int64_t)r * K : nullptr;
        }
        u32x4 xv[CST][NLD];
#pragma unroll
        for (int t = 0; t < CST; ++t)
#pragma unroll
            for (int i = 0; i < NLD; ++i) {
                const int k = 4 * XH * (wv + NW * t) + 8 * ((64 * i + lane) % PR);
                xv[t][i] = u32x4{0u, 0u, 0u, 0u};
                if (xrow[i] && k < K) xv[t][i] = *reinterpret_cast<const u32x4 *>(xrow[i] + k);
            }
        float4_t accx = zero4;
#pragma unroll
        for (int t = 0; t < CST; ++t) {
#pragma unroll
            for (int i = 0; i < NLD; ++i) {
                const int P = 64 * i + lane, row = P / PR;
                if (row < MA) *reinterpret_cast<u32x4 *>(&xs[wv][row][8 * (P % PR)]) = xv[t][i];
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if constexpr (MA == 16) {
                const u32x4 *row = reinterpret_cast<const u32x4 *>(&xs[wv][j][XH * g]);
                uint32_t x32[XH / 2];
#pragma unroll
                for (int q = 0; q < XH / 8; ++q) {
                    const u32x4 v = row[q];
                    x32[4 * q] = v[0]; x32[4 * q + 1] = v[1]; x32[4 * q + 2] = v[2]; x32[4 * q + 3] = v[3];
                }
#pragma unroll
                for (int op = 0; op < NOP; ++op)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // 2-bit: values 16 q + op and its partner 8 on; 1.6-bit: 5 (4 (op % 2) + q) + op / 2 and 40 on
                        const int e = TWO ? 16 * q + op : 5 * (4 * (op % 2) + q) + op / 2, f = e + (TWO ? 8 : 40);
                        a[t][op][q] = (e & 1) ? pair_halves<1>(x32[f >> 1], x32[e >> 1]) : pair_halves<0>(x32[f >> 1], x32[e >> 1]);
                    }
            } else {
                const int aa = j % MA, c = MA == 1 ? min(j, CL - 1) : j / MA;
#pragma unroll
                for (int q = 0; q < NA; ++q) {
                    const int op = CL * q + c;
                    const uint16_t *x = &xs[wv][aa][XH * g + (TWO ? op : 20 * (op & 1) + (op >> 1))];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint32_t lo = x[TWO ? 16 * v : 5 * v], hi = x[TWO ? 16 * v + 8 : 5 * v + 40];
                        a[t][q][v] = lo | hi << 16;
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int q = 0; q < NA; ++q) accx = mfma(a[t][q], ones, accx);
        }
        // sum_k x of every row: each product of an A operand counts once
        if constexpr (MA == 16) {
            if (j == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sxw[wv][4 * g + e] = accx[e];
            }
        } else if constexpr (MA == 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = accx[e], q = accx[e];
                swap32(p, q);
                if (j == 0 && g < 2) sxw[wv][4 * g + e] = p + q;
            }
        } else {
            float v = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) v += 4 * g + c < CL ? accx[c] : 0.f;
            v = sum_over_rows(v);
            if (lane == 0) sxw[wv][0] = v;
        }
    }
    __syncthreads();
    if (threadIdx.x < MA) {
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < NW; ++q) t += sxw[q][threadIdx.x];
        sxt[threadIdx.x] = t;                    // (read after the first block's barrier)
    }
    float scale[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q) scale[q] = ex.scale[q][et.e];

    auto contract = [&](const u32x4 (&x)[NA], const u32x4 v, float4_t (&ac)[NACC]) __attribute__((always_inline)) {
        auto A = [&](int op) -> const u32x4 & { return x[MA == 16 ? op : op / CL]; };
        if constexpr (TWO) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = i ^ 4;             // (positions 4 and 5 need no shift)
                ac[p % NACC] = mfma(A(p), digits_2bit(v, p), ac[p % NACC]);
            }
        } else {
            uint32_t d[8][5];
#pragma unroll
            for (int q = 0; q < 8; ++q) base3_digits_normal(byte_pair(v, q), d[q]);
#pragma unroll
            for (int op = 0; op < 10; ++op) {
                const int p = op / 2, q = 4 * (op % 2), c = op % NACC;
                ac[c] = mfma(A(op), u32x4{d[q][p], d[q + 1][p], d[q + 2][p], d[q + 3][p]}, ac[c]);
            }
        }
    };
    auto unit = [&](int c) { return TWO && c % 2 == 0 ? 4.f : 1.f; };   // (2-bit digits of even positions: 2^-16)
    auto run = [&](const u32x4 (&wc)[NM][CST], int buf, int held) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            float4_t acc[NACC];
#pragma unroll
            for (int c = 0; c < NACC; ++c) acc[c] = zero4;
#pragma unroll
            for (int i = 0; i < CST; ++i) contract(a[i], wc[q][i], acc);
            // product op's rows of the result lie in A rows MA c + a, c = op % CL: lane group (MA c + a) / 4
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NACC; ++c) {
                if constexpr (MA == 1) {
                    v[0] += g == c / 4 ? acc[c][c % 4] * unit(c) : 0.f;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = acc[c][e] * unit(c);
                        v[e] += MA == 16 || (g >> 1) == c % 2 ? t : 0.f;
                    }
                }
            }
            const int col = 16 * q + j;
            if constexpr (MA == 16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) red[buf][wv][4 * g + e][col] = v[e];
            } else if constexpr (MA == 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = v[e], y = v[e];
                    swap32(x, y);
                    if (g < 2) red[buf][wv][4 * g + e][col] = x + y;
                }
            } else {
                const float t = sum_over_rows(v[0]);
                if (g == 0) red[buf][wv][0][col] = t;
            }
        }
        __syncthreads();
        for (int o = threadIdx.x; o < 16 * MA; o += 64 * NW) {
            const int m = o / 16, c = o % 16;
            float sd[NM] = {};
#pragma unroll
            for (int q = 0; q < NW; ++q)
#pragma unroll
                for (int p = 0; p < NM; ++p) sd[p] += red[buf][q][m][16 * p + c];
            float y = (sd[0] * 16384.f - sxt[m]) * scale[0];
            if constexpr (PAIR) y = y / (1.f + __expf(-y)) * ((sd[NM - 1] * 16384.f - sxt[m]) * scale[NM - 1]);
            done[held][m][c] = __builtin_bit_cast(uint16_t, (_Float16)y);
        }
    };
    // Results wait in LDS and are written kHeld blocks at a time: a store between the loads would be waited for with
    // them, by every wave at the next barrier.
    int first = b, held = 0;                     // results of blocks first, + G, ... (held of them) wait
    auto flush = [&]() __attribute__((always_inline)) {
        __syncthreads();
        for (int o = (int)threadIdx.x; o < held * MA * 16; o += 64 * NW) {
            const int i = o / (MA * 16), m = o / 16 % MA, n = 16 * (first + i * G) + o % 16;
            if (n < N && source[m] >= 0) ex.Y[(int64_t)(et.r0 + m) * N + n] = done[i][m][o % 16];
        }
        __syncthreads();
        first += held * G;
        held = 0;
    };
    int buf = 0;
    for (; b < nblk; b += D * G) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (b + i * G < nblk) {
                if (D > 1 && b + (i + D - 1) * G < nblk) load_w(b + (i + D - 1) * G, w[(i + D - 1) % D]);
                run(w[i], buf, held++);
                if (D == 1 && b + G < nblk) load_w(b + G, w[0]);
                buf ^= 1;
            }
        }
        if (held > kHeld - D) flush();
    }
    flush();
}

// ---------------------------------------------------------------- combination

// Bound by memory: 2048 tokens of six results of 4096 values take 28.9 us, 134 MB at 4.65 TB/s (a large copy: 4.92).
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
    auto go_ep = [&](auto h) {
        constexpr bool H = decltype(h)::value;
        if (E <= 16) go(k_route<H, 1>);
        else if (E <= 32) go(k_route<H, 2>);
        else if (E <= 64) go(k_route<H, 4>);
        else if (E <= 128) go(k_route<H, 8>);
        else go(k_route<H, 16>);
    };
    if (half) go_ep(std::true_type{});
    else go_ep(std::false_type{});
    if (!single) {
        const bool scan = blocks > kRouteScanBlocks;
        if (scan) hipLaunchKernelGGL(k_route_scan, dim3(E + 1), dim3(kRouteThreads), 0, s, blocks, E + 1, hist);
        hipLaunchKernelGGL(k_route_place, dim3(blocks), dim3(kRouteThreads), 0, s, T, E, topk, scan ? 1 : 0, ids, hist,
                           offsets, rows, pos);
    }
    return launched();
}

namespace {

template <int FMT, int MA, bool PAIR, bool VEC>
void experts_go(const Experts &ex, hipStream_t s)
{
    const int C = (int)(row_bytes(ex.K, FMT) / 16);
    const int64_t slots = expert_slots(ex.R, ex.E, MA);
    for (int64_t s0 = 0; s0 < slots; s0 += 65535) {   // (the second grid dimension's limit)
        const dim3 grid((ex.N + 15) / 16, (unsigned)(slots - s0 < 65535 ? slots - s0 : 65535));
        hipLaunchKernelGGL((k_experts_mv<FMT, MA, PAIR, VEC>), grid, dim3(512), 0, s, ex, C, (int)s0);
    }
}

template <int FMT, int MA, int CST, bool PAIR>
bool loop_go(const Experts &ex, hipStream_t s)
{
    constexpr int D = loop_depth(FMT, MA, CST, PAIR), EU = loop_waves(FMT, MA, CST, PAIR);
    constexpr auto kernel = k_experts_loop<FMT, MA, CST, PAIR, D, EU>;
    const int C = (int)(row_bytes(ex.K, FMT) / 16);
    const int64_t slots = expert_slots(ex.R, ex.E, MA), most = slots * ((ex.N + 15) / 16);
    const int64_t resident = (int64_t)cu_count() * resident_per_cu<kernel>(512), least = resident > slots ? resident : slots;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(most < least ? most : least)), dim3(512), 0, s, ex, C);
    return true;
}

// The fewest steps per wave that cover the row; false where the A operands would not stay in registers.
template <int FMT, int MA, bool PAIR>
bool loop_cst(const Experts &ex, hipStream_t s)
{
    constexpr int kLong = FMT == TRI_FMT_2BIT ? 6 : 5;
    const int cst = (int)((row_bytes(ex.K, FMT) / 16 + 31) / 32);
    if (cst <= 1) return loop_go<FMT, MA, 1, PAIR>(ex, s);
    if (cst <= 2) return loop_go<FMT, MA, 2, PAIR>(ex, s);
    if constexpr (MA <= 8) {
        if (cst <= 4) return loop_go<FMT, MA, 4, PAIR>(ex, s);
        if (cst <= kLong) return loop_go<FMT, MA, kLong, PAIR>(ex, s);
    }
    return false;
}

// The tile height by the mean number of places per expert, R / E; false: the tiled GEMM.  Measured on eight experts, two
// per token (us; MA = 1 / 8 / 16 / GEMM, 2-bit):
//   gate and up, 4096 -> 11008   R/E = 1/4: 12.3 / 16.5 / 16.6 / 29.7,  1: 38.0 / 32.9 / 34.2 / 63.7,
//                                4: - / 45.5 / 43.4 / 69.8,  16: - / 96.4 / 60.1 / 74.3,  32: - / 156 / 87 / 118
//   down, 11008 -> 4096          R/E = 1: 19.4 / 23.0 / - / 45.3,  4: - / 29.5 / - / 53.8,  16: - / 58.7 / - / 66.3,
//                                24: - / 77.0 / - / 67.5
// (MA = 4 won nowhere by more than 3%.  Taken with digits as subnormals: the loop's times are now 4% less to 4% more.)
template <int FMT, bool PAIR>
bool loop_ma(const Experts &ex, hipStream_t s)
{
    const int one = FMT == TRI_FMT_2BIT && !PAIR ? ex.E : ex.E / 2;
    if (ex.R <= one) return loop_cst<FMT, 1, PAIR>(ex, s);
    if (ex.R / 2 > ex.E && ex.R / (FMT == TRI_FMT_2BIT ? 32 : 16) <= ex.E && loop_cst<FMT, 16, PAIR>(ex, s)) return true;
    if (ex.R / 16 <= ex.E) return loop_cst<FMT, 8, PAIR>(ex, s);
    return false;
}

template <int FMT, bool PAIR, bool VEC>
int experts_ma(const Experts &ex, hipStream_t s)
{
    if constexpr (VEC) {
        if (loop_ma<FMT, PAIR>(ex, s)) return launched();
        if (ex.R / 2 > ex.E && experts_gemm_fits(ex, FMT)) return launch_experts_gemm(ex, FMT, s);
    }
    // rows too long for the loop, or no whole 16-byte pieces
    if (ex.R <= ex.E) experts_go<FMT, 4, PAIR, VEC>(ex, s);
    else experts_go<FMT, 16, PAIR, VEC>(ex, s);
    return launched();
}

template <int FMT>
int experts_fmt(const Experts &ex, hipStream_t s)
{
    const bool vec = ex.K % 8 == 0;
    if (ex.Wp[1]) return vec ? experts_ma<FMT, true, true>(ex, s) : experts_ma<FMT, true, false>(ex, s);
    return vec ? experts_ma<FMT, false, true>(ex, s) : experts_ma<FMT, false, false>(ex, s);
}

}  // namespace

int launch_experts(const Experts &ex, int fmt, hipStream_t s)
{
    return fmt == TRI_FMT_2BIT ? experts_fmt<TRI_FMT_2BIT>(ex, s) : experts_fmt<TRI_FMT_1P6BIT>(ex, s);
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
