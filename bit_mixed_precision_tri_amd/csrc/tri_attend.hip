// tri_attend.hip -- causal attention of new tokens over the 8-bit cache (tri_cache_attend).
//
// With q a row, k_j and v_j codes, s_j and u_j the scales of the keys' and values' pages, everything in base 2:
//     x_j = scale log2(e) s_j (q . k_j),   y_j = x_j + log2 u_j,   m = max y_j,   w_j = 2^(y_j - m + 10),
//     o = sum_j w_j v_j / sum_j (w_j / u_j).
// The values' scales sit in the exponents, so that w_j (rounded to fp16: normal numbers down to 2^-24 of the largest) is the
// operand of the second product and the codes, exact in fp16, are the other; however small a scale is, nothing underflows.
// m, the two sums and o run on over the tokens (when m grows, the others shrink by 2^(m - m')).  What the rounding of a weight to
// fp16 leaves off is an operand of its own, with the same codes: weights are exact to 2^-22, and results carry little more than their
// own rounding to fp16 (an error of 2.1e-4 of their size, as with weights of fp32).
//
// Both products are taken transposed: S^T = K Q^T (a row of A is a token, a column of B a query row), O^T = V^T W^T.  A lane of
// S^T then holds weights of one query row, and they are its part of the second product's B operand as they lie: the
// weights never leave their lanes.  Which token a row of A is can be chosen freely; rows are taken so that a lane's 16
// weights are of 16 consecutive tokens, all in one page.
//
// Few rows are bound by reading the cache.  Each wave reads whole steps of 64 tokens by itself, straight from the pages into
// its operands (no LDS, no barrier), the next step's codes while it works on this one's: 64 sequences of about 8192 tokens, 8
// heads of 128 (810 MB), take 140 us, 5.8 TB/s (a plain read of as many bytes 122); 16 over windows of 4096, 32 heads (538 MB),
// 98 - 101 us (82).  Vector instructions take a quarter of a wave's cycles there, waiting for loads and results 30%.  One
// sequence alone is bound by latency: 333 tokens 6.7 us; 32768 tokens of 8 heads (67 MB, a read of which takes 11) 15 and the
// join of their splits 4.
#include "tri_attend.h"
#include <algorithm>

namespace tri {

namespace {

// v_mfma_f32_16x16x32_f16 (see mfma16).
__device__ __forceinline__ float4_t mfma(half8_t a, u32x4 b, float4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// Few rows: 16 CT query rows of one key/value head, a split's steps dealt out to the NW waves.  splits > 1: unnormalised
// sums, their maximum and denominator go to the workspace (part: row, split, D + 4), to be joined by k_join.
template <int D, int FMT, int CT, int NW>
__device__ __forceinline__ void attend_few(const Attend &at, float *__restrict__ part, int splits, int chunk, int split, int h,
                                           int r0, int b)
{
    constexpr int KL = D / 16, DT = D / 16, CS = D + 4;  // 16-byte loads of keys of a step and lane; tiles of 16 values; LDS stride
    __shared__ alignas(16) float so[NW][16][CS];
    __shared__ float sm[NW][16 * CT], sl[NW][16 * CT];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, j = lane & 15;
    const tri_cache &c = at.c;
    const int P = c.page, lp = 31 - __builtin_clz(P), i0 = split * chunk;
    const int64_t head_bytes = (int64_t)P * D;

    // Pages of the step of token t0: of this lane's rows of A in the first product (tokens 16 (j / 4) ..), and of its tokens in
    // the second (16 g ..); as the table holds them, looked up a step before they are used.
    const int32_t *table = at.sq.table + (int64_t)b * at.sq.width;
    const int64_t last_page = at.sq.width - 1;
    auto look = [&](int64_t t0, int &pk, int &pv) {
        pk = table[min((t0 + 16 * (j >> 2)) >> lp, last_page)];
        pv = table[min((t0 + 16 * g) >> lp, last_page)];
    };
    int i = i0 + wv, pk, pv, nk, nv;
    if (at.window == 0) {                        // (steps are in order from 0 on: no need to know the sequence's length first)
        look((int64_t)i * kStep, pk, pv);
        look((int64_t)(i + NW) * kStep, nk, nv);
    }

    const Tile t = tile_of(at, b, r0, 16 * CT);
    if (t.rows == 0) return;
    const int steps = t.st.count(), i1 = split == splits - 1 ? steps : min(steps, i0 + chunk);
    if (split > 0 && i0 >= steps) return;        // (split 0 writes the zeros of rows that see nothing)
    if (at.window > 0) {
        look((int64_t)t.st.at(i) * kStep, pk, pv);
        look((int64_t)t.st.at(i + NW) * kStep, nk, nv);
    }

    // Keys.  A load is of whole 128-byte lines: for dim 64 rows of A are tokens (16 (j / 4) + 4 n + j % 4 of the step in load n:
    // four in a row); for more, rows 2 x and 2 x + 1 are the halves of a line of token 16 (x / 2) + 2 n + x % 2, each multiplied by
    // both halves of the queries, and the scores are the sums of what belongs together (the matrix cores have time for
    // twice the products here; half lines read 5.4 TB/s instead of 6.2).
    constexpr bool kHalves = D >= 128;
    constexpr int LINES = kHalves ? D / 128 : 1;
    auto q_at = [&](int n) {                     // operand n: of line n / 4, half n / 2 % 2, eight values each
        return kHalves ? 128 * (n / 4) + 64 * (n / 2 % 2) + 16 * g + 8 * (n % 2) : 16 * g + 8 * n;
    };
    const int krow = kHalves ? 16 * (j >> 2) + (j >> 1 & 1) : 16 * (j >> 2) + (j & 3), kbyte = kHalves ? 16 * (g + 4 * (j & 1)) : 16 * g;
    const uint32_t flip = at.scale < 0.f ? 0x80008000u : 0u;     // (the scale's sign goes into the queries)
    const float ck = fabsf(at.scale) * 1.44269504088896f * kCodeUnit<FMT>;
    u32x4 q[CT][D / 32];
    int pos[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int r = r0 + 16 * ct + j, n = r / at.G;
        const bool live = 16 * ct + j < t.rows;
        pos[ct] = live ? t.sp.p0 + n : -1;
        const uint16_t *x = at.Q + (int64_t)(t.sp.r0 + (live ? n : 0)) * at.q_stride + (h * at.G + (live ? r % at.G : 0)) * D;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) q[ct][s] = *reinterpret_cast<const u32x4 *>(x + q_at(s)) ^ flip;
    }

    float m[CT], l[CT];
    float4_t o[CT][DT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        m[ct] = kNone;
        l[ct] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[ct][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    auto streamed = [](const uint8_t *x) { return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x)); };
    u32x4 kr[KL], vr[DT];
    float sk, sv;
    bool here;                                   // whether this lane's tokens (16 g .. of the step) have a page
    auto load_keys = [&](int64_t t0) {           // (a page that is not there: any one's codes)
        const uint8_t *x = c.K + ((int64_t)((uint32_t)pk < (uint32_t)c.pages ? pk : 0) * c.heads + h) * head_bytes + kbyte;
#pragma unroll
        for (int n = 0; n < KL; ++n) {
            const int row = (int)(t0 + krow + (kHalves ? 2 * (n / LINES) : 4 * n)) & (P - 1);
            kr[n] = streamed(x + row * D + (kHalves ? 128 * (n % LINES) : 0));
        }
        const bool ok = (uint32_t)pv < (uint32_t)c.pages;
        const int64_t s = (int64_t)(ok ? pv : 0) * c.heads + h;
        sk = c.K_scale[s];
        sv = c.V_scale[s];
        here = ok && (t0 + 16 * g) >> lp <= last_page;
    };
    // Values: rows of a page's tokens, so of whole lines but for pages of 128 tokens, whose lines another wave reads the rest of.
    auto load_values = [&](int64_t t0) {
        const uint8_t *x = c.V + ((int64_t)((uint32_t)pv < (uint32_t)c.pages ? pv : 0) * c.heads + h) * head_bytes + ((int)(t0 + 16 * g) & (P - 1));
        if (P <= 64) {
#pragma unroll
            for (int d = 0; d < DT; ++d) vr[d] = streamed(x + (16 * d + j) * P);
        } else {
#pragma unroll
            for (int d = 0; d < DT; ++d) vr[d] = *reinterpret_cast<const u32x4 *>(x + (16 * d + j) * P);
        }
    };

    if (i < i1) {
        const int64_t t0 = (int64_t)t.st.at(i) * kStep;
        load_keys(t0);
        load_values(t0);
    }
    for (; i < i1; i += NW) {
        const int t0 = t.st.at(i) * kStep;
        const bool more = i + NW < i1;
        const int64_t t1 = (int64_t)t.st.at(i + NW) * kStep;
        float s[CT][16];                         // the lane's tokens' scores
        if constexpr (kHalves) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                float4_t x[CT][2];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int half = 0; half < 2; ++half) x[ct][half] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 2 * LINES; ++k) {
                    const u32x4 w = kr[n * LINES + k / 2];
                    const half8_t a = decode8<FMT>(w[2 * (k % 2)], w[2 * (k % 2) + 1]);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int half = 0; half < 2; ++half) x[ct][half] = mfma(a, q[ct][4 * (k / 2) + 2 * half + k % 2], x[ct][half]);
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    s[ct][2 * n] = x[ct][0][0] + x[ct][1][1];
                    s[ct][2 * n + 1] = x[ct][0][2] + x[ct][1][3];
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const half8_t lo = decode8<FMT>(kr[n][0], kr[n][1]), hi = decode8<FMT>(kr[n][2], kr[n][3]);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const float4_t x = mfma(hi, q[ct][1], mfma(lo, q[ct][0], float4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[ct][4 * n + e] = x[e];
                }
            }
        }
        const float u = usable(sv), a = usable(ck * sk), lu = log2_(u), iu = 1.f / u;
        const bool there = here;
        // every row sees all of the step, unless it reaches past the first row's position, before the last one's window
        // (and behind the first tokens), or onto a page that is not there
        const bool whole = t0 + kStep - 1 <= t.pa && (at.window == 0 || t.pb - t0 < at.window || t0 + kStep <= at.sinks) && __all(there);
        pk = nk;
        pv = nv;
        if (more) {
            load_keys(t1);
            look((int64_t)t.st.at(i + 2 * NW) * kStep, nk, nv);
        }
        u32x4 w[CT][2], wl[CT][2];               // weights, and what their rounding to fp16 left off
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            if (!whole) {
                const uint32_t seen = there ? (uint32_t)seen_of(pos[ct], t0 + 16 * g, at.window, at.sinks) : 0u;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if ((seen >> e & 1u) == 0u) s[ct][e] = -INFINITY;
            }
            float top = s[ct][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, s[ct][e]);
            const float mx = max_over_rows(fmaxf(kNone, fmaf(top, a, lu)));    // (a > 0)
            if (__any(mx - m[ct] > kSlack)) {
                const float mn = fmaxf(m[ct], mx), f = exp2_(m[ct] - mn);
                m[ct] = mn;
                l[ct] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[ct][d] *= f;
            }
            float shift = lu + (kLift - m[ct]), f = a, sum = 0.f;
            if (is_far(m[ct])) {                 // (by row: no row goes by what others hold)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[ct][e] = fmaf(s[ct][e], a, lu) - m[ct];
                shift = kLift;
                f = 1.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y0 = exp2_(fmaf(s[ct][2 * e], f, shift)), y1 = exp2_(fmaf(s[ct][2 * e + 1], f, shift));
                sum += y0 + y1;
                const uint32_t x = pack2(y0, y1);
                w[ct][e / 4][e % 4] = x;
                wl[ct][e / 4][e % 4] = pack2(y0 - h2f((uint16_t)x), y1 - h2f((uint16_t)(x >> 16)));
            }
            l[ct] = fmaf(sum, iu, l[ct]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const half8_t lo = decode8<FMT>(vr[d][0], vr[d][1]), hi = decode8<FMT>(vr[d][2], vr[d][3]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                o[ct][d] = mfma(hi, w[ct][1], mfma(lo, w[ct][0], mfma(hi, wl[ct][1], mfma(lo, wl[ct][0], o[ct][d]))));
        }
        if (more) load_values(t1);
    }

    // the waves' sums, in the waves' order
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        l[ct] = sum_over_rows(l[ct]);
        if (g == 0) {
            sm[wv][16 * ct + j] = m[ct];
            sl[wv][16 * ct + j] = l[ct];
        }
    }
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        float top = kNone;
#pragma unroll
        for (int k = 0; k < NW; ++k) top = fmaxf(top, sm[k][16 * ct + j]);
        const float f = exp2_(m[ct] - top);
        if (ct > 0) __syncthreads();             // (the last tile's sums have been read)
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<float4_t *>(&so[wv][j][16 * d + 4 * g]) = o[ct][d] * f;
        __syncthreads();
        for (int e = threadIdx.x; e < 16 * (D / 4); e += 64 * NW) {
            const int col = e / (D / 4), d = 4 * (e % (D / 4)), r = r0 + 16 * ct + col;
            if (16 * ct + col >= t.rows) continue;
            float tp = kNone, den = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) tp = fmaxf(tp, sm[k][16 * ct + col]);
            float4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                v += *reinterpret_cast<const float4_t *>(&so[k][col][d]);
                den = fmaf(sl[k][16 * ct + col], exp2_(sm[k][16 * ct + col] - tp), den);
            }
            const int64_t row = (int64_t)(t.sp.r0 + r / at.G);
            const int head = h * at.G + r % at.G;
            if (splits == 1) {
                store_row<FMT>(at.O + row * at.o_stride + head * D + d, v, den);
            } else {
                float *y = part + ((row * at.H + head) * splits + split) * (D + 4);
                *reinterpret_cast<float4_t *>(y + d) = v;
                if (d == 0) {
                    y[D] = tp;
                    y[D + 1] = den;
                }
            }
        }
    }
}

// Workgroups: split (fastest), key/value head, row tile, sequence.
template <int D, int FMT, int CT, int NW>
__global__ __launch_bounds__(64 * NW) void k_attend_few(const Attend at, float *__restrict__ part, const AttendPlan p, const Grid gd)
{
    const uint32_t k = blockIdx.x / p.splits, n = k / at.c.heads;
    attend_few<D, FMT, CT, NW>(at, part, p.splits, p.chunk, (int)(blockIdx.x % p.splits), (int)(k % at.c.heads),
                               (gd.tile0 + (int)(n % gd.tiles)) * 16 * CT, gd.seq0 + (int)(n / gd.tiles));
}

// A row's splits joined: a workgroup per row, D/4 threads for each of several splits at a time, joined in LDS in order.
template <int D, int FMT>
__global__ __launch_bounds__(256) void k_join(const Attend at, const float *__restrict__ part, int splits, int chunk, int height)
{
    constexpr int GR = 256 / (D / 4);
    __shared__ float4_t so[GR][D / 4];
    __shared__ float sm[GR], sl[GR];
    const int64_t rows = (int64_t)at.T * at.H;
    const int grp = threadIdx.x / (D / 4), d = threadIdx.x % (D / 4);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float *x = part + row * splits * (D + 4);
        // the first splits' sums are on their way before it is known how many there are
        constexpr int AHEAD = 4;
        float4_t w[AHEAD];
        float2 md[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const float *y = x + (int64_t)min(grp + q * GR, splits - 1) * (D + 4);
            w[q] = *reinterpret_cast<const float4_t *>(y + 4 * d);
            md[q] = *reinterpret_cast<const float2 *>(y + D);
        }
        const int tok = (int)(row / at.H), head = (int)(row % at.H), b = owner(at.sq, tok);
        const Span sp = span_of(at.sq, at.T, b);
        const int i = tok - sp.r0;
        if (i < 0 || i >= sp.n) continue;        // (the same for the whole workgroup)
        const int r = i * at.G + head % at.G;
        const Tile t = tile_of(at, b, r - r % height, height);
        const int n = min(splits, max(1, (t.st.count() + chunk - 1) / chunk));
        float m = kNone, den = 0.f;
        float4_t v = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](const float4_t &w, const float2 &md) {
            const float mn = fmaxf(m, md.x), f = exp2_(m - mn), e = exp2_(md.x - mn);
            m = mn;
            den = den * f + md.y * e;
            v = v * f + w * e;
        };
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (grp + q * GR < n) add(w[q], md[q]);
        for (int k = grp + AHEAD * GR; k < n; k += GR) {
            const float *y = x + (int64_t)k * (D + 4);
            add(*reinterpret_cast<const float4_t *>(y + 4 * d), *reinterpret_cast<const float2 *>(y + D));
        }
        __syncthreads();                         // (the last row's sums have been read)
        so[grp][d] = v;
        if (d == 0) sm[grp] = m, sl[grp] = den;
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int k = 1; k < GR; ++k) {
                const float mn = fmaxf(m, sm[k]), f = exp2_(m - mn), e = exp2_(sm[k] - mn);
                m = mn;
                den = den * f + sl[k] * e;
                v = v * f + so[k][d] * e;
            }
            store_row<FMT>(at.O + (int64_t)tok * at.o_stride + head * D + 4 * d, v, den);
        }
    }
}

// Waves of k_attend_few: eight where 256 registers hold what one works on, else four.
constexpr int few_waves(int dim, int ct) { return dim == 256 || (dim == 128 && ct == 2) ? 4 : 8; }
// Workgroups of k_join: it takes further rows in a loop.
constexpr int64_t kMostGroups = 1 << 20;

// (positions end before 2^31, and so do steps before 2^25)
int room_of(const tri_cache &c, const tri_sequences &sq)
{
    return (int)std::min((sq.width * c.page + kStep - 1) / kStep, (int64_t)1 << 25);
}

AttendPlan plan_of(const tri_cache &c, const tri_sequences &sq, int T, int H, int64_t window, int64_t sinks)
{
    AttendPlan p;
    const int64_t G = H / c.heads, most = sq.max_new < T ? sq.max_new : T, rows = most * G;
    p.tall = rows > 32;
    p.height = p.tall ? kTallRows : rows <= 16 || c.dim == 256 ? 16 : 32;
    p.tiles = (int)((rows + p.height - 1) / p.height);
    int64_t steps = std::min((sq.max_len + kStep - 1) / kStep, (int64_t)room_of(c, sq));
    if (window > 0) {
        const int64_t seen = (window + p.height + kStep - 2) / kStep + 1 + ((sinks < sq.max_len ? sinks : sq.max_len) + kStep - 1) / kStep;
        steps = steps < seen ? steps : seen;
    }
    const int64_t groups = sq.B * c.heads * p.tiles, cus = cu_count();
    // Tall tiles: one pass over a tile's steps, unless the tiles leave half the CUs idle (what joins splits moves as much as many
    // steps do).  Up to two tiles per CU, the longest tile's steps are what the call waits for: two groups of waves share them
    // (2048 tokens of 32 heads, 512 tiles: 75 us without, 68 with; 1008 tiles over a window: 119 us without, 137 with).
    p.pair = p.tall && groups <= 2 * cus;
    const int64_t want = p.tall ? (groups * 2 > cus ? 1 : cus / groups) : (cus + groups - 1) / groups;
    int64_t chunk = (steps + want - 1) / want;
    const int64_t least = p.tall ? 16 : few_waves(c.dim, p.height / 16);
    chunk = chunk < least ? least : chunk;
    p.chunk = (int)chunk;
    p.splits = (int)((steps + chunk - 1) / chunk);
    return p;
}

template <int D, int FMT>
void attend_dim(const Attend &at, const AttendPlan &p, float *part, hipStream_t s)
{
    if (!p.tall)
        for_grids(at.sq.B, p.tiles, (int64_t)at.c.heads * p.splits, [&](const Grid &gd, uint32_t groups) {
            if (p.height == 16) k_attend_few<D, FMT, 1, few_waves(D, 1)><<<groups, 64 * few_waves(D, 1), 0, s>>>(at, part, p, gd);
            else if constexpr (D < 256) k_attend_few<D, FMT, 2, few_waves(D, 2)><<<groups, 64 * few_waves(D, 2), 0, s>>>(at, part, p, gd);
        });
    if (p.splits > 1) {
        const int64_t rows = (int64_t)at.T * at.H;
        k_join<D, FMT><<<dim3((uint32_t)(rows < kMostGroups ? rows : kMostGroups)), 256, 0, s>>>(at, part, p.splits, p.chunk, p.height);
    }
}

}  // namespace

int64_t attend_workspace_bytes(const tri_cache &c, const tri_sequences &sq, int T, int H, int64_t window, int64_t sinks)
{
    const AttendPlan p = plan_of(c, sq, T, H, window, sinks);
    return p.splits > 1 ? (int64_t)T * H * p.splits * (c.dim + 4) * 4 : 0;
}

int launch_attend(Attend at, void *workspace, hipStream_t s)
{
    at.room = room_of(at.c, at.sq);
    const AttendPlan p = plan_of(at.c, at.sq, at.T, at.H, at.window, at.sinks);
    float *part = static_cast<float *>(workspace);
    if (p.tall) launch_attend_tall(at, p, part, s);
    auto dims = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (at.c.dim == 64) attend_dim<64, F>(at, p, part, s);
        else if (at.c.dim == 128) attend_dim<128, F>(at, p, part, s);
        else attend_dim<256, F>(at, p, part, s);
    };
    if (at.c.fmt == TRI_KV_INT8) dims(std::integral_constant<int, TRI_KV_INT8>{});
    else dims(std::integral_constant<int, TRI_KV_E4M3>{});
    return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
}

}  // namespace tri
