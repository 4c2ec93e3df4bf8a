// tri_attend_tall.hip -- attention over the 8-bit cache for many query rows of a key/value head (prefill).
//
// A workgroup takes 128 rows, 32 a wave, and walks the steps that they see.  A step's codes are read once,
// decoded to fp16 once, and lie in LDS for all waves (two buffers: while one is used, the next step's codes are written
// into the other and those after are on their way).  Both products are transposed as in tri_attend.hip, on
// v_mfma_f32_32x32x16_f16: a lane holds 16 weights of one row for every 32 tokens, which are its B operand of the second
// product as they lie; values are stored in LDS in the order of a lane's tokens, so that an A operand is one 16-byte read.
//
// A weight is the sum of two fp16 numbers, each a product with the values' codes: as one alone it would be off by up to 2^-11,
// more than the scores are, and than the rounding of a result where values cancel; a call's size would show in its results.  The
// third product of a step costs 2048 tokens of 32 heads 57.5 -> 66 us, 1000 over a window of 1024 101 -> 115, long contexts, which the
// matrix cores bound, up to 29% (2048 over 16384: 621 -> 800).  In which order the two products of the weights are issued changes nothing.
//
// Otherwise the softmax and the decoding (vector ALU) and the products (matrix cores) overlap only across the two waves of a SIMD,
// and waves wait a third of their cycles (barriers, the ends of tiles of uneven length).  2048 tokens of 32 heads of 128 (34.4 GFLOP
// below the diagonal) take 64 - 69 us from card to card, 500 - 535 TFLOP/s; 1000 tokens over a window of 1024, 64 heads (59.6
// GFLOP), 113 - 119, 500 - 530.  Measured and not taken, with one product of the weights (57.5 us): the groups in strict turns with
// two barriers a round (67 - 76), one step's weights beside the last step's values in a wave (60).
#include "tri_attend.h"

namespace tri {

namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

// v_mfma_f32_32x32x16_f16: lane (h = lane / 32, l = lane % 32) supplies A[l][8h..8h+7] and B[8h..8h+7][l] and holds
// D[8 (i / 4) + 4 h + i % 4][l] in register i.
__device__ __forceinline__ float16_t mfma32(half8_t a, half8_t b, float16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <int D> constexpr int kTallStep = D == 256 ? 32 : 64;   // tokens of a step here
constexpr int kWaves = kTallRows / 32;                           // waves that share a step, 32 rows each
// LDS of a group in 16-byte chunks: two buffers of keys, values and what belongs to 16 tokens.
template <int D> constexpr int kTallLds = 4 * D * (kTallStep<D> / 8) + 2 * (kTallStep<D> / 16);

// 16-byte chunk c of row r among rows of N chunks: placed so that 16 lanes that read one chunk of 16 rows meet all banks.
template <int N>
__device__ __forceinline__ int chunk_at(int r, int c)
{
    constexpr int per = N >= 16 ? 1 : 16 / N;    // rows in 256 bytes
    return r * N + (c ^ ((r / per) & (N >= 16 ? 15 : N - 1)));
}

template <int D, int FMT, int NG>
__device__ __forceinline__ void attend_tall(const Attend &at, float *__restrict__ part, int splits, int chunk, int split, int h, int r0,
                                            int b, u32x4 *lds)
{
    constexpr int STEP = kTallStep<D>, NT = 64 * kWaves;
    constexpr int KC = D / 8, VC = STEP / 8;             // chunks of a key's and a value's row
    constexpr int KU = STEP * D / 16 / NT, VU = KU;      // 16-byte pieces of codes per thread
    constexpr int BLK = STEP / 16, TT = STEP / 32, DT = D / 32;
    const int gr = __builtin_amdgcn_readfirstlane(threadIdx.x / NT), tid = threadIdx.x % NT;
    u32x4 *const all = lds;
    lds += gr * kTallLds<D>;
    u32x4 *const meta_at = lds + 4 * D * VC;             // (a, log2 u, 1 / u, whether the page is there) of 16 tokens
    const int lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), hf = lane >> 5, l = lane & 31;
    const tri_cache &c = at.c;
    const Tile t = tile_of(at, b, r0, kTallRows);
    if (t.rows == 0) return;
    // (the plan counts steps of 64 tokens; a split's share in steps of this kernel's)
    constexpr int F = kStep / STEP;
    const int steps64 = t.st.count(), i0 = split * chunk, i1 = split == splits - 1 ? steps64 : min(steps64, i0 + chunk);
    if (split > 0 && i0 >= steps64) return;
    const int P = c.page, lp = 31 - __builtin_clz(P);
    const int64_t head_bytes = (int64_t)P * D;
    const float ck = fabsf(at.scale) * 1.44269504088896f * kCodeUnit<FMT>;    // (the scale's sign goes into q)
    const uint32_t flip = at.scale < 0.f ? 0x80008000u : 0u;
    const int n0 = i0 * F + gr, n1 = i1 * F, rounds = (n1 - i0 * F + NG - 1) / NG;    // (the same for all groups)
    auto token_of = [&](int n) { return t.st.at(n / F) * kStep + (n % F) * STEP; };

    // this wave's rows, and this lane's: row `mine` of the tile, of new token tok and query head `head`
    const int mine = wv * 32 + l, tok = (r0 + mine) / at.G, head = h * at.G + (r0 + mine) % at.G;
    const bool live = mine < t.rows;
    const int pos = live ? t.sp.p0 + tok : -1;
    int wa = 0x7fffffff, wb = -1;                        // positions of the wave's first and last row that exist
    half8_t q[D / 16];
    {
        const uint16_t *x = at.Q + (int64_t)(t.sp.r0 + (live ? tok : 0)) * at.q_stride + (live ? head : h * at.G) * D + 8 * hf;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) q[s] = __builtin_bit_cast(half8_t, *reinterpret_cast<const u32x4 *>(x + 16 * s) ^ flip);
        const int w0 = wv * 32, w1 = min(w0 + 32, t.rows) - 1;
        if (w0 <= w1) {
            wa = t.sp.p0 + (r0 + w0) / at.G;
            wb = t.sp.p0 + (r0 + w1) / at.G;
        }
    }

    // Codes on their way to LDS; pages are looked up a step ahead of the codes.  A wave's piece of keys is of 16 tokens at most,
    // so of one page (its number goes into scalar registers); its values are of one page where a page holds the step, else of
    // a page per lane.
    const int32_t *table = at.sq.table + (int64_t)b * at.sq.width;
    const int last_page = (int)at.sq.width - 1;
    const bool big = P >= STEP;
    u32x4 kr[KU], vr[VU];
    float sk = 0.f, sv = 0.f;
    bool here = false;
    int kid[KU], vid = 0;
    static_assert(NT % BLK == 0 && 64 / (D / 16) <= 16, "");
    const int koff = ((tid / (D / 16)) & (P - 1)) * D + 16 * (tid % (D / 16)), ktok = wv * 64 / (D / 16);
    const int voff = (tid / BLK) * P + ((16 * (tid % BLK)) & (P - 1));
    auto look = [&](int n) {                             // (what the table holds: nothing here waits for it)
        const int t0 = token_of(n);
#pragma unroll
        for (int k = 0; k < KU; ++k)
            if (k == 0 || !big) kid[k] = table[min((t0 + k * (NT / (D / 16)) + ktok) >> lp, last_page)];
        if (!big) vid = table[min((t0 + 16 * (tid % BLK)) >> lp, last_page)];
    };
    auto load = [&](int n) {
        const int t0 = token_of(n), in = t0 & (P - 1);   // (0 where a page is smaller than a step)
        const int first = __builtin_amdgcn_readfirstlane(kid[0]);
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            const int id = big ? first : __builtin_amdgcn_readfirstlane(kid[k]);
            const uint8_t *x = c.K + ((int64_t)((uint32_t)id < (uint32_t)c.pages ? id : 0) * c.heads + h) * head_bytes;   // (none: any one's)
            kr[k] = *reinterpret_cast<const u32x4 *>(x + (big ? (in + k * (NT / (D / 16))) * D : ((k * (NT / (D / 16))) & (P - 1)) * D) + koff);
        }
        if (big) {
            const bool ok = (uint32_t)first < (uint32_t)c.pages;
            const int64_t pg = (int64_t)(ok ? first : 0) * c.heads + h;
            const uint8_t *x = c.V + pg * head_bytes + in;
#pragma unroll
            for (int k = 0; k < VU; ++k) vr[k] = *reinterpret_cast<const u32x4 *>(x + (k * (NT / BLK) * P + voff));
            here = ok && (t0 >> lp) <= last_page;
            sk = c.K_scale[pg];
            sv = c.V_scale[pg];
        } else {
            const bool ok = (uint32_t)vid < (uint32_t)c.pages;
            const int64_t pg = (int64_t)(ok ? vid : 0) * c.heads + h;
            const uint8_t *x = c.V + pg * head_bytes;
#pragma unroll
            for (int k = 0; k < VU; ++k) vr[k] = *reinterpret_cast<const u32x4 *>(x + (k * (NT / BLK) * P + voff));
            if (tid < BLK) {
                here = ok && (t0 + 16 * tid) >> lp <= last_page;
                sk = c.K_scale[pg];
                sv = c.V_scale[pg];
            }
        }
    };
    // where they go: rows k * NT / .. further lie that much further on (chunk_at's pattern repeats within them)
    const int kput = 16 * chunk_at<KC>(tid / (D / 16), 2 * (tid % (D / 16)));
    const int vput = 16 * (STEP * KC + chunk_at<VC>(tid / BLK, 2 * (tid % BLK)));
    static_assert(NT / (D / 16) % 16 == 0 && NT / BLK % 16 == 0, "");
    auto put = [&](int buf) {
        char *const x = reinterpret_cast<char *>(lds) + buf * (2 * D * VC * 16);
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            *reinterpret_cast<half8_t *>(x + kput + k * (NT / (D / 16) * KC * 16)) = decode8<FMT>(kr[k][0], kr[k][1]);
            *reinterpret_cast<half8_t *>(x + (kput ^ 16) + k * (NT / (D / 16) * KC * 16)) = decode8<FMT>(kr[k][2], kr[k][3]);
        }
#pragma unroll
        for (int k = 0; k < VU; ++k) {
            char *const v = x + k * (NT / BLK * VC * 16);
            *reinterpret_cast<half8_t *>(v + vput) = decode8<FMT>(vr[k][0], vr[k][2]);
            *reinterpret_cast<half8_t *>(v + (vput ^ 16)) = decode8<FMT>(vr[k][1], vr[k][3]);
        }
        if (tid < BLK) {
            const float u = usable(sv);
            meta_at[buf * BLK + tid] = u32x4{__float_as_uint(usable(ck * sk)), __float_as_uint(log2_(u)), __float_as_uint(1.f / u),
                                             here ? 1u : 0u};
        }
    };

    const float minus = minus_one();
    float m = kNone, sum = 0.f;
    float16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.f;

    // A operands: chunk 2 k + hf of a row, where chunk_at puts it (its exclusive or with 2 k is one of the byte address, too)
    const char *const bytes = reinterpret_cast<const char *>(lds);
    const int key0 = 16 * chunk_at<KC>(l, hf), val0 = 16 * (STEP * KC + chunk_at<VC>(l, hf));
    auto key = [&](int buf, int tt, int k) {
        return *reinterpret_cast<const half8_t *>(bytes + buf * (2 * D * VC * 16) + (key0 ^ (32 * k)) + tt * (32 * KC * 16));
    };
    auto val = [&](int buf, int d, int k) {
        return *reinterpret_cast<const half8_t *>(bytes + buf * (2 * D * VC * 16) + (val0 ^ (32 * k)) + d * (32 * VC * 16));
    };
    float16_t s[TT];
    half8_t w[BLK], wl[BLK];                             // weights, and what their rounding to fp16 left off
    // Operands are read two products ahead: the groups of the schedule keep the compiler to that.
    auto values = [&](int buf) {
        half8_t va[2][DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) va[0][d] = val(buf, d, 0);
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            if (k + 1 < BLK) {
#pragma unroll
                for (int d = 0; d < DT; ++d) va[(k + 1) & 1][d] = val(buf, d, k + 1);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] = mfma32(va[k & 1][d], w[k], o[d]);
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] = mfma32(va[k & 1][d], wl[k], o[d]);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, DT + 1, 0);
#pragma unroll
        for (int i = 0; i < BLK * DT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
    };
    auto scores = [&](int buf) {
        half8_t ka[3][TT];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) ka[k][tt] = key(buf, tt, k);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            if (k + 2 < D / 16) {
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) ka[(k + 2) % 3][tt] = key(buf, tt, k + 2);
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                if (k == 0) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[tt][e] = 0.f;
                }
                s[tt] = mfma32(ka[k % 3][tt], q[k], s[tt]);
            }
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * TT + 1, 1);
#pragma unroll
        for (int i = 0; i < TT * D / 16; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        }
    };
    // the scores' weights
    auto weigh = [&](int buf, int t0) {
        float a[BLK], lu[BLK], iu[BLK];
        uint32_t there = 1u;
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            const u32x4 x = meta_at[buf * BLK + k];
            a[k] = __uint_as_float(x[0]);
            lu[k] = __uint_as_float(x[1]);
            iu[k] = __uint_as_float(x[2]);
            there &= x[3];
        }
        const bool whole = t0 + STEP - 1 <= wa && (at.window == 0 || wb - t0 < at.window || t0 + STEP <= at.sinks) &&
                           __builtin_amdgcn_readfirstlane(there) != 0;
        if (!whole) {
            const unsigned long long seen = seen_of(pos, t0 + 4 * hf, at.window, at.sinks);
            uint32_t part_of[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
            for (int k = 0; k < BLK; ++k)
                if (meta_at[buf * BLK + k][3] == 0u) part_of[k / 2] &= k % 2 ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
            for (int k = 0; k < BLK; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((part_of[k / 2] >> (16 * (k % 2) + 8 * (e / 4) + e % 4) & 1u) == 0u) s[k / 2][8 * (k % 2) + e] = -INFINITY;
        }
        // the largest y of a block is its largest score's (a > 0)
        float mx = kNone;
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            float top = s[k / 2][8 * (k % 2)];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, s[k / 2][8 * (k % 2) + e]);
            mx = fmaxf(mx, fmaf(top, a[k], lu[k]));
        }
        float other = mx;
        swap32(mx, other);
        mx = fmaxf(mx, other);
        // m need not be the maximum: within 2^kSlack of it, weights still are fp16 numbers and o stays as it is
        if (__any(mx - m > kSlack)) {
            const float mn = fmaxf(m, mx), f = exp2_(m - mn);
            m = mn;
            sum *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
        }
        float f[BLK], shift[BLK];
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            f[k] = a[k];
            shift[k] = lu[k] + (kLift - m);
        }
        if (is_far(m)) {                         // (by row: no row goes by what others hold)
#pragma unroll
            for (int k = 0; k < BLK; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = 8 * (k % 2) + e;
                    s[k / 2][at] = fmaf(s[k / 2][at], a[k], lu[k]) - m;
                }
                f[k] = 1.f;
                shift[k] = kLift;
            }
        }
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            float den = 0.f;
            u32x4 hi, lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 8 * (k % 2) + 2 * e;
                const float y0 = exp2_(fmaf(s[k / 2][at], f[k], shift[k])), y1 = exp2_(fmaf(s[k / 2][at + 1], f[k], shift[k]));
                den += y0 + y1;
                const uint2 x = split2(y0, y1, minus);
                hi[e] = x.x;
                lo[e] = x.y;
            }
            w[k] = __builtin_bit_cast(half8_t, hi);
            wl[k] = __builtin_bit_cast(half8_t, lo);
            sum = fmaf(den, iu[k], sum);
        }
    };

    if (n0 < n1) {
        look(n0);
        load(n0);
        if (n0 + NG < n1) look(n0 + NG);
        put(0);
        if (n0 + NG < n1) load(n0 + NG);
        if (n0 + 2 * NG < n1) look(n0 + 2 * NG);
    }
    // The second group decodes the next step's codes at the end of a round, the first at its start: so one's waves feed the
    // matrix cores while the other's, on the same SIMDs, use the vector ALU.
    for (int it = 0; it < rounds; ++it) {
        const int n = n0 + it * NG, buf = it & 1, t0 = token_of(n < n1 ? n : n0);
        // nothing of the step for this wave: there is none, it lies behind its last row, or between the first tokens and its first
        // row's window
        const bool idle = n >= n1 || t0 > wb || (at.window > 0 && wa - (t0 + STEP - 1) >= at.window && t0 >= at.sinks);
        auto next = [&]() {
            if (n + NG < n1) put(buf ^ 1);
            if (n + 2 * NG < n1) load(n + 2 * NG);
            if (n + 3 * NG < n1) look(n + 3 * NG);
        };
        __syncthreads();
        if (gr == 0) next();
        if (!idle) {
            scores(buf);
            weigh(buf, t0);
            values(buf);
        }
        if (gr != 0) next();
    }

    // the groups' sums, one after the other through LDS
#pragma unroll
    for (int from = 1; from < NG; ++from) {
        __syncthreads();
        if (gr == from) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    reinterpret_cast<float4_t *>(all)[(d * 4 + e) * NT + tid] =
                        float4_t{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            reinterpret_cast<float2 *>(all + DT * 4 * NT)[tid] = make_float2(m, sum);
        }
        __syncthreads();
        if (gr == 0) {
            const float2 x = reinterpret_cast<const float2 *>(all + DT * 4 * NT)[tid];
            const float mn = fmaxf(m, x.x), f = exp2_(m - mn), g = exp2_(x.x - mn);
            m = mn;
            sum = sum * f + x.y * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4_t v = reinterpret_cast<const float4_t *>(all)[(d * 4 + e) * NT + tid];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d][4 * e + i] = o[d][4 * e + i] * f + v[i] * g;
                }
        }
    }
    if (gr != 0) return;
    float other = sum, den = sum;
    swap32(den, other);
    den += other;
    if (!live) return;
    const int64_t row = (int64_t)(t.sp.r0 + tok);
    uint16_t *y = at.O + row * at.o_stride + head * D;
    float *p = part + ((row * at.H + head) * splits + split) * (D + 4);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4_t v = {o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            const int at_d = 32 * d + 8 * e + 4 * hf;
            if (splits == 1) store_row<FMT>(y + at_d, v, den);
            else *reinterpret_cast<float4_t *>(p + at_d) = v;
        }
    if (splits > 1 && hf == 0) {
        p[D] = m;
        p[D + 1] = den;
    }
}

// Workgroups: key/value head and sequence (fastest: the tiles of one head go to one XCD where their number is a multiple of 8),
// split, row tile, the last one (which sees most) first.
template <int D, int FMT, int NG>
__global__ __launch_bounds__(64 * kWaves * NG, D == 256 ? 1 : 2) void k_attend_tall(const Attend at, float *__restrict__ part, const AttendPlan p,
                                                                                    const Grid gd)
{
    __shared__ u32x4 lds[NG * kTallLds<D>];
    static_assert(NG <= 2 && (NG == 1 || NG * kTallLds<D> >= (D / 32) * 4 * 64 * kWaves + 32 * kWaves), "the groups' sums");
    const uint32_t pairs = gd.seqs * at.c.heads, k = blockIdx.x % pairs, n = blockIdx.x / pairs;
    const int tile = gd.tile0 + gd.tiles - 1 - (int)(n / p.splits);
    attend_tall<D, FMT, NG>(at, part, p.splits, p.chunk, (int)(n % p.splits), (int)(k % at.c.heads), tile * kTallRows,
                            gd.seq0 + (int)(k / at.c.heads), lds);
}

}  // namespace

void launch_attend_tall(const Attend &at, const AttendPlan &p, float *part, hipStream_t s)
{
    auto go = [&](auto dim, auto fmt) {
        constexpr int D = decltype(dim)::value, F = decltype(fmt)::value;
        for_grids(at.sq.B, p.tiles, (int64_t)at.c.heads * p.splits, [&](const Grid &gd, uint32_t groups) {
            if constexpr (D < 256) {
                if (p.pair) {
                    k_attend_tall<D, F, 2><<<groups, 128 * kWaves, 0, s>>>(at, part, p, gd);
                    return;
                }
            }
            k_attend_tall<D, F, 1><<<groups, 64 * kWaves, 0, s>>>(at, part, p, gd);
        });
    };
    auto dims = [&](auto fmt) {
        if (at.c.dim == 64) go(std::integral_constant<int, 64>{}, fmt);
        else if (at.c.dim == 128) go(std::integral_constant<int, 128>{}, fmt);
        else go(std::integral_constant<int, 256>{}, fmt);
    };
    if (at.c.fmt == TRI_KV_INT8) dims(std::integral_constant<int, TRI_KV_INT8>{});
    else dims(std::integral_constant<int, TRI_KV_E4M3>{});
}

}  // namespace tri
