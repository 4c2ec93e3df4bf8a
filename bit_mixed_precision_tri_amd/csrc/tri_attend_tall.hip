// tri_attend_tall.hip -- attention over the 8-bit cache for many query rows of a key/value head (prefill).
//
// A workgroup takes NW * 32 * QT rows, 32 QT a wave, and walks the steps that they see.  A step's codes are read once,
// decoded to fp16 once, and lie in LDS for all waves (two buffers: while one is used, the next step's codes are written
// into the other and those after are on their way).  Both products are transposed as in tri_attend.hip, on
// v_mfma_f32_32x32x16_f16: a lane holds 16 weights of one row for every 32 tokens, which are its B operand of the second
// product as they lie; values are stored in LDS in the order of a lane's tokens, so that an A operand is one 16-byte read.
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
template <int D> constexpr int kTallWaves = 4;
template <int D> constexpr int kTallCols = 1;

// 16-byte chunk c of row r among rows of N chunks: placed so that 16 lanes that read one chunk of 16 rows meet all banks.
template <int N>
__device__ __forceinline__ int chunk_at(int r, int c)
{
    constexpr int per = N >= 16 ? 1 : 16 / N;    // rows in 256 bytes
    return r * N + (c ^ ((r / per) & (N >= 16 ? 15 : N - 1)));
}

template <int D, int FMT, int QT, int NW>
__device__ __forceinline__ void attend_tall(const Attend &at, float *__restrict__ part, int splits, int chunk, int split, int h, int r0,
                                            int b, u32x4 *lds)
{
    constexpr int STEP = kTallStep<D>, NT = 64 * NW, HEIGHT = 32 * QT * NW;
    constexpr int KC = D / 8, VC = STEP / 8;             // chunks of a key's and a value's row
    constexpr int KU = STEP * D / 16 / NT, VU = KU;      // 16-byte pieces of codes per thread
    constexpr int BLK = STEP / 16, TT = STEP / 32, DT = D / 32;
    constexpr int BUF = STEP * KC + D * VC;              // chunks of a buffer
    u32x4 *const meta_at = lds + 2 * BUF;                // (a, log2 u, 1 / u, whether the page is there) of 16 tokens
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), hf = lane >> 5, l = lane & 31;
    const tri_cache &c = at.c;
    const Tile t = tile_of(at, b, r0, HEIGHT);
    if (t.rows == 0) return;
    // (the plan counts steps of 64 tokens; a split's share in steps of this kernel's)
    constexpr int F = kStep / STEP;
    const int steps64 = t.st.count(), i0 = split * chunk, i1 = split == splits - 1 ? steps64 : min(steps64, i0 + chunk);
    if (split > 0 && i0 >= steps64) return;
    const int P = c.page, lp = 31 - __builtin_clz(P);
    const int64_t head_bytes = (int64_t)P * D;
    const float ck = at.scale * 1.44269504088896f * kCodeUnit<FMT>;
    const int n0 = i0 * F, n1 = i1 * F;
    auto token_of = [&](int n) { return t.st.at(n / F) * kStep + (n % F) * STEP; };

    // this wave's rows
    half8_t q[QT][D / 16];
    int pos[QT], wa = 0x7fffffff, wb = -1;               // positions of the wave's first and last row that exist
#pragma unroll
    for (int ct = 0; ct < QT; ++ct) {
        const int w = (wv * QT + ct) * 32 + l, r = r0 + w, i = r / at.G;
        const bool live = w < t.rows;
        pos[ct] = live ? t.sp.p0 + i : -1;
        const uint16_t *x = at.Q + (int64_t)(t.sp.r0 + (live ? i : 0)) * at.q_stride + (h * at.G + (live ? r % at.G : 0)) * D + 8 * hf;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) q[ct][s] = *reinterpret_cast<const half8_t *>(x + 16 * s);
    }
    {
        const int w0 = wv * QT * 32, w1 = min(w0 + QT * 32, t.rows) - 1;
        if (w0 <= w1) {
            wa = t.sp.p0 + (r0 + w0) / at.G;
            wb = t.sp.p0 + (r0 + w1) / at.G;
        }
    }

    // codes on their way to LDS
    const int32_t *table = at.sq.table + (int64_t)b * at.sq.width;
    u32x4 kr[KU], vr[VU];
    float sk = 0.f, sv = 0.f;
    bool here = false;
    auto page_of = [&](int64_t token) {
        const int64_t a = token >> lp;
        const int id = a < at.sq.width ? table[a] : -1;
        return id >= 0 && id < (int)c.pages ? id : -1;
    };
    auto load = [&](int n) {
        const int t0 = token_of(n);
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            const int u = k * NT + tid, tok = u / (D / 16), piece = u % (D / 16);
            const int id = max(page_of((int64_t)t0 + tok), 0);
            kr[k] = *reinterpret_cast<const u32x4 *>(c.K + ((int64_t)id * c.heads + h) * head_bytes + ((t0 + tok) & (P - 1)) * D + 16 * piece);
        }
#pragma unroll
        for (int k = 0; k < VU; ++k) {
            const int u = k * NT + tid, blk = u % BLK, d = u / BLK;
            const int id = max(page_of((int64_t)t0 + 16 * blk), 0);
            vr[k] = *reinterpret_cast<const u32x4 *>(c.V + ((int64_t)id * c.heads + h) * head_bytes + d * P + ((t0 + 16 * blk) & (P - 1)));
        }
        if (tid < BLK) {
            const int id = page_of((int64_t)t0 + 16 * tid);
            here = id >= 0;
            sk = c.K_scale[(int64_t)max(id, 0) * c.heads + h];
            sv = c.V_scale[(int64_t)max(id, 0) * c.heads + h];
        }
    };
    auto put = [&](int buf) {
        u32x4 *kb = lds + buf * BUF, *vb = kb + STEP * KC;
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            const int u = k * NT + tid, tok = u / (D / 16), piece = u % (D / 16);
            kb[chunk_at<KC>(tok, 2 * piece)] = __builtin_bit_cast(u32x4, decode8<FMT>(kr[k][0], kr[k][1]));
            kb[chunk_at<KC>(tok, 2 * piece + 1)] = __builtin_bit_cast(u32x4, decode8<FMT>(kr[k][2], kr[k][3]));
        }
#pragma unroll
        for (int k = 0; k < VU; ++k) {
            const int u = k * NT + tid, blk = u % BLK, d = u / BLK;
            vb[chunk_at<VC>(d, 2 * blk)] = __builtin_bit_cast(u32x4, decode8<FMT>(vr[k][0], vr[k][2]));
            vb[chunk_at<VC>(d, 2 * blk + 1)] = __builtin_bit_cast(u32x4, decode8<FMT>(vr[k][1], vr[k][3]));
        }
        if (tid < BLK) {
            const float u = here ? sv : 1.f;
            meta_at[buf * BLK + tid] = u32x4{__float_as_uint(ck * sk), __float_as_uint(log2_(u)), __float_as_uint(1.f / u), here ? 1u : 0u};
        }
    };

    float m[QT], sum[QT];
    float16_t o[QT][DT];
#pragma unroll
    for (int ct = 0; ct < QT; ++ct) {
        m[ct] = kNone;
        sum[ct] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[ct][d][e] = 0.f;
    }

    if (n0 < n1) {
        load(n0);
        put(0);
        if (n0 + 1 < n1) load(n0 + 1);
    }
    for (int n = n0; n < n1; ++n) {
        const int buf = (n - n0) & 1, t0 = token_of(n);
        __syncthreads();
        if (n + 1 < n1) put(buf ^ 1);
        if (n + 2 < n1) load(n + 2);
        // nothing of the step for this wave: it lies behind its last row, or between the first tokens and its first row's window
        if (t0 > wb || (at.window > 0 && wa - (t0 + STEP - 1) >= at.window && t0 >= at.sinks)) continue;
        const u32x4 *kb = lds + buf * BUF, *vb = kb + STEP * KC;
        float16_t s[QT][TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
            for (int ct = 0; ct < QT; ++ct)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[ct][tt][e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const half8_t a = __builtin_bit_cast(half8_t, kb[chunk_at<KC>(32 * tt + l, 2 * k + hf)]);
#pragma unroll
                for (int ct = 0; ct < QT; ++ct) s[ct][tt] = mfma32(a, q[ct][k], s[ct][tt]);
            }
        }
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
        half8_t w[QT][BLK];
#pragma unroll
        for (int ct = 0; ct < QT; ++ct) {
            float mx = kNone;
#pragma unroll
            for (int k = 0; k < BLK; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &x = reinterpret_cast<float *>(&s[ct][k / 2])[8 * (k % 2) + e];
                    x = fmaf(x, a[k], lu[k]);
                    if (!whole) {
                        const int j = t0 + 16 * k + 8 * (e / 4) + 4 * hf + e % 4;
                        if (meta_at[buf * BLK + k][3] == 0u || !sees(pos[ct], j, at.window, at.sinks)) x = -INFINITY;
                    }
                    mx = fmaxf(mx, x);
                }
            float other = mx;
            swap32(mx, other);
            mx = fmaxf(mx, other);
            if (__any(mx > m[ct])) {
                const float mn = fmaxf(m[ct], mx), f = exp2_(m[ct] - mn);
                m[ct] = mn;
                sum[ct] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[ct][d] *= f;
            }
            const float shift = kLift - m[ct];
#pragma unroll
            for (int k = 0; k < BLK; ++k) {
                float y[8], add = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = exp2_(s[ct][k / 2][8 * (k % 2) + e] + shift);
                    add += y[e];
                }
                sum[ct] = add == 0.f ? sum[ct] : fmaf(add, iu[k], sum[ct]);    // (a scale that no visible token has may be anything)
                w[ct][k] = __builtin_bit_cast(half8_t, u32x4{pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])});
            }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < BLK; ++k) {
                const half8_t v = __builtin_bit_cast(half8_t, vb[chunk_at<VC>(32 * d + l, 2 * k + hf)]);
#pragma unroll
                for (int ct = 0; ct < QT; ++ct) o[ct][d] = mfma32(v, w[ct][k], o[ct][d]);
            }
    }

#pragma unroll
    for (int ct = 0; ct < QT; ++ct) {
        float other = sum[ct], den = sum[ct];
        swap32(den, other);
        den += other;
        const int w = (wv * QT + ct) * 32 + l, r = r0 + w;
        if (w >= t.rows) continue;
        const int64_t row = (int64_t)(t.sp.r0 + r / at.G);
        const int head = h * at.G + r % at.G;
        uint16_t *y = at.O + row * at.o_stride + head * D;
        float *p = part + ((row * at.H + head) * splits + split) * (D + 4);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4_t v = {o[ct][d][4 * e], o[ct][d][4 * e + 1], o[ct][d][4 * e + 2], o[ct][d][4 * e + 3]};
                const int at_d = 32 * d + 8 * e + 4 * hf;
                if (splits == 1) store_row<FMT>(y + at_d, v, den);
                else *reinterpret_cast<float4_t *>(p + at_d) = v;
            }
        if (splits > 1 && hf == 0) {
            p[D] = m[ct];
            p[D + 1] = den;
        }
    }
}

// Jobs: key/value head and sequence (fastest: the tiles of one head go to one XCD where their number is a multiple of 8), split,
// row tile, the last one (which sees most) first.
template <int D, int FMT, int QT, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void k_attend_tall(const Attend at, float *__restrict__ part, int splits, int chunk, int tiles,
                                                            int64_t jobs)
{
    constexpr int STEP = kTallStep<D>;
    __shared__ u32x4 lds[2 * (STEP * (D / 8) + D * (STEP / 8)) + 2 * (STEP / 16)];
    const int64_t pairs = at.sq.B * at.c.heads;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t k = job % pairs, n = job / pairs;
        if (job != blockIdx.x) __syncthreads();  // (the last job's steps have been read)
        attend_tall<D, FMT, QT, NW>(at, part, splits, chunk, (int)(n % splits), (int)(k % at.c.heads),
                                    (tiles - 1 - (int)(n / splits)) * (32 * QT * NW), (int)(k / at.c.heads), lds);
    }
}

}  // namespace

int tall_height(int dim)
{
    return dim == 64 ? 32 * kTallCols<64> * kTallWaves<64> : dim == 128 ? 32 * kTallCols<128> * kTallWaves<128>
                                                                        : 32 * kTallCols<256> * kTallWaves<256>;
}

void launch_attend_tall(const Attend &at, const AttendPlan &p, float *part, hipStream_t s)
{
    const int64_t jobs = (int64_t)p.splits * at.c.heads * p.tiles * at.sq.B;
    const dim3 grid((uint32_t)(jobs < kMostGroups ? jobs : kMostGroups));
    auto go = [&](auto dim, auto fmt) {
        constexpr int D = decltype(dim)::value, F = decltype(fmt)::value;
        k_attend_tall<D, F, kTallCols<D>, kTallWaves<D>><<<grid, 64 * kTallWaves<D>, 0, s>>>(at, part, p.splits, p.chunk, p.tiles, jobs);
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
