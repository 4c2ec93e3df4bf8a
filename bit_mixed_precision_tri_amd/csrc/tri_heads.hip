// tri_heads.hip -- norm and rotation of heads (tri_heads_rotate), and new keys and values into the pages of an 8-bit cache
// (tri_cache_append).
//
// A head's row of D values lies in D/16 lanes, two pieces of 8 values (16 bytes) each: pieces i and i + dims/16 where pairs
// are (x[i], x[i + dims/2]), so that a lane holds both values of its eight pairs and the rotation crosses no lanes; the
// pieces behind the rotated ones go two by two.  The sum of squares crosses 4, 8 or 16 lanes by DPP.
//
// Rotation reads and writes every value once and is bound by memory: 2048 tokens of 64 heads of 128 (68 MB) take 14.1 us in
// a graph, copying as much at the rate of a large copy 11.1; one token takes 2.4, an empty launch 1.6.  Two units of heads per
// wave have their loads on their way together (one: 15.2 us; four: 15 - 16).  Appending has two latencies more: where the page
// lies (three dependent reads), and the scale, which all of a page's values decide before the first is written: 2048 tokens
// of 32 heads with the queries' rotation (85 MB) take 22 us, one token 3.4.  With the queries' workgroups first, or mixed with
// the pages', the former takes 22.4 and 23.4.
#include "tri_cache.h"

namespace tri {

namespace {

struct Sets {
    tri_heads set[TRI_MAX_GROUPS];
    int first[TRI_MAX_GROUPS + 1];               // a token's waves: set q owns first[q] .. first[q+1]-1
    int G;
};

// Sum over the D/16 lanes of a row (aligned groups of 4, 8 or 16 lanes), in every one of them.
template <int D>
__device__ __forceinline__ float row_sum(float v)
{
    v += dpp<0xB1>(v);                           // quad_perm: lane ^ 1
    v += dpp<0x4E>(v);                           // lane ^ 2
    if constexpr (D >= 128) v += dpp<0x141>(v);  // row_half_mirror
    if constexpr (D >= 256) v += dpp<0x140>(v);  // row_mirror
    return v;
}

// A lane's sixteen values of a row: piece ca (a) and piece cb (b).
struct Piece2 {
    u32x4 a, b;
};
__device__ __forceinline__ void pieces_of(int i, int dims, int &ca, int &cb)
{
    const int nr = dims / 16;
    ca = i < nr ? i : 2 * i;
    cb = i < nr ? i + nr : 2 * i + 1;
}

// What a lane's values are turned with: the gains of its pieces and the (cos, sin) of its eight pairs.
struct Turn {
    Piece2 gain;
    float4_t cs[4];
};
__device__ __forceinline__ void load_gain(Turn &tn, const tri_rotary &rot, const uint16_t *gain, int i)
{
    int ca, cb;
    pieces_of(i, rot.dims, ca, cb);
    const u32x4 one = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    tn.gain = Piece2{one, one};
    if (rot.norm && gain)
        tn.gain = Piece2{*reinterpret_cast<const u32x4 *>(gain + 8 * ca), *reinterpret_cast<const u32x4 *>(gain + 8 * cb)};
}
// (p: a position that the table has)
__device__ __forceinline__ void load_angles(Turn &tn, const tri_rotary &rot, int p, int i)
{
    if (i >= rot.dims / 16) return;
    int ca, cb;
    pieces_of(i, rot.dims, ca, cb);
    const float4_t *t = reinterpret_cast<const float4_t *>(rot.table + (int64_t)p * rot.dims);
    const int a = rot.interleaved ? 2 * ca : 4 * i, b = rot.interleaved ? 2 * cb : 4 * i + 2;
    tn.cs[0] = t[a], tn.cs[1] = t[a + 1], tn.cs[2] = t[b], tn.cs[3] = t[b + 1];
}

// Norm and rotation of a lane's values, in fp32, rounded to fp16 at the end.
template <int D>
__device__ __forceinline__ void turn_row(Piece2 &v, const tri_rotary &rot, const Turn &tn, int i)
{
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = h2f((uint16_t)(v.a[e / 2] >> (16 * (e % 2))));
        x[8 + e] = h2f((uint16_t)(v.b[e / 2] >> (16 * (e % 2))));
    }
    if (rot.norm) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s = fmaf(x[e], x[e], s);
        const float r = 1.f / sqrtf(row_sum<D>(s) * (1.f / D) + rot.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= r * h2f((uint16_t)(tn.gain.a[e / 2] >> (16 * (e % 2))));
            x[8 + e] *= r * h2f((uint16_t)(tn.gain.b[e / 2] >> (16 * (e % 2))));
        }
    }
    if (i < rot.dims / 16) {
        if (rot.interleaved) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float c = tn.cs[p / 2][2 * (p % 2)], s = tn.cs[p / 2][2 * (p % 2) + 1], a = x[2 * p], b = x[2 * p + 1];
                x[2 * p] = a * c - b * s;
                x[2 * p + 1] = a * s + b * c;
            }
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float c = tn.cs[p / 2][2 * (p % 2)], s = tn.cs[p / 2][2 * (p % 2) + 1], a = x[p], b = x[8 + p];
                x[p] = a * c - b * s;
                x[8 + p] = a * s + b * c;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const half2_t a = {(_Float16)x[2 * q], (_Float16)x[2 * q + 1]}, b = {(_Float16)x[8 + 2 * q], (_Float16)x[9 + 2 * q]};
        v.a[q] = __builtin_bit_cast(uint32_t, a);
        v.b[q] = __builtin_bit_cast(uint32_t, b);
    }
}

// The heads of N units (of a token's) from `w` on of token t, at position p; a unit is as many heads as a wave has rows of lanes.
template <int D, int N>
__device__ __forceinline__ void rotate_units(const Sets &sets, const tri_rotary &rot, int t, int w, int p)
{
    const int lane = threadIdx.x & 63, i = lane % (D / 16), per = sets.first[sets.G];
    int ca, cb;
    pieces_of(i, rot.dims, ca, cb);
    uint16_t *y[N];
    Piece2 v[N];
    Turn tn[N];                                  // (all of them have the token's angles)
#pragma unroll
    for (int n = 0; n < N; ++n) {
        tri_heads hs = sets.set[0];
        int first = 0;
#pragma unroll
        for (int q = 1; q < TRI_MAX_GROUPS; ++q)
            if (q < sets.G && w + n >= sets.first[q]) hs = sets.set[q], first = sets.first[q];
        const int h = (w + n - first) * (1024 / D) + lane / (D / 16);
        y[n] = nullptr;
        load_gain(tn[n], rot, reinterpret_cast<const uint16_t *>(hs.gain), i);
        if (w + n < per && h < hs.heads) {       // (whole rows of lanes)
            const uint16_t *x = reinterpret_cast<const uint16_t *>(hs.X) + (int64_t)t * hs.x_stride + h * D;
            y[n] = reinterpret_cast<uint16_t *>(hs.Y) + (int64_t)t * hs.y_stride + h * D;
            v[n] = Piece2{*reinterpret_cast<const u32x4 *>(x + 8 * ca), *reinterpret_cast<const u32x4 *>(x + 8 * cb)};
        }
    }
    load_angles(tn[0], rot, p, i);
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (y[n]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) tn[n].cs[q] = tn[0].cs[q];
            turn_row<D>(v[n], rot, tn[n], i);
            *reinterpret_cast<u32x4 *>(y[n] + 8 * ca) = v[n].a;
            *reinterpret_cast<u32x4 *>(y[n] + 8 * cb) = v[n].b;
        }
}

// A position's place in the rotation's table, or none.
__device__ __forceinline__ bool turns(const tri_rotary &rot, int p) { return rot.dims == 0 || (p >= 0 && p < (int)rot.rows); }

// A wave takes N units of a token's heads.
template <int D, int N>
__global__ __launch_bounds__(256) void k_rotate(const Sets sets, const tri_rotary rot, const int32_t *__restrict__ positions, uint32_t waves)
{
    const uint32_t per = (sets.first[sets.G] + N - 1) / N;
    for (uint32_t u = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < waves; u += gridDim.x * 4) {
        const int t = (int)(u / per), p = positions[t];
        if (turns(rot, p)) rotate_units<D, N>(sets, rot, t, (int)(u % per) * N, p);
    }
}

struct Append {
    tri_cache c;
    tri_sequences sq;
    tri_rotary rot;                              // (dims 0 and no norm where keys are taken as they are)
    const uint16_t *X[2];                        // keys, values
    int64_t stride[2];
    const uint16_t *gain;
    int T, slots, turn;                          // slots: pages that one sequence's tokens may touch; turn: keys have a norm or rotation
};

// A sequence's new tokens in one of the pages that they touch, for one head's keys (which 0) or values (1).
struct Part {
    const uint16_t *x;                           // the first token's values; token r's are r * stride further
    uint8_t *codes;                              // the page
    float *scale;
    float was;                                   // the page's scale where it holds earlier tokens, else 0
    int first, cnt, pos;                         // the first token's place in the page, their number, the first one's position
};
template <int D>
__device__ __forceinline__ bool find_part(const Append &ap, int which, int b, int h, int slot, Part &pt)
{
    const tri_cache &c = ap.c;
    const Span sp = span_of(ap.sq, ap.T, b);
    // (positions are below 2^31 - 256, and so are the ends of the pages that hold them)
    const int P = c.page, lp = 31 - __builtin_clz(P), from = max(sp.p0, 0), end = sp.p0 + sp.n;
    const int to = ap.rot.dims > 0 ? (int)min((int64_t)end, ap.rot.rows) : end;
    const int pi = (from >> lp) + slot;
    if (pi > (to - 1) >> lp || from >= to) return false;
    const int lo = max(from, pi << lp), hi = min(to, (pi + 1) << lp);
    const int id = page_at(ap.sq, c, b, pi);
    if (id < 0) return false;
    const int64_t at = (int64_t)id * c.heads + h;
    pt.first = lo - (pi << lp);
    pt.cnt = hi - lo;
    pt.pos = lo;
    pt.x = ap.X[which] + (int64_t)(sp.r0 + (lo - sp.p0)) * ap.stride[which] + h * D;
    pt.codes = (which ? c.V : c.K) + at * P * D;
    pt.scale = (which ? c.V_scale : c.K_scale) + at;
    pt.was = pt.first > 0 ? *pt.scale : 0.f;
    return true;
}

// With the largest magnitude of the new values: the page's scale from now on, written where it changes, its earlier codes
// rounded to it (byte by byte: a page's scale grows a few times at most).  Returns fp32(1 / scale).
template <int D, int FMT, int NT>
__device__ __forceinline__ float settle_scale(const Part &pt, int P, int which, uint32_t most)
{
    const float need = __uint_as_float((uint32_t)(scale_exponent<FMT>(most) + 127) << 23);
    const bool grow = !(pt.was >= need);
    const float inv = 1.f / (grow ? need : pt.was);
    if (grow) {
        if (threadIdx.x == 0) *pt.scale = need;
        const float ratio = pt.was * inv;
        for (int e = threadIdx.x; e < pt.first * D; e += NT) {
            uint8_t *p = which == 0 ? pt.codes + e : pt.codes + (e / pt.first) * P + e % pt.first;
            *p = (uint8_t)encode4<FMT>(code_value<FMT>(*p), 0.f, 0.f, 0.f, ratio);
        }
    }
    return inv;
}

__device__ __forceinline__ uint32_t magnitude2(uint32_t v) { return max(magnitude(v & 0xFFFFu), magnitude(v >> 16)); }
__device__ __forceinline__ uint32_t magnitude8(const u32x4 &v)
{
    return max(max(magnitude2(v[0]), magnitude2(v[1])), max(magnitude2(v[2]), magnitude2(v[3])));
}
template <int NT>
__device__ __forceinline__ uint32_t most_of_all(uint32_t v, uint32_t *sm)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, m));
    if constexpr (NT > 64) {
        __syncthreads();                         // (the last job's reads of sm are done)
        if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NT / 64; ++k) v = max(v, sm[k]);
    }
    return v;
}

template <int FMT>
__device__ __forceinline__ uint2 encode8(const u32x4 &v, float inv)
{
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = plain_value((v[e / 2] >> (16 * (e % 2))) & 0xFFFFu);
    return make_uint2(encode4<FMT>(f[0], f[1], f[2], f[3], inv), encode4<FMT>(f[4], f[5], f[6], f[7], inv));
}

// Keys of a page: rows of D/16 lanes, NT / (D/16) of them in a pass, held while the largest value is found.
template <int D, int FMT, int NT, int PASSES>
__device__ __forceinline__ void append_keys(const Append &ap, const Part &pt, uint32_t *sm)
{
    constexpr int LPR = D / 16, RPP = NT / LPR;
    const int i = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
    int ca, cb;
    pieces_of(i, ap.rot.dims, ca, cb);
    Piece2 v[PASSES];
    Turn tn[PASSES];
    uint32_t most = 0;
    load_gain(tn[0], ap.rot, ap.gain, i);
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int r = s * RPP + r0;
        v[s] = Piece2{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
        if (r < pt.cnt) {
            load_angles(tn[s], ap.rot, pt.pos + r, i);
            const uint16_t *x = pt.x + r * ap.stride[0];
            v[s] = Piece2{*reinterpret_cast<const u32x4 *>(x + 8 * ca), *reinterpret_cast<const u32x4 *>(x + 8 * cb)};
        }
    }
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int r = s * RPP + r0;
        tn[s].gain = tn[0].gain;
        if (ap.turn && r < pt.cnt) turn_row<D>(v[s], ap.rot, tn[s], i);
        most = max(most, max(magnitude8(v[s].a), magnitude8(v[s].b)));
    }
    const float inv = settle_scale<D, FMT, NT>(pt, ap.c.page, 0, most_of_all<NT>(most, sm));
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int r = s * RPP + r0;
        if (r >= pt.cnt) continue;
        uint8_t *row = pt.codes + (pt.first + r) * D;
        *reinterpret_cast<uint2 *>(row + 8 * ca) = encode8<FMT>(v[s].a, inv);
        *reinterpret_cast<uint2 *>(row + 8 * cb) = encode8<FMT>(v[s].b, inv);
    }
}

// Values of a page: a unit is four tokens (a dword of a stored row) times eight values; UNITS of them per thread.
template <int D, int FMT, int NT, int UNITS>
__device__ __forceinline__ void append_values(const Append &ap, const Part &pt, uint32_t *sm)
{
    const int P = ap.c.page, quads = P / 4;
    u32x4 w[UNITS][4];
    uint32_t most = 0;
#pragma unroll
    for (int s = 0; s < UNITS; ++s) {
        const int u = s * NT + threadIdx.x, q = u % quads, dc = u / quads;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 4 * q + k - pt.first;
            w[s][k] = u32x4{0u, 0u, 0u, 0u};
            if (dc < D / 8 && r >= 0 && r < pt.cnt) w[s][k] = *reinterpret_cast<const u32x4 *>(pt.x + r * ap.stride[1] + 8 * dc);
        }
    }
#pragma unroll
    for (int s = 0; s < UNITS; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, magnitude8(w[s][k]));
    const float inv = settle_scale<D, FMT, NT>(pt, P, 1, most_of_all<NT>(most, sm));
#pragma unroll
    for (int s = 0; s < UNITS; ++s) {
        const int u = s * NT + threadIdx.x, q = u % quads, dc = u / quads;
        const int r = 4 * q - pt.first;          // the unit's first token among the new ones
        if (dc >= D / 8 || r <= -4 || r >= pt.cnt) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = plain_value((w[s][k][e / 2] >> (16 * (e % 2))) & 0xFFFFu);
            const uint32_t four = encode4<FMT>(f[0], f[1], f[2], f[3], inv);
            uint8_t *p = pt.codes + (8 * dc + e) * P + 4 * q;
            if (r >= 0 && r + 4 <= pt.cnt) *reinterpret_cast<uint32_t *>(p) = four;
            else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r + k >= 0 && r + k < pt.cnt) p[k] = (uint8_t)(four >> (8 * k));
            }
        }
    }
}

// One token's keys or values of a head, by one wave.  Keys: every row of lanes computes the same, the first one writes.
template <int D, int FMT>
__device__ __forceinline__ void append_one(const Append &ap, const Part &pt, int which)
{
    const int lane = threadIdx.x;
    if (which == 0) {
        const int i = lane % (D / 16);
        int ca, cb;
        pieces_of(i, ap.rot.dims, ca, cb);
        Piece2 v = {*reinterpret_cast<const u32x4 *>(pt.x + 8 * ca), *reinterpret_cast<const u32x4 *>(pt.x + 8 * cb)};
        if (ap.turn) {
            Turn tn;
            load_gain(tn, ap.rot, ap.gain, i);
            load_angles(tn, ap.rot, pt.pos, i);
            turn_row<D>(v, ap.rot, tn, i);
        }
        const uint32_t most = most_of_all<64>(max(magnitude8(v.a), magnitude8(v.b)), nullptr);
        const float inv = settle_scale<D, FMT, 64>(pt, ap.c.page, 0, most);
        if (lane < D / 16) {
            uint8_t *row = pt.codes + pt.first * D;
            *reinterpret_cast<uint2 *>(row + 8 * ca) = encode8<FMT>(v.a, inv);
            *reinterpret_cast<uint2 *>(row + 8 * cb) = encode8<FMT>(v.b, inv);
        }
    } else {
        constexpr int N = D / 64;
        uint32_t x[N], most = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] = pt.x[64 * k + lane];
            most = max(most, magnitude(x[k]));
        }
        most = most_of_all<64>(most, nullptr);
        const float inv = settle_scale<D, FMT, 64>(pt, ap.c.page, 1, most);
#pragma unroll
        for (int k = 0; k < N; ++k)
            pt.codes[(64 * k + lane) * ap.c.page + pt.first] = (uint8_t)encode4<FMT>(plain_value(x[k]), 0.f, 0.f, 0.f, inv);
    }
}

// Workgroups: `pages` of them for keys and values of a head in a page slot of a sequence (gd.tile0 ..: slots), then the query
// heads' waves, of N units each.  PASSES 0: one token each.
template <int D, int FMT, int NT, int PASSES, int N>
__global__ __launch_bounds__(NT) void k_append(const Append ap, const Sets sets, const Grid gd, uint32_t pages, uint32_t waves)
{
    __shared__ uint32_t sm[NT / 64];
    if (blockIdx.x < pages) {
        const uint32_t which = blockIdx.x & 1, k = blockIdx.x >> 1, h = k % ap.c.heads, r = k / ap.c.heads;
        Part pt;                                 // (the same in every thread of the workgroup)
        if (!find_part<D>(ap, which, gd.seq0 + (int)(r / gd.tiles), (int)h, gd.tile0 + (int)(r % gd.tiles), pt)) return;
        if constexpr (PASSES == 0) append_one<D, FMT>(ap, pt, which);
        else if (which == 0) append_keys<D, FMT, NT, PASSES>(ap, pt, sm);
        else append_values<D, FMT, NT, (PASSES + 1) / 2>(ap, pt, sm);
        return;
    }
    const uint32_t per = (sets.first[sets.G] + N - 1) / N, step = (gridDim.x - pages) * (NT / 64);
    for (uint32_t u = (blockIdx.x - pages) * (NT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < waves; u += step) {
        const int t = (int)(u / per), b = owner(ap.sq, t);
        const Span sp = span_of(ap.sq, ap.T, b);
        const int i = t - sp.r0, p = sp.p0 + i;
        if (i >= 0 && i < sp.n && p >= 0 && turns(ap.rot, p)) rotate_units<D, N>(sets, ap.rot, t, (int)(u % per) * N, p);
    }
}

Sets make_sets(const tri_heads *heads, int G, int dim)
{
    Sets s{};
    s.G = G;
    for (int q = 0; q < G; ++q) {
        s.set[q] = heads[q];
        s.first[q + 1] = s.first[q] + (heads[q].heads + 1024 / dim - 1) / (1024 / dim);
    }
    for (int q = G; q < TRI_MAX_GROUPS; ++q) s.first[q + 1] = s.first[G];
    return s;
}

// Units of a wave: one while there are few, so that the chip fills, else two.
constexpr int kUnits = 2;
bool many_units(int64_t T, const Sets &s) { return T * s.first[s.G] >= 16 * (int64_t)cu_count(); }

// Waves are taken in a loop past this many workgroups.
constexpr int64_t kMostGroups = 1 << 20;

template <int D, int FMT>
void append_dim(const Append &ap, const Sets &sets, hipStream_t s)
{
    bool first = true;
    for_grids(ap.sq.B, ap.slots, 2 * (int64_t)ap.c.heads, [&](const Grid &gd, uint32_t pages) {
        auto go = [&](auto kernel, int nt, int units) {
            const int64_t waves = first ? ap.T * (int64_t)((sets.first[sets.G] + units - 1) / units) : 0;
            const int64_t more = (waves + nt / 64 - 1) / (nt / 64);
            kernel<<<dim3(pages + (uint32_t)(more < kMostGroups ? more : kMostGroups)), nt, 0, s>>>(ap, sets, gd, pages, (uint32_t)waves);
        };
        const int size = ap.c.page * D;
        // one new token per sequence: a wave each; else a page's tokens are held in registers by 256 to 1024 threads, at most 32
        // values each
        if (ap.sq.max_new == 1) go(k_append<D, FMT, 64, 0, 1>, 64, 1);
        else if (size <= 4096) go(k_append<D, FMT, 256, 1, kUnits>, 256, kUnits);
        else if (size <= 8192) go(k_append<D, FMT, 256, 2, kUnits>, 256, kUnits);
        else if (size <= 16384) go(k_append<D, FMT, 512, 2, kUnits>, 512, kUnits);
        else go(k_append<D, FMT, 1024, 2, kUnits>, 1024, kUnits);
        first = false;
    });
}

}  // namespace

int launch_rotate(const tri_heads *heads, int G, int T, int dim, const tri_rotary &rot, const int32_t *positions, hipStream_t s)
{
    const Sets sets = make_sets(heads, G, dim);
    const bool many = many_units(T, sets);
    const int units = many ? kUnits : 1;
    const int64_t waves = T * (int64_t)((sets.first[G] + units - 1) / units), wg = (waves + 3) / 4;
    const dim3 grid((uint32_t)(wg < kMostGroups ? wg : kMostGroups));
    auto go = [&](auto one, auto more) {
        if (many) more<<<grid, 256, 0, s>>>(sets, rot, positions, (uint32_t)waves);
        else one<<<grid, 256, 0, s>>>(sets, rot, positions, (uint32_t)waves);
    };
    if (dim == 64) go(k_rotate<64, 1>, k_rotate<64, kUnits>);
    else if (dim == 128) go(k_rotate<128, 1>, k_rotate<128, kUnits>);
    else go(k_rotate<256, 1>, k_rotate<256, kUnits>);
    return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
}

int launch_append(const tri_cache &c, const tri_sequences &sq, int T, const uint16_t *K, int64_t ks, const uint16_t *V,
                  int64_t vs, const tri_rotary *rot, const uint16_t *gain, const tri_heads *queries, hipStream_t s)
{
    Append ap{};
    ap.c = c;
    ap.sq = sq;
    if (rot) ap.rot = *rot;
    ap.turn = rot != nullptr;
    ap.X[0] = K;
    ap.X[1] = V;
    ap.stride[0] = ks;
    ap.stride[1] = vs;
    ap.gain = gain;
    ap.T = T;
    const int64_t most = sq.max_new < T ? sq.max_new : T;
    ap.slots = (int)((most + c.page - 2) / c.page + 1);
    const Sets sets = make_sets(queries, queries ? 1 : 0, c.dim);
    auto dims = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (c.dim == 64) append_dim<64, F>(ap, sets, s);
        else if (c.dim == 128) append_dim<128, F>(ap, sets, s);
        else append_dim<256, F>(ap, sets, s);
    };
    if (c.fmt == TRI_KV_INT8) dims(std::integral_constant<int, TRI_KV_INT8>{});
    else dims(std::integral_constant<int, TRI_KV_E4M3>{});
    return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
}

}  // namespace tri
