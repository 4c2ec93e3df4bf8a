// tri_attend.h -- what the kernels of attention over the 8-bit cache share (tri_attend.hip says what they compute).
#pragma once
#include "tri_cache.h"

namespace tri {

constexpr int kStep = 64;                        // tokens of a step
// Weights are lifted by 2^10; the running maximum follows only when it is 2^5 behind: a weight stays below 2^15, and the sums
// need no scaling in most steps.
constexpr float kLift = 10.f, kSlack = 5.f;
constexpr float kNone = -3.402823466e38f;        // the running maximum of a row that has seen nothing
// A running maximum this far from 0 is off from its score's exponent, which is rounded once and elsewhere, by as much as a weight may
// be off; much further, by more than fp16's exponents hold.  There exponents are differences of rounded numbers, at one operation
// more per score, so that the largest is 0.
constexpr float kFar = 1048576.f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m > kNone; }

// The steps that rows of positions pa .. pb (pa <= pb) see some token of: 0 .. head-1, then from .. from + tail - 1.  None of them
// lies behind the `room` steps that the table of pages has places for, whatever a length says.
struct Steps {
    int head, from, tail;
    __device__ __forceinline__ int count() const { return head + tail; }
    __device__ __forceinline__ int at(int i) const { return i < head ? i : from + (i - head); }
};
__device__ __forceinline__ Steps steps_of(int pa, int pb, int window, int sinks, int room)
{
    if (pb < 0) return Steps{0, 0, 0};
    const int last = min(pb / kStep + 1, room);
    if (window == 0) return Steps{0, 0, last};
    const int from = min(max((int)((int64_t)pa - window + 1 < 0 ? 0 : pa - window + 1), 0) / kStep, last);
    const int head = min((int)(((int64_t)min(sinks, pb + 1) + kStep - 1) / kStep), from);
    return Steps{head, from, last - from};
}

// A row tile's sequence, rows and steps.  Rows are a sequence's (new token, head of the group) pairs.
struct Tile {
    Span sp;
    int rows, pa, pb;                            // rows of the tile that exist; positions of the first and the last
    Steps st;
};
__device__ __forceinline__ Tile tile_of(const Attend &at, int b, int r0, int height)
{
    Tile t;
    t.sp = span_of(at.sq, at.T, b);
    const int64_t R = (int64_t)t.sp.n * at.G;
    t.rows = (int)min(max(R - r0, (int64_t)0), (int64_t)height);
    t.pa = t.sp.p0 + r0 / at.G;
    t.pb = t.sp.p0 + (r0 + t.rows - 1) / at.G;
    t.st = t.rows > 0 ? steps_of(t.pa, t.pb, at.window, at.sinks, at.room) : Steps{0, 0, 0};
    return t;
}

// Which of the tokens j0 .. j0 + 63 position p sees, a bit each (p < 0: none).
__device__ __forceinline__ unsigned long long seen_of(int p, int j0, int window, int sinks)
{
    auto upto = [](int x) { return x < 0 ? 0ull : x >= 63 ? ~0ull : (2ull << x) - 1; };
    const int reach = p - j0;                    // (p < 0 comes with j0 >= 0)
    unsigned long long seen = p < 0 ? 0ull : upto(reach);
    if (window > 0) seen &= ~upto(max(reach, -1) - window) | upto(sinks - j0 - 1);
    return seen;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_(float x) { return __builtin_amdgcn_logf(x); }

// A scale within the normal numbers: where no token is visible a page's may be anything, and nothing may come of it that is
// no number (a visible token's is positive and finite; 0 times the call's scale counts as 10^-37).
__device__ __forceinline__ float usable(float s) { return fminf(fmaxf(s, 1e-37f), 1e37f); }

// Maximum over lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_rows(float v)
{
    float a = v, b = v;
    swap32(a, b);
    a = fmaxf(a, b);
    b = a;
    swap16(a, b);
    return fmaxf(a, b);
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const half2_t h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
}

// Two weights, each as the sum of two fp16 numbers: x the nearest ones, y what these leave off.  (minus: -1, in a register that the
// compiler cannot see through, so that a weight less its fp16 number is one fma that takes the half as it lies.)
__device__ __forceinline__ float minus_one()
{
    float x = -1.f;
    asm("" : "+v"(x));
    return x;
}
__device__ __forceinline__ uint2 split2(float a, float b, float minus)
{
    uint32_t hi = pack2(a, b);
    asm("" : "+v"(hi));
    return make_uint2(hi, pack2(fmaf(h2f((uint16_t)hi), minus, a), fmaf(h2f((uint16_t)(hi >> 16)), minus, b)));
}

// Four results of a row: its sum over its denominator; 0 for a row that saw nothing (its sum is 0, too).
template <int FMT>
__device__ __forceinline__ void store_row(uint16_t *y, const float4_t &v, float den)
{
    const float n = den == 0.f ? 0.f : kCodeUnit<FMT> / den;
    *reinterpret_cast<uint2 *>(y) = make_uint2(pack2(v[0] * n, v[1] * n), pack2(v[2] * n, v[3] * n));
}

// How a call is cut: row tiles of `height` rows, `tiles` of them for a sequence at most, and a tile's steps (at most) into
// splits of chunk steps.  tall: k_attend_tall's tiles; pair: with two groups of waves each, which take the steps in turn.
struct AttendPlan {
    int height, tiles, splits, chunk;
    bool tall, pair;
};

// tri_attend_tall.hip: rows of a tile, and the launch.
constexpr int kTallRows = 128;
void launch_attend_tall(const Attend &at, const AttendPlan &p, float *part, hipStream_t s);

}  // namespace tri
