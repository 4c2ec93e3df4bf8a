// tri_api.hip -- the extern "C" entry points of libtri: argument checks and dispatch.
// Every check runs on the host before any launch; see include/tri.h for the contract.
#include "tri_internal.h"

using namespace tri;
static_assert(TRI_MAX_GROUPS == kMaxGroups, "group table size");

namespace {

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool misaligned_to(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
bool known_group(int group) { return group == 32 || group == 64 || group == 128; }
bool known_fmt(int fmt) { return fmt == TRI_FMT_2BIT || fmt == TRI_FMT_1P6BIT; }
constexpr int64_t kMaxDim = (int64_t)1 << 31;   // K, N and one packed row are indexed with 32-bit ints

int check_pack(const void *W, int64_t N, int64_t K, const void *Wp)
{
    if (!W || !Wp || N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim) return TRI_EINVAL;
    if (misaligned(Wp)) return TRI_EALIGN;
    return TRI_OK;
}

int check_linear(const void *X, const void *Wp, int64_t M, int64_t N, int64_t K, int fmt, const void *Y)
{
    if (!X || !Wp || !Y || M < 1 || N < 1 || K < 1 || !known_fmt(fmt)) return TRI_EINVAL;
    if (N >= kMaxDim || K >= kMaxDim || M >= kMaxDim) return TRI_EINVAL;
    if (misaligned(X) || misaligned(Wp) || misaligned(Y)) return TRI_EALIGN;
    return TRI_OK;
}

// The kernel family for a shape.  Up to 16 rows, the small-M kernels (at M = 1 the MFMA kernel
// beats the VALU GEMV).  Above, the small-M kernels take one pass over the weights per 16-row
// slice of X, while the GEMM's parallelism comes from its output tiles alone, so with few tiles
// most CUs idle.  Both costs per unit of K, from fits to measured times on MI355X (M = 17 .. 768;
// K x N = 4096 x 4096, 4096 x 11008, 11008 x 4096, 8192 x 28672, 28672 x 8192; both formats):
//   small-M  ceil(M/16) * N * c,  c = 0.10 ps (2-bit) / 0.127 ps (1.6-bit) per trit and slice;
//            rows past eight steps per wave 1.6x / 1.2x that, rows past sixteen (the streaming
//            kernel) 5x / 1.9x;
//   GEMM     with T64 = ceil(M/64) * ceil(N/512) tiles of 64 rows: at most 64 of them, one round
//            of 64 x 128 workgroups, 4.8 ns (2-bit) / 6.3 ns (1.6-bit); at most 128, 8.8 / 10.7
//            ns; beyond, u * R with u = 13 / 16 ns per round of 128 x 256 workgroups and R the
//            rounds of the launch of 128-row tiles (a last round of at most 128 tiles runs at half
//            width).
int select_algo(int64_t M, int64_t N, int64_t K, int fmt)
{
    if (M <= 16) return TRI_ALGO_SMALLM;
    const int64_t cus = cu_count();
    const bool two = fmt == TRI_FMT_2BIT;
    double c = two ? 0.10 : 0.127;               // ps
    if (K > (two ? 32768 : 35840)) c *= two ? 5.0 : 1.9;
    else if (K > (two ? 16384 : 20480)) c *= two ? 1.6 : 1.2;
    const int64_t tn = (N + 511) / 512;
    const int64_t T64 = ((M + 63) / 64) * tn, T = ((M + 127) / 128) * tn;
    const int64_t r = T % cus;
    const int64_t R = (r > 0 && r <= cus / 2) ? 2 * (T / cus) + 1 : 2 * ((T + cus - 1) / cus);
    const double small = (double)((M + 15) / 16) * (double)N * c;
    const double gemm = T64 <= cus / 4 ? (two ? 4800.0 : 6300.0)
                      : T64 <= cus / 2 ? (two ? 8800.0 : 10700.0)
                                        : (two ? 13000.0 : 16000.0) * (double)R;
    return small < gemm ? TRI_ALGO_SMALLM : TRI_ALGO_GEMM;
}

int run_linear(const _Float16 *X, const uint8_t *Wp, float scale, int64_t M, int64_t N, int64_t K, int fmt,
               _Float16 *Y, int algo, hipStream_t s)
{
    const uint16_t *x = reinterpret_cast<const uint16_t *>(X);
    uint16_t *y = reinterpret_cast<uint16_t *>(Y);
    switch (algo) {
    case TRI_ALGO_GEMV:
        if (M != 1 || fmt != TRI_FMT_2BIT) return TRI_EINVAL;
        return launch_gemv2(x, Wp, scale, (int)N, (int)K, y, s);
    case TRI_ALGO_SMALLM:
        if (M > 16) {
            // one launch over 16-row slices of X where the batched kernel serves the shape,
            // else one small-M call per slice
            int n = (int)N;
            const Groups gr = make_groups(1, &Wp, &scale, &n, &y);
            if (launch_mvm(x, gr, (int)M, (int)K, fmt, s)) return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
            for (int64_t m0 = 0; m0 < M; m0 += 16) {
                const int64_t mm = (M - m0) < 16 ? (M - m0) : 16;
                const int rc = run_linear(X + m0 * K, Wp, scale, mm, N, K, fmt, Y + m0 * N, TRI_ALGO_SMALLM, s);
                if (rc != TRI_OK) return rc;
            }
            return TRI_OK;
        }
        if (launch_decode(x, Wp, scale, (int)M, (int)N, (int)K, fmt, y, s))
            return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
        return launch_smallm(x, Wp, scale, (int)M, (int)N, (int)K, fmt, y, s);   // long rows: streaming variant
    case TRI_ALGO_GEMM:
        return launch_gemm(x, Wp, scale, M, (int)N, (int)K, fmt, y, s);
    default:
        return TRI_EINVAL;
    }
}

int run_experts(const _Float16 *X, int64_t T, const int32_t *offsets, const int32_t *rows, int64_t R, const uint8_t *Wp,
                const float *scale, const uint8_t *Wp_up, const float *scale_up, bool pair, int E, int64_t N, int64_t K,
                int fmt, _Float16 *Y, hipStream_t s)
{
    if (!X || !offsets || !Wp || !scale || !Y || (pair && (!Wp_up || !scale_up)) || !known_fmt(fmt)) return TRI_EINVAL;
    if (T < 1 || R < 1 || N < 1 || K < 1 || T >= kMaxDim || R >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
        return TRI_EINVAL;
    if (E < 1 || E > TRI_MAX_EXPERTS || (!rows && T < R)) return TRI_EINVAL;
    // a workgroup of 512 threads per 16 outputs, fewer than 2^32 threads in a row of the grid; 32-bit offsets in a block of rows
    if (N > kMaxDim / 16 - 16 || K >= kMaxDim / 32) return TRI_EINVAL;
    if (rows && T > (((int64_t)1 << 31) - 8) / K) return TRI_EINVAL;   // gathered rows: 32-bit buffer offsets
    if (misaligned(X) || misaligned(Wp) || misaligned(Wp_up) || misaligned(Y)) return TRI_EALIGN;
    if (misaligned_to(offsets, 4) || misaligned_to(rows, 4) || misaligned_to(scale, 4) || misaligned_to(scale_up, 4))
        return TRI_EALIGN;
    Experts ex{};
    ex.X = reinterpret_cast<const uint16_t *>(X);
    ex.offsets = offsets;
    ex.rows = rows;
    ex.Wp[0] = Wp;
    ex.Wp[1] = Wp_up;
    ex.scale[0] = scale;
    ex.scale[1] = scale_up;
    ex.Y = reinterpret_cast<uint16_t *>(Y);
    ex.T = (int)T;
    ex.R = (int)R;
    ex.E = E;
    ex.N = (int)N;
    ex.K = (int)K;
    return launch_experts(ex, fmt, s);
}

}  // namespace

int tri::cu_count()
{
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (dev >= 0 && dev < kMaxDevices) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) return 256;
    if (dev >= 0 && dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

extern "C" {

int64_t tri_row_bytes(int64_t K, int fmt) { return row_bytes(K, fmt); }

int64_t tri_quantize_workspace_bytes(int64_t N, int64_t K)
{
    if (N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim) return -1;
    return quant_workspace_bytes(N * K);
}

int tri_quantize(const float *W, int64_t N, int64_t K, int fmt, uint8_t *Wp, float *scale_out, void *workspace,
                 int64_t workspace_bytes, hipStream_t stream)
{
    if (!W || !Wp || !scale_out || !workspace || !known_fmt(fmt)) return TRI_EINVAL;
    if (N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim) return TRI_EINVAL;
    if (workspace_bytes < quant_workspace_bytes(N * K)) return TRI_EINVAL;
    if (misaligned(W) || misaligned(Wp) || misaligned(workspace) || (reinterpret_cast<uintptr_t>(scale_out) & 3u))
        return TRI_EALIGN;
    return launch_quantize(W, N, K, fmt, Wp, scale_out, workspace, stream);
}

int tri_quantize_noalloc(const float *W, int64_t N, int64_t K, int fmt, uint8_t *Wp, float *scale_out,
                         hipStream_t stream)
{
    if (!W || !Wp || !scale_out || !known_fmt(fmt)) return TRI_EINVAL;
    if (N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim) return TRI_EINVAL;
    if (quant_workspace_bytes(N * K) > quant_scratch_bytes()) return TRI_EINVAL;
    if (misaligned(W) || misaligned(Wp) || (reinterpret_cast<uintptr_t>(scale_out) & 3u)) return TRI_EALIGN;
    void *ws = quant_scratch();
    if (!ws) return TRI_EHIP;
    return launch_quantize(W, N, K, fmt, Wp, scale_out, ws, stream);
}

int tri_pack2(const int8_t *W, int64_t N, int64_t K, uint8_t *Wp, hipStream_t stream)
{
    const int rc = check_pack(W, N, K, Wp);
    return rc != TRI_OK ? rc : launch_pack(W, N, K, TRI_FMT_2BIT, Wp, stream);
}

int tri_pack16(const int8_t *W, int64_t N, int64_t K, uint8_t *Wp, hipStream_t stream)
{
    const int rc = check_pack(W, N, K, Wp);
    return rc != TRI_OK ? rc : launch_pack(W, N, K, TRI_FMT_1P6BIT, Wp, stream);
}

int tri_unpack(const uint8_t *Wp, int64_t N, int64_t K, int fmt, int8_t *W, hipStream_t stream)
{
    if (!known_fmt(fmt)) return TRI_EINVAL;
    const int rc = check_pack(W, N, K, Wp);
    return rc != TRI_OK ? rc : launch_unpack(Wp, N, K, fmt, W, stream);
}

int tri_select_algo(int64_t M, int64_t N, int64_t K, int fmt)
{
    if (M < 1 || N < 1 || K < 1 || !known_fmt(fmt) || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return TRI_EINVAL;
    return select_algo(M, N, K, fmt);
}

int tri_linear(const _Float16 *X, const uint8_t *Wp, float scale, int64_t M, int64_t N, int64_t K, int fmt,
               _Float16 *Y, hipStream_t stream)
{
    const int rc = check_linear(X, Wp, M, N, K, fmt, Y);
    return rc != TRI_OK ? rc : run_linear(X, Wp, scale, M, N, K, fmt, Y, select_algo(M, N, K, fmt), stream);
}

int tri_linear_algo(const _Float16 *X, const uint8_t *Wp, float scale, int64_t M, int64_t N, int64_t K, int fmt,
                    _Float16 *Y, int algo, hipStream_t stream)
{
    const int rc = check_linear(X, Wp, M, N, K, fmt, Y);
    if (rc != TRI_OK) return rc;
    if (algo == TRI_ALGO_AUTO) algo = select_algo(M, N, K, fmt);
    return run_linear(X, Wp, scale, M, N, K, fmt, Y, algo, stream);
}

int tri_linear_grouped(const _Float16 *X, const uint8_t *const *Wp, const float *scale, int64_t M, const int64_t *N,
                       int64_t K, int fmt, _Float16 *const *Y, int G, hipStream_t stream)
{
    if (!Wp || !scale || !N || !Y || G < 1 || G > TRI_MAX_GROUPS) return TRI_EINVAL;
    for (int g = 0; g < G; ++g) {
        const int rc = check_linear(X, Wp[g], M, N[g], K, fmt, Y[g]);
        if (rc != TRI_OK) return rc;
    }
    int64_t blocks = 0;
    for (int g = 0; g < G; ++g) blocks += (N[g] + 15) / 16;
    if (blocks >= ((int64_t)1 << 31)) return TRI_EINVAL;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(X);
    bool small = true;                           // every matrix on the small-M kernels
    for (int g = 0; g < G; ++g) small = small && select_algo(M, N[g], K, fmt) == TRI_ALGO_SMALLM;
    if (small) {
        int n[kMaxGroups];
        uint16_t *y[kMaxGroups];
        for (int g = 0; g < G; ++g) {
            n[g] = (int)N[g];
            y[g] = reinterpret_cast<uint16_t *>(Y[g]);
        }
        const Groups gr = make_groups(G, Wp, scale, n, y);
        const bool done = M == 1 ? launch_mv1(x, gr, (int)K, fmt, stream)
                          : (M <= 4 && launch_mvr(x, gr, (int)M, (int)K, fmt, stream)) ||
                                launch_mvm(x, gr, (int)M, (int)K, fmt, stream);
        if (done) return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
    }
    // shapes outside the grouped kernels' range: one call per matrix
    for (int g = 0; g < G; ++g) {
        const int rc = run_linear(X, Wp[g], scale[g], M, N[g], K, fmt, Y[g], select_algo(M, N[g], K, fmt), stream);
        if (rc != TRI_OK) return rc;
    }
    return TRI_OK;
}

int tri_linear_fused(const _Float16 *X, const uint8_t *const *Wp, const float *scale, int64_t M, const int64_t *N,
                     int64_t K, int fmt, _Float16 *const *Y, int G, const tri_glue *glue, hipStream_t stream)
{
    if (!glue || !Wp || !scale || !N || !Y || G < 1 || G > TRI_MAX_GROUPS) return TRI_EINVAL;
    const bool pair = glue->pair != 0;
    if (pair && (G != 2 || N[0] != N[1])) return TRI_EINVAL;
    for (int g = 0; g < G; ++g) {
        const int rc = check_linear(X, Wp[g], M, N[g], K, fmt, (pair && g == 1) ? Y[0] : Y[g]);
        if (rc != TRI_OK) return rc;
    }
    if (M > 16 || (K % 8) != 0) return TRI_EINVAL;
    if ((glue->norm || pair) && K > (fmt == TRI_FMT_2BIT ? 16384 : 20480)) return TRI_EINVAL;
    int64_t blocks = 0;
    for (int g = 0; g < G; ++g) blocks += (N[g] + 15) / 16;
    if (blocks >= ((int64_t)1 << 31)) return TRI_EINVAL;
    if (glue->norm && !(glue->norm_eps >= 0.f && glue->norm_eps <= 3.4e38f)) return TRI_EINVAL;   // (NaN fails)
    if (misaligned(glue->norm_gain)) return TRI_EALIGN;
    Fusion fu{};
    fu.gain = glue->norm ? reinterpret_cast<const uint16_t *>(glue->norm_gain) : nullptr;
    fu.norm = glue->norm ? 1 : 0;
    fu.eps = glue->norm_eps;
    fu.pair = pair ? 1 : 0;
    for (int g = 0; g < G; ++g) {
        const _Float16 *r = glue->residual ? glue->residual[g] : nullptr;
        if (pair && g == 1 && r) return TRI_EINVAL;
        if (misaligned(r)) return TRI_EALIGN;
        fu.res[g] = reinterpret_cast<const uint16_t *>(r);
    }
    int n[kMaxGroups];
    uint16_t *y[kMaxGroups];
    for (int g = 0; g < G; ++g) {
        n[g] = (int)N[g];
        y[g] = reinterpret_cast<uint16_t *>(Y[g]);
    }
    Groups gr = make_groups(G, Wp, scale, n, y);
    if (pair) gr.blk[2] = gr.blk[1];            // the grid covers matrix 0's rows; each workgroup reads both
    const uint16_t *x = reinterpret_cast<const uint16_t *>(X);
    const bool done =
        M == 1 ? launch_mv1(x, gr, (int)K, fmt, stream, &fu)
               : (M <= 4 && launch_mvr(x, gr, (int)M, (int)K, fmt, stream, &fu)) ||
                     launch_mvm(x, gr, (int)M, (int)K, fmt, stream, &fu);
    if (!done) return TRI_EINVAL;                // a shape the glue variants do not serve
    return hipGetLastError() == hipSuccess ? TRI_OK : TRI_EHIP;
}

int64_t tri_int4_bytes(int64_t N, int64_t K, int group, int zeros)
{
    if (N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim || !known_group(group)) return -1;
    return int4_bytes(N, K, group, zeros != 0);
}

int tri_int4_pack(const uint8_t *Q, const _Float16 *S, const uint8_t *Z, int64_t N, int64_t K, int group, uint8_t *Wp,
                  hipStream_t stream)
{
    if (!Q || !S || !Wp || tri_int4_bytes(N, K, group, Z != nullptr) < 0) return TRI_EINVAL;
    if (misaligned(Wp) || misaligned_to(S, 2)) return TRI_EALIGN;
    return launch_int4_pack(Q, reinterpret_cast<const uint16_t *>(S), Z, (int)N, (int)K, group, Wp, stream);
}

int tri_int4_unpack(const uint8_t *Wp, int64_t N, int64_t K, int group, int zeros, uint8_t *Q, _Float16 *S, uint8_t *Z,
                    hipStream_t stream)
{
    if (!Wp || !Q || !S || (zeros && !Z) || tri_int4_bytes(N, K, group, zeros) < 0) return TRI_EINVAL;
    if (misaligned(Wp) || misaligned_to(S, 2)) return TRI_EALIGN;
    return launch_int4_unpack(Wp, (int)N, (int)K, group, zeros != 0, Q, reinterpret_cast<uint16_t *>(S), Z, stream);
}

int tri_int4_quantize(const float *W, int64_t N, int64_t K, int group, int zeros, uint8_t *Wp, hipStream_t stream)
{
    if (!W || !Wp || tri_int4_bytes(N, K, group, zeros) < 0) return TRI_EINVAL;
    if (misaligned(Wp) || misaligned_to(W, 4)) return TRI_EALIGN;
    return launch_int4_quantize(W, (int)N, (int)K, group, zeros != 0, Wp, stream);
}

int tri_int4_linear(const _Float16 *X, const uint8_t *Wp, int64_t M, int64_t N, int64_t K, int group, int zeros,
                    const _Float16 *residual, _Float16 *Y, hipStream_t stream)
{
    if (!X || !Wp || !Y || M < 1 || M >= kMaxDim || tri_int4_bytes(N, K, group, zeros) < 0) return TRI_EINVAL;
    if (misaligned(X) || misaligned(Wp) || misaligned(residual) || misaligned(Y)) return TRI_EALIGN;
    return launch_int4_linear(reinterpret_cast<const uint16_t *>(X), Wp, (int)M, (int)N, (int)K, group, zeros != 0,
                              reinterpret_cast<const uint16_t *>(residual), reinterpret_cast<uint16_t *>(Y), stream);
}

int64_t tri_experts_route_workspace_bytes(int64_t T, int E, int topk)
{
    if (T < 1 || E < 1 || E > TRI_MAX_EXPERTS || topk < 1 || topk > E || topk > TRI_MAX_TOPK || T >= kMaxDim / 16 ||
        T * topk >= kMaxDim)
        return -1;
    return route_workspace_bytes(T, E, topk);
}

int tri_experts_route(const void *logits, int dtype, int64_t T, int E, int topk, int renorm, int32_t *ids,
                      float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                      int64_t workspace_bytes, hipStream_t stream)
{
    const int64_t need = tri_experts_route_workspace_bytes(T, E, topk);
    if (need < 0 || (dtype != TRI_F16 && dtype != TRI_F32)) return TRI_EINVAL;
    if (!logits || !ids || !weights || !offsets || !rows || !pos) return TRI_EINVAL;
    if (need > 0 && (!workspace || workspace_bytes < need)) return TRI_EINVAL;
    if (misaligned_to(logits, dtype == TRI_F16 ? 2 : 4) || misaligned_to(ids, 4) || misaligned_to(weights, 4) ||
        misaligned_to(offsets, 4) || misaligned_to(rows, 4) || misaligned_to(pos, 4) || misaligned(workspace))
        return TRI_EALIGN;
    return launch_route(logits, dtype == TRI_F16, (int)T, E, topk, renorm != 0, ids, weights, offsets, rows, pos,
                        workspace, stream);
}

int tri_experts_linear(const _Float16 *X, int64_t T, const int32_t *offsets, const int32_t *rows, int64_t R,
                       const uint8_t *Wp, const float *scale, int E, int64_t N, int64_t K, int fmt, _Float16 *Y,
                       hipStream_t stream)
{
    return run_experts(X, T, offsets, rows, R, Wp, scale, nullptr, nullptr, false, E, N, K, fmt, Y, stream);
}

int tri_experts_pair(const _Float16 *X, int64_t T, const int32_t *offsets, const int32_t *rows, int64_t R,
                     const uint8_t *Wp, const float *scale, const uint8_t *Wp_up, const float *scale_up, int E,
                     int64_t N, int64_t K, int fmt, _Float16 *Y, hipStream_t stream)
{
    return run_experts(X, T, offsets, rows, R, Wp, scale, Wp_up, scale_up, true, E, N, K, fmt, Y, stream);
}

int tri_experts_combine(const _Float16 *Z, int64_t R, const int32_t *pos, const float *weights,
                        const _Float16 *residual, int64_t T, int topk, int64_t N, _Float16 *Y, hipStream_t stream)
{
    if (!Z || !pos || !weights || !Y || R < 1 || T < 1 || N < 1 || topk < 1 || topk > TRI_MAX_TOPK) return TRI_EINVAL;
    if (R >= kMaxDim || T >= kMaxDim || N >= kMaxDim) return TRI_EINVAL;
    if (misaligned(Z) || misaligned(residual) || misaligned(Y) || misaligned_to(pos, 4) || misaligned_to(weights, 4))
        return TRI_EALIGN;
    return launch_combine(reinterpret_cast<const uint16_t *>(Z), R, pos, weights,
                          reinterpret_cast<const uint16_t *>(residual), (int)T, topk, (int)N,
                          reinterpret_cast<uint16_t *>(Y), stream);
}

const char *tri_status_string(int code)
{
    switch (code) {
    case TRI_OK: return "ok";
    case TRI_EINVAL: return "invalid argument";
    case TRI_EALIGN: return "pointer not 16-byte aligned";
    case TRI_EHIP: return "HIP launch error";
    default: return "unknown status";
    }
}

int tri_probe_read(const void *src, int64_t bytes, uint32_t *sink, hipStream_t stream)
{
    if (!src || !sink || bytes < 16 || (bytes % 16) != 0) return TRI_EINVAL;
    if (misaligned(src)) return TRI_EALIGN;
    return launch_probe_read(src, bytes, sink, stream);
}

int tri_probe_copy(const void *src, void *dst, int64_t bytes, hipStream_t stream)
{
    if (!src || !dst || bytes < 16 || (bytes % 16) != 0) return TRI_EINVAL;
    if (misaligned(src) || misaligned(dst)) return TRI_EALIGN;
    return launch_probe_copy(src, dst, bytes, stream);
}

int tri_probe_empty(int64_t workgroups, int threads, uint32_t *sink, hipStream_t stream)
{
    if (!sink || workgroups < 1 || workgroups >= kMaxDim || threads < 64 || threads > 1024 || (threads % 64) != 0)
        return TRI_EINVAL;
    return launch_probe_empty(workgroups, threads, sink, stream);
}

int tri_probe_rows(const _Float16 *X, const uint8_t *Wp, int64_t N, int64_t K, int fmt, int waves, _Float16 *Y,
                   hipStream_t stream)
{
    if (!X || !Wp || !Y || N < 1 || K < 1 || N >= kMaxDim || K >= kMaxDim || !known_fmt(fmt)) return TRI_EINVAL;
    if (waves != 4 && waves != 8) return TRI_EINVAL;
    if ((row_bytes(K, fmt) / 16 + 4 * waves - 1) / (4 * waves) > 8 || N * row_bytes(K, fmt) >= kMaxDim)
        return TRI_EINVAL;
    if (misaligned(X) || misaligned(Wp)) return TRI_EALIGN;
    return launch_probe_rows(reinterpret_cast<const uint16_t *>(X), Wp, (int)N, (int)K, fmt, waves,
                             reinterpret_cast<uint16_t *>(Y), stream);
}

int tri_probe_stream(const void *src, int64_t bytes, int workgroups, int unroll, uint32_t *sink, hipStream_t stream)
{
    if (!src || !sink || bytes < 16 || (bytes % 16) != 0 || bytes >= kMaxDim || workgroups < 1) return TRI_EINVAL;
    if (unroll != 1 && unroll != 2 && unroll != 4 && unroll != 8) return TRI_EINVAL;
    if (misaligned(src)) return TRI_EALIGN;
    return launch_probe_stream(src, bytes, workgroups, unroll, sink, stream);
}

}  // extern "C"
