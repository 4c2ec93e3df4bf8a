/*
 * tri.h -- C ABI of libtri, the gfx950 (MI355X) ternary linear layer.
 *
 * The layer (Pith review of "Spectra 1.1: Scaling Laws and Efficient Inference
 * for Ternary Language Models", section "What carries the argument"): a weight
 * matrix W with entries in {-1, 0, +1} times one shared floating-point scale,
 * applied to fp16 activations,
 *
 *     Y[m][n] = fp16_rne( scale * sum_k W[n][k] * X[m][k] ),   accumulated in fp32.
 *
 * Weights are stored losslessly in one of two packings (same review, "Core
 * claim" and "What carries the argument": 2^p > 3^k, so 5 trits fit in 8 bits):
 *
 *   TRI_FMT_2BIT    base-4: byte = sum_{j<4} (t[4b+j] + 1) * 4^j
 *                   (trit 4b+j in bits 2j..2j+1; digit 3 never produced)
 *   TRI_FMT_1P6BIT  base-3: byte = sum_{j<5} (t[5b+j] + 1) * 3^j   (0..242)
 *
 * Layout of a packed matrix: N rows (output features) one after another, each
 * tri_row_bytes(K, fmt) bytes long; a row is padded with zero trits to a
 * multiple of 64 trits (2-bit) or 80 trits (1.6-bit), so every row is a whole
 * number of 16-byte chunks and starts 16-byte aligned.
 *
 * Conventions for every call:
 *  - All array pointers are DEVICE pointers owned by the caller.  The library
 *    allocates no memory.  The only state it keeps is, per device, the compute
 *    unit count and the resident workgroups of a few kernel variants, each
 *    queried from the HIP runtime once and never changed; calls are thread-safe
 *    and deterministic (no atomics; the reduction order is fixed).
 *  - Work is enqueued asynchronously on `stream` (0 = the null stream).  A
 *    device fault surfaces at the caller's next synchronisation.
 *  - Argument checks run on the host before anything is launched; on failure
 *    nothing is launched and a negative status is returned.
 *  - Outputs must not alias inputs.
 */
#ifndef TRI_H
#define TRI_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { TRI_FMT_2BIT = 0, TRI_FMT_1P6BIT = 1 };

enum {
    TRI_OK = 0,
    TRI_EINVAL = -1,   /* a size < 1 (or too large), a null pointer, an unknown format or algorithm */
    TRI_EALIGN = -2,   /* a pointer that must be 16-byte aligned is not */
    TRI_EHIP = -3      /* the HIP runtime reported an error at launch */
};

/* Kernel families of tri_linear (see tri_linear_algo). */
enum {
    TRI_ALGO_AUTO = 0,     /* pick from (M, fmt): the default of tri_linear */
    TRI_ALGO_GEMV = 1,     /* M == 1, 2-bit only: VALU dot products, lanes own K-slices */
    TRI_ALGO_SMALLM = 2,   /* any M, in 16-row slices of X: MFMA 16x16x32 f16 with trits decoded
                              in registers, one pass over the weights per slice (the choice up to
                              M = 16, M = 1 included, and above while the GEMM has too few tiles
                              to fill the chip) */
    TRI_ALGO_GEMM = 3      /* any M: tiled MFMA 32x32x16 f16 GEMM, activations staged in LDS and
                              trits decoded in registers (prefill) */
};

/* Bytes of one packed row of K trits: 16*ceil(K/64) (2-bit) or 16*ceil(K/80)
 * (1.6-bit).  The densities are the pages' (Pith review, "Core claim": base-4 and
 * base-3 encodings; "What carries the argument": 5 trits in 8 bits since
 * 3^5 < 2^8); the row padding is this library's reading of a layout the pages
 * leave open: every row is padded with zero trits to whole 16-byte chunks (64
 * trits in 2-bit, 80 in 1.6-bit), so a row starts 16-byte aligned and is read
 * with 16-byte loads.  At K a multiple of 64 the 2-bit row is exactly K/4 bytes;
 * a 1.6-bit row exceeds ceil(K/5) by at most 15 bytes.
 * Returns -1 if K < 1 or fmt is unknown; pure host arithmetic, launches nothing. */
int64_t tri_row_bytes(int64_t K, int fmt);

/* 2-bit packing (Pith review, "Core claim": base-4 encoding).
 * W: N*K int8, row-major (row n = output feature n).  Any int8 is accepted and
 * sign(w) is encoded.  Wp: N*tri_row_bytes(K, TRI_FMT_2BIT) bytes, 16-byte aligned.
 * Errors: TRI_EINVAL (N < 1, K < 1, null), TRI_EALIGN (Wp), TRI_EHIP. */
int tri_pack2(const int8_t *W, int64_t N, int64_t K, uint8_t *Wp, hipStream_t stream);

/* 1.6-bit packing (Pith review, "What carries the argument": 3^5 = 243 < 2^8,
 * 1.6 bits per weight; "Core claim": base-3 encoding).  Same arguments as
 * tri_pack2 with rows of tri_row_bytes(K, TRI_FMT_1P6BIT) bytes. */
int tri_pack16(const int8_t *W, int64_t N, int64_t K, uint8_t *Wp, hipStream_t stream);

/* Unpack (Pith review, "Significance": the packing correctness theorem of the
 * paper's Appendix E; "Referee Report" minor comment 5: the 1.6-bit decode is
 * the repeated-division sequence b'_i -> x_i).  Defined for every byte value:
 * a 2-bit code 3 gives 0, and 1.6-bit bytes 243..255 go through the same
 * repeated division by 3 (five digits).  Writes the first K trits of each row.
 * Wp: N rows of tri_row_bytes(K, fmt) bytes, 16-byte aligned; W: N*K int8.
 * Errors: TRI_EINVAL, TRI_EALIGN (Wp), TRI_EHIP. */
int tri_unpack(const uint8_t *Wp, int64_t N, int64_t K, int fmt, int8_t *W, hipStream_t stream);

/* Workspace (device bytes, a multiple of 8) that tri_quantize needs for an N x K
 * matrix; -1 if N or K is < 1 or >= 2^31.  It depends on N*K only. */
int64_t tri_quantize_workspace_bytes(int64_t N, int64_t K);

/* Quantise latent full-precision weights to trits and one scale, and pack them
 * (Pith review, "What carries the argument": latent full-precision weights rounded
 * on the fly to {-1,0,1} times one shared scale; the review's domain assumptions:
 * round-to-nearest).  The pages do not give the scale rule; the one taken is
 *     scale = float32( sum_{n,k} |W[n][k]| / (N*K) )   (summed in float64),
 *     t     = round_half_to_even(W / scale) clipped to [-1, 1]; 0 when scale == 0,
 * so a weight becomes sign(w) exactly when 2|w| > scale, ties giving 0.
 * W: N*K float32 row-major, 16-byte aligned, finite (non-finite weights give an
 * unspecified scale and trits).  Wp: N*tri_row_bytes(K, fmt) bytes, 16-byte
 * aligned, written as tri_pack2 / tri_pack16 would pack the trits.  scale_out: one
 * float, 4-byte aligned, written on the stream (read it after synchronising).
 * workspace: at least tri_quantize_workspace_bytes(N, K) bytes, 16-byte aligned,
 * owned by the caller, overwritten; calls that share a workspace must be ordered
 * on one stream.  W must not alias Wp, scale_out or workspace.
 * Errors: TRI_EINVAL (a size < 1 or >= 2^31, null, unknown fmt, workspace too
 * small), TRI_EALIGN, TRI_EHIP. */
int tri_quantize(const float *W, int64_t N, int64_t K, int fmt, uint8_t *Wp, float *scale_out,
                 void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* tri_quantize for callers that cannot allocate device memory or pass a workspace
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same launches and results, with the partial sums kept in a
 * static device array of the library (16 KB per device, TRI_QUANTIZE_SCRATCH_BYTES,
 * held until the process ends), so the call allocates nothing.  The array is
 * enough for every N x K (at most 2048 partial sums); a matrix needing more is
 * rejected with TRI_EINVAL.  Every call on one device shares that device's array
 * and overwrites it (nothing in it needs to start at zero): calls that may overlap
 * on one device (several streams, several threads) race and must be ordered by the
 * caller.  Arguments and errors as tri_quantize without the workspace; TRI_EHIP also
 * if the array's device address cannot be obtained. */
enum { TRI_QUANTIZE_SCRATCH_BYTES = 16384 };
int tri_quantize_noalloc(const float *W, int64_t N, int64_t K, int fmt, uint8_t *Wp, float *scale_out,
                         hipStream_t stream);

/* The ternary linear layer (Pith review, "What carries the argument"):
 *   Y[m][n] = fp16_rne(scale * sum_k t[n][k] * X[m][k]), fp32 accumulation.
 * X: M*K fp16 row-major (row stride K); Wp: packed weights as above; Y: M*N fp16
 * row-major.  X, Wp and Y must be 16-byte aligned.  scale is any finite fp32.
 * Wp must hold bytes produced by tri_pack2 / tri_pack16 for this K (2-bit code
 * 3 and 1.6-bit bytes above 242 give unspecified, finite results).  X is
 * expected finite (a non-finite x may give NaN in every output it touches).
 * Errors: TRI_EINVAL (a size < 1, K or N >= 2^31, null, unknown fmt),
 * TRI_EALIGN, TRI_EHIP. */
int tri_linear(const _Float16 *X, const uint8_t *Wp, float scale,
               int64_t M, int64_t N, int64_t K, int fmt, _Float16 *Y, hipStream_t stream);

/* tri_linear with the kernel family chosen by the caller (for measurement and
 * tests).  TRI_ALGO_GEMV needs M == 1 and TRI_FMT_2BIT, else TRI_EINVAL.  Results of every family satisfy the same
 * error bound; they are not bitwise equal to one another. */
int tri_linear_algo(const _Float16 *X, const uint8_t *Wp, float scale,
                    int64_t M, int64_t N, int64_t K, int fmt, _Float16 *Y,
                    int algo, hipStream_t stream);

/* Several ternary linear layers that read the same activations, in one launch (for
 * example the Q, K and V projections of a block, or its gate and up projections): for
 * g < G,  Y[g] = fp16_rne(scale[g] * X W_g^T)  with W_g of N[g] rows packed for this K and
 * fmt, exactly as tri_linear would compute each one.  Wp, scale, N and Y are HOST arrays of
 * G entries (the pointers they hold are device pointers, with tri_linear's alignment and
 * aliasing rules); 1 <= G <= TRI_MAX_GROUPS.  Where tri_linear would pick TRI_ALGO_SMALLM for
 * every matrix, one launch serves all G (the launch's fixed cost is paid once); other shapes
 * run one call per matrix.
 * Errors: those of tri_linear for any matrix, TRI_EINVAL for a bad G or a null array. */
enum { TRI_MAX_GROUPS = 4 };
int tri_linear_grouped(const _Float16 *X, const uint8_t *const *Wp, const float *scale, int64_t M,
                       const int64_t *N, int64_t K, int fmt, _Float16 *const *Y, int G,
                       hipStream_t stream);

/* The glue of a decode block folded into a grouped layer (tri_linear_fused).  The
 * pages name the parts of a block, not this placement (Pith review, "If this is
 * right": the end-to-end speed-up trails the layer's because of the work outside
 * the linear layers). */
typedef struct {
    const _Float16 *norm_gain;         /* K fp16, or NULL for a gain of 1 */
    int norm;                          /* non-zero: RMS-normalise each input row:
                                          x * gain / sqrt(mean_k(x^2) + norm_eps) */
    float norm_eps;                    /* >= 0 and finite */
    int pair;                          /* non-zero: G == 2 and N[0] == N[1]; matrices 0 and 1
                                          are the gate and up projections of a gated MLP and
                                          only Y[0] = fp16(silu(y0) * y1) is written, with
                                          silu(z) = z / (1 + e^-z) (Y[1] may be NULL) */
    const _Float16 *const *residual;   /* NULL, or a HOST array of G pointers, each NULL or an
                                          M*N[g] fp16 residual added before rounding (it may
                                          be Y[g] itself: an in-place residual add); with
                                          pair, residual[1] must be NULL */
} tri_glue;

/* tri_linear_grouped with the glue: for g < G (g = 0 only with pair),
 *   y_g  = scale[g] * (x' W_g^T),  x' = rmsnorm(X) if norm, else X;
 *   Y[g] = fp16_rne( residual[g] + (pair ? silu(y_0) * y_1 : y_g) ).
 * The y_g are fp32 (never rounded on their own); the gained activations are
 * rounded to fp16 as an unfused RMSNorm output would be.  Served by the small-M
 * kernels in one launch for all G matrices; needs M <= 16 and K % 8 == 0.  With
 * norm or pair, K <= 16384 (2-bit) or K <= 20480 (1.6-bit), and for M > 8 also
 * K <= 15360 (1.6-bit with norm) and K <= 8192 / 10240 (2-bit / 1.6-bit with
 * pair); with neither, the row limits of tri_linear's MFMA small-M kernels apply
 * (K <= 16384 / 20480 at least).  Other shapes are rejected with TRI_EINVAL
 * before anything is launched.  norm_gain and the residuals must be 16-byte aligned
 * device pointers and must not alias Wp or (except residual[g] == Y[g]) any Y.
 * Errors: those of tri_linear_grouped, TRI_EINVAL for a null glue, a bad eps, a
 * bad pair or a shape outside the range above, TRI_EALIGN. */
int tri_linear_fused(const _Float16 *X, const uint8_t *const *Wp, const float *scale, int64_t M,
                     const int64_t *N, int64_t K, int fmt, _Float16 *const *Y, int G,
                     const tri_glue *glue, hipStream_t stream);

/* ---- 4-bit layers with group scales ---------------------------------------
 * For the layers of a mixed-precision model that ternary weights do not serve: 4-bit codes
 * with one fp16 scale, and optionally one zero point, per group of `group` consecutive
 * weights of a row,
 *
 *     W[n][k] = S[n][k / group] * (Q[n][k] - Z[n][k / group]),   Q, Z in 0..15,
 *
 * Z = 8 everywhere where a matrix is stored without zero points (zeros == 0).  group is 32,
 * 64 or 128.
 *
 * Layout of a packed matrix (tri_int4_bytes bytes), with NB = ceil(N/16) blocks of 16 rows,
 * KS = ceil(K/128) steps of 128 values and gps = 128/group groups per step:
 *   codes   32-bit word ((b*KS + s)*64 + 16*g + j)*4 + p holds the eight values
 *           k = 128 s + 32 p + 8 g + i (i < 8) of row 16 b + j, value i in the four bits from
 *           bit 4*(i/2) + 16*(i%2): the tile of a block and a step is 1 KB in a row, and the
 *           word that lane 16 g + j of a wave feeds to a matrix instruction is whole;
 *   scales  fp16 ((b*KS + s)*16 + j)*gps + i: row 16 b + j, group i of step s;
 *   zeros   (only if zeros != 0) bytes 0..15, indexed like the scales.
 * Rows past N and values past K hold code 8, scale 0 and zero point 8; groups that begin past K
 * likewise. */

/* Bytes of a packed N x K matrix; -1 if a size is < 1, N >= 2^31, K >= 2^25, the group is unknown
 * or the matrix has 2^22 tiles or more (8.6e9 weights): every call here rejects such a matrix. */
int64_t tri_int4_bytes(int64_t N, int64_t K, int group, int zeros);

/* Lay out codes that are given.  Q: N*K bytes (their low four bits count); S: N * ceil(K/group)
 * fp16; Z: N * ceil(K/group) bytes (low four bits), or NULL for a matrix without zero points;
 * all row-major.  Wp: tri_int4_bytes(N, K, group, Z != NULL) bytes, 16-byte aligned.
 * Errors: TRI_EINVAL, TRI_EALIGN (Wp; S not 2-byte aligned), TRI_EHIP. */
int tri_int4_pack(const uint8_t *Q, const _Float16 *S, const uint8_t *Z, int64_t N, int64_t K, int group,
                  uint8_t *Wp, hipStream_t stream);

/* The inverse of tri_int4_pack: writes Q, S and, if zeros != 0, Z (else Z is not used). */
int tri_int4_unpack(const uint8_t *Wp, int64_t N, int64_t K, int group, int zeros, uint8_t *Q, _Float16 *S,
                    uint8_t *Z, hipStream_t stream);

/* Quantise full-precision weights to nearest, group by group, and lay them out.  W: N*K float32
 * row-major, 4-byte aligned, finite.  In fp32, with m the group's largest |w| (zeros == 0):
 *     S = fp16_rne(m / 7) (at most 65504),  Q = clip(round_half_even(w / S), -8, 7) + 8;
 * with lo, hi the group's smallest and largest value, 0 included (zeros != 0):
 *     S = fp16_rne((hi - lo) / 15) (at most 65504),  Z = clip(round_half_even(-lo / S), 0, 15),
 *     Q = clip(round_half_even(w / S) + Z, 0, 15);
 * a group whose S is 0 has Q = Z = 8.  Errors as tri_int4_pack. */
int tri_int4_quantize(const float *W, int64_t N, int64_t K, int group, int zeros, uint8_t *Wp, hipStream_t stream);

/* The 4-bit layer:  Y[m][n] = fp16_rne( residual[m][n] + sum_k W[n][k] X[m][k] ), accumulated in
 * fp32 (codes minus zero points are exact in fp16; a group's sum is scaled in fp32).
 * X: M*K fp16 row-major; Wp: as packed for this N, K, group and zeros; residual: M*N fp16 or
 * NULL (it may be Y itself); Y: M*N fp16.  X, Wp, residual and Y must be 16-byte aligned; any M,
 * and any N and K that tri_int4_bytes takes.  Y must not alias X or Wp.  X is expected finite (a
 * row that is not spoils no other row's results).
 * Errors: TRI_EINVAL (a size < 1, M >= 2^31, N and K past tri_int4_bytes, null, unknown group),
 * TRI_EALIGN, TRI_EHIP. */
int tri_int4_linear(const _Float16 *X, const uint8_t *Wp, int64_t M, int64_t N, int64_t K, int group, int zeros,
                    const _Float16 *residual, _Float16 *Y, hipStream_t stream);

/* ---- Experts: ternary layers of which every row takes a few ----------------
 * A router gives every token a logit per expert; the token takes the top-k of them.  The
 * (token, expert) pairs are ordered by expert (tri_experts_route), the experts' products run
 * over that order, whose ragged sizes stay on the device (tri_experts_linear,
 * tri_experts_pair), and each token's results are weighted and added (tri_experts_combine).
 * No call waits for the device, allocates, or reads anything back. */
enum { TRI_MAX_EXPERTS = 256, TRI_MAX_TOPK = 16 };
enum { TRI_F16 = 0, TRI_F32 = 1 };                /* types of logits */

/* Workspace (device bytes) of tri_experts_route; -1 for sizes it does not take. */
int64_t tri_experts_route_workspace_bytes(int64_t T, int E, int topk);

/* logits: T*E row-major, fp16 (TRI_F16, 2-byte aligned) or fp32 (TRI_F32, 4-byte aligned).
 * Token t takes its topk largest logits, the lower expert first among equal ones; a logit of
 * -inf or NaN is never taken (a masked expert; a row of them is a token of padding).  Outputs:
 *   ids      T*topk: the experts, largest logit first; -1 where fewer than topk can be taken;
 *   weights  T*topk fp32: exp(x_j - max) / D, D the sum of exp(x - max) over the taken logits
 *            (renorm != 0) or over all of the row (renorm == 0); 0 where ids is -1.  Logits of
 *            +inf share the weight among themselves;
 *   offsets  E+1: expert e owns the places offsets[e] .. offsets[e+1]-1 of the order by expert
 *            (within one expert by token);
 *   rows     T*topk: the token at each place; -1 behind offsets[E];
 *   pos      T*topk: the place of pair (t, j); -1 where ids is -1.
 * All are int32 but the weights, 4-byte aligned.  1 <= E <= TRI_MAX_EXPERTS,
 * 1 <= topk <= min(E, TRI_MAX_TOPK), T < 2^27, T*topk < 2^31.  workspace: 16-byte aligned, at least
 * tri_experts_route_workspace_bytes bytes, overwritten; NULL where that is 0.  Calls that share
 * one must be ordered.  Errors: TRI_EINVAL, TRI_EALIGN, TRI_EHIP. */
int tri_experts_route(const void *logits, int dtype, int64_t T, int E, int topk, int renorm, int32_t *ids,
                      float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                      int64_t workspace_bytes, hipStream_t stream);

/* For every place r of expert e:  Y[r][n] = fp16_rne( scale[e] * sum_k t_e[n][k] X[x(r)][k] ),
 * x(r) = rows[r], or r itself where rows is NULL.  X: T*K fp16 (T >= R where rows is NULL); Wp: E
 * packed N x K matrices one after another, as tri_pack2 / tri_pack16 give them (for one matrix
 * of E*N rows, too); scale: E fp32 on the DEVICE (as tri_quantize writes them); offsets: E+1
 * int32, not decreasing, at most R (values outside are clamped); rows: R int32; Y: R*N fp16.
 * Rows of Y behind offsets[E] stay as they are, so do rows whose x(r) lies outside 0..T-1.  X,
 * Wp and Y must be 16-byte aligned, the rest 4-byte.  1 <= E <= TRI_MAX_EXPERTS,
 * N <= 2^27 - 16, K < 2^26; with rows, X of at most 4 GiB - 16.  Y must not alias an input.  X is expected
 * finite (a row that is not spoils only the places that name it).
 * Errors: TRI_EINVAL (a size < 1 or >= 2^31, null, unknown fmt), TRI_EALIGN, TRI_EHIP. */
int tri_experts_linear(const _Float16 *X, int64_t T, const int32_t *offsets, const int32_t *rows, int64_t R,
                       const uint8_t *Wp, const float *scale, int E, int64_t N, int64_t K, int fmt, _Float16 *Y,
                       hipStream_t stream);

/* tri_experts_linear's product with two matrices per expert, the gate and up projections of a
 * gated MLP:  Y[r] = fp16_rne( silu(g) * u ),  g and u the fp32 results of the two (never rounded
 * on their own), silu(z) = z / (1 + e^-z).  Wp_up and scale_up: as Wp and scale. */
int tri_experts_pair(const _Float16 *X, int64_t T, const int32_t *offsets, const int32_t *rows, int64_t R,
                     const uint8_t *Wp, const float *scale, const uint8_t *Wp_up, const float *scale_up, int E,
                     int64_t N, int64_t K, int fmt, _Float16 *Y, hipStream_t stream);

/* Y[t][n] = fp16_rne( residual[t][n] + sum_j weights[t][j] * Z[pos[t][j]][n] ), added in fp32, j
 * rising; pairs whose pos lies outside 0..R-1 are left out (nothing is read for them).  Z: R*N
 * fp16; pos, weights: T*topk; residual: T*N fp16 or NULL (it may be Y itself, no other input may); Y: T*N fp16.  Z,
 * residual and Y must be 16-byte aligned, pos and weights 4-byte.  1 <= topk <= TRI_MAX_TOPK.
 * Errors: TRI_EINVAL, TRI_EALIGN, TRI_EHIP. */
int tri_experts_combine(const _Float16 *Z, int64_t R, const int32_t *pos, const float *weights,
                        const _Float16 *residual, int64_t T, int topk, int64_t N, _Float16 *Y, hipStream_t stream);

/* ---- Heads, and an 8-bit cache of keys and values ---------------------------
 * What a decoder block computes between its Q/K/V layers and its O layer: every head of the
 * queries and keys normalised and rotated by its token's position (tri_heads_rotate), the new keys
 * and values rounded to 8 bits into the pages of a cache (tri_cache_append, which also does the
 * first for a call's queries and keys), and causal attention over that cache
 * (tri_cache_attend).  Sizes that change from step to step (how many tokens a sequence gets, how
 * long it is, which pages it has) stay on the device: no call waits, allocates, or reads anything
 * back, and a captured call follows them. */
enum { TRI_KV_INT8 = 0, TRI_KV_E4M3 = 1 };

/* T tokens of `heads` heads of dim values: value d of head h of token t is X[t*x_stride + h*dim + d]
 * (fp16), and of the results Y[t*y_stride + h*dim + d].  Strides are multiples of 8 and at least
 * heads*dim; X and Y are 16-byte aligned; Y may be X with the same stride, and overlap nothing else.
 * gain: dim fp16, 16-byte aligned, or NULL (a gain of 1); used only with a norm.  heads <= 65535. */
typedef struct tri_heads {
    const _Float16 *X;
    _Float16 *Y;
    const _Float16 *gain;
    int64_t x_stride, y_stride;
    int heads;
} tri_heads;

/* Norm and rotation.  norm != 0: x' = x / sqrt(mean_d x^2 + eps) * gain, eps >= 0.  table: rows x
 * dims/2 pairs (cos, sin) of fp32, 16-byte aligned: position p turns pair i of the first dims values,
 * (a, b) -> (a c - b s, a s + b c) with (c, s) = table[p][i]; the pair is (x[i], x[i + dims/2]), or
 * (x[2i], x[2i+1]) where interleaved != 0.  dims is a multiple of 16, at most dim; 0 (table is then
 * not used, and any position will do): no rotation.  All in fp32, rounded once. */
typedef struct tri_rotary {
    const float *table;
    int64_t rows;
    int dims, interleaved, norm;
    float eps;
} tri_rotary;

/* Y = the heads of X, normalised and rotated; G <= TRI_MAX_GROUPS sets of heads (queries and keys) of the
 * same T tokens in one launch.  positions: T int32; the rows of a token whose position lies outside
 * 0..rows-1 are not written.  dim: 64, 128 or 256.  T times the sets' heads together < 2^31.
 * Errors: TRI_EINVAL (T < 1, a size or stride out of range, null), TRI_EALIGN, TRI_EHIP. */
int tri_heads_rotate(const tri_heads *heads, int G, int64_t T, int dim, const tri_rotary *rot,
                     const int32_t *positions, hipStream_t stream);

/* A cache of `pages` pages of `page` tokens, `heads` key/value heads of dim values each:
 *   K        codes, (page, head, token, dim);
 *   V        codes, (page, head, dim, token);
 *   K_scale, V_scale   fp32, (page, head): a code stands for its value times its page's and head's scale.
 * Codes are int8 (two's complement, -127..127; TRI_KV_INT8) or OCP e4m3 (TRI_KV_E4M3; the two codes
 * that are no numbers are not written, and read as +-480).  page: 16, 32, 64 or 128; dim: 64, 128 or 256;
 * heads <= 65535; pages < 2^31.  Codes 16-byte aligned, scales 4-byte.  Scales are expected positive
 * and finite where a token is visible. */
typedef struct tri_cache {
    uint8_t *K, *V;
    float *K_scale, *V_scale;
    int64_t pages;
    int heads, dim, page, fmt;
} tri_cache;

/* A batch of B sequences with new tokens.  offsets: B+1 int32 on the device, not decreasing (values are
 * clamped to 0..T): rows offsets[b] .. offsets[b+1]-1 of a call's T rows are the new tokens of sequence
 * b.  lens: B int32 (clamped to 0..2^31 - 256), a sequence's tokens with the new ones: they stand at its last positions, row t at
 * lens[b] - offsets[b+1] + t.  table: B x width int32, row b the pages of sequence b in order; places past
 * its tokens, and pages that a window has left behind, may hold anything.  max_new, max_len: what a
 * sequence's new tokens and length are at most; grids are sized by them.  Only the first max_new new
 * tokens of a sequence are taken; a longer one than max_len is taken whole, if more slowly.  B <= 65535,
 * width, max_new, max_len < 2^31 - 128.  Pointers 4-byte aligned. */
typedef struct tri_sequences {
    const int32_t *offsets, *lens, *table;
    int64_t B, width, max_new, max_len;
} tri_sequences;

/* Round the T new tokens' keys and values to 8 bits, each at its position's page and place.  K, V: rows of
 * cache->heads heads, strides and alignment as in tri_heads.  rot: NULL, or the norm (with k_gain, dim
 * fp16 or NULL) and rotation that the keys go through first, rounded to fp16 there.
 * The scale of a page and head is a power of two: the least 2^e >= 2^-30 at which the largest of the
 * page's new values is at most 127 (int8) or 448 (e4m3) times it.  A page that holds earlier
 * tokens keeps its scale if that is as large; else it grows to the new one, and the earlier tokens'
 * codes are rounded again.  A code is the value times fp32(1 / scale), rounded to nearest, ties to even;
 * infinities count as +-65504, NaN as 0.  The places behind the new tokens stay as they are.
 * A token's keys and values are left out where its position is negative, has no place in the table of
 * pages or (rot->dims > 0) in the rotation's, or where its page is outside 0..pages-1.
 * queries: NULL, or (only with rot) query heads of the same T tokens, which are normalised and
 * rotated by the same launch, as tri_heads_rotate would at these positions; rows of no sequence, behind
 * a sequence's first max_new, or at a position that is negative or outside the rotation's table are
 * not written.
 * A page that gets new tokens must belong to one sequence and stand there once; calls that write the same
 * pages must be ordered.  K, V and queries must not overlap the cache.
 * Errors: TRI_EINVAL, TRI_EALIGN, TRI_EHIP. */
int tri_cache_append(const tri_cache *cache, const tri_sequences *seqs, int64_t T, const _Float16 *K,
                     int64_t k_stride, const _Float16 *V, int64_t v_stride, const tri_rotary *rot,
                     const _Float16 *k_gain, const tri_heads *queries, hipStream_t stream);

/* Workspace (device bytes, a multiple of 16, or 0) that tri_cache_attend needs for these arguments; it reads no
 * device memory.  -1 for sizes that it does not take. */
int64_t tri_cache_attend_workspace_bytes(const tri_cache *cache, const tri_sequences *seqs, int64_t T, int heads,
                                         int64_t window, int64_t sinks);

/* Causal attention of the T new tokens' queries over the cache, in which their own keys and values stand
 * already:  O[t][h] = sum_j p_j v_j,  p = softmax_j(scale q . k_j) over the visible positions j of the
 * token's sequence, k_j and v_j those of key/value head h / (heads / cache->heads).  Position p sees
 * j <= p; with window > 0 only j > p - window and the first `sinks` ones (window = 0: sinks is not
 * used).  A position whose page is outside 0..pages-1, or that has no place in the table, is not seen.
 * A row that sees nothing is 0; rows of no sequence (before offsets[0] or behind offsets[B]) and
 * rows behind a sequence's first max_new stay as they are.
 * Scores, softmax and sums are fp32 (a score that, times log2(e), passes fp32's range spoils its row); a
 * weight enters the second product as the sum of two fp16 numbers (off by 2^-22 of itself, or 2^-35 of
 * the largest product of a weight and its value's scale).  Q, O: rows of `heads` heads, as X and Y of tri_heads
 * (O must not overlap Q); heads is a multiple of cache->heads; scale is finite; T*heads < 2^31.
 * workspace: 16-byte aligned, of at least tri_cache_attend_workspace_bytes bytes, overwritten; NULL where
 * that is 0.  Calls that share one must be ordered.  Errors: TRI_EINVAL, TRI_EALIGN, TRI_EHIP. */
int tri_cache_attend(const tri_cache *cache, const tri_sequences *seqs, int64_t T, const _Float16 *Q, int64_t q_stride,
                     int heads, float scale, int64_t window, int64_t sinks, _Float16 *O, int64_t o_stride,
                     void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* The algorithm tri_linear would pick for (M, N, K, fmt); TRI_EINVAL if invalid.  Up to
 * M = 16 it is TRI_ALGO_SMALLM; above, whichever of TRI_ALGO_SMALLM and TRI_ALGO_GEMM a cost
 * model fitted to MI355X timings says is faster (the small-M kernels' time grows with the
 * number of 16-row slices; the GEMM's is flat while its 64 x 512 tiles fill at most half the
 * CUs, then grows with its rounds of 128 x 512 tiles). */
int tri_select_algo(int64_t M, int64_t N, int64_t K, int fmt);

/* Human-readable name of a status code (static string, never NULL). */
const char *tri_status_string(int code);

/* ---- Measurement aids (not part of the layer) ----------------------------
 * tri_probe_read streams `bytes` bytes (a multiple of 16, 16-byte aligned) with
 * 16-byte loads and writes one word to `sink` (4 bytes) only if a
 * data-dependent test that practically never holds passes; it is the
 * size-matched read floor for the weight stream.  tri_probe_copy copies
 * `bytes` bytes (a multiple of 16, both 16-byte aligned) from src to dst; it
 * calibrates hardware byte counters.  Errors: TRI_EINVAL, TRI_EALIGN, TRI_EHIP. */
int tri_probe_read(const void *src, int64_t bytes, uint32_t *sink, hipStream_t stream);
int tri_probe_copy(const void *src, void *dst, int64_t bytes, hipStream_t stream);

/* Launch-cost and read-pattern probes of the decode floor (measurement aids).
 * tri_probe_empty launches an empty kernel of `workgroups` workgroups of
 * `threads` threads (64..1024, a multiple of 64); sink (4 bytes) is never written.
 * tri_probe_rows issues exactly the loads of the one-row decode kernel over an N x
 * tri_row_bytes(K, fmt) packed matrix and a K-wide fp16 row X (16 rows per
 * workgroup of `waves` = 4 or 8 waves, the same chunk of every lane and the same
 * whole-line activation loads) and nothing else: it writes one 16-bit word per
 * matrix row to Y (N fp16 slots) that folds the bytes it read; rows longer than 8
 * steps of 4 chunks per wave give TRI_EINVAL.  tri_probe_stream reads `bytes`
 * bytes (a multiple of 16, below 2^31) with a grid of `workgroups` workgroups of
 * 256 threads, each lane keeping `unroll` (1, 2, 4 or 8) 16-byte loads in flight
 * per round; sink is written only if a data-dependent test that practically never
 * holds passes.  Errors: TRI_EINVAL, TRI_EALIGN (X, Wp, src), TRI_EHIP. */
int tri_probe_empty(int64_t workgroups, int threads, uint32_t *sink, hipStream_t stream);
int tri_probe_rows(const _Float16 *X, const uint8_t *Wp, int64_t N, int64_t K, int fmt, int waves,
                   _Float16 *Y, hipStream_t stream);
int tri_probe_stream(const void *src, int64_t bytes, int workgroups, int unroll, uint32_t *sink,
                     hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_H */
