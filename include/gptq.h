/*
 * gptq.h -- C ABI of the MI355X (gfx950) GPTQ layer-quantization library.
 *
 * The operation is GPTQ as derived on the pages
 *   [derivation] hbblog.cn  "GPTQ 从零推导：4-bit 权重量化为什么能“量化一列，补偿一列”"
 *   [teardown]   pinghaoyang.com.cn "GPTQ 完全拆解：二阶信息驱动的权重量化"
 * for one linear layer y = W x, W in R^{m x d}:
 *   1. H = (2/N) X X^T from N calibration inputs           ([derivation] eq. (9))
 *   2. dead-feature fix, optional act-order, damping       ([derivation] section 10, eq. (12), (34))
 *   3. R = upper Cholesky factor of (H + damp I)^-1        ([derivation] eq. (37)-(40))
 *   4. column-by-column b-bit affine quantization with the OBS feedback
 *      eta = (w - q) / R_jj folded into later columns, all rows in parallel,
 *      and the lazy block update W[:, T] -= E R[B, T]        ([derivation] eq. (36), (42), (46);
 *                                                            [teardown] Algorithm 1)
 *
 * Conventions shared by every entry point
 *   - Pointers are DEVICE pointers unless marked [host].  The caller owns every
 *     buffer; the library never allocates or frees device memory.  State it
 *     keeps between calls, per device, until the process ends: one internal
 *     non-blocking stream and two events (created, under a mutex, by the
 *     first factorisation on that device, with the caller stream's device
 *     current); a library-owned static scratch array and its address (see
 *     gptq_hessian_accumulate_noalloc).  Calls that share a workspace must
 *     not overlap.
 *   - Sizes: every matrix dimension (d, and m for the quantizer) is at most
 *     65535 (one grid dimension per row/column in several launches); larger
 *     values are rejected with GPTQ_ERR_INVALID_ARG.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Work is enqueued on it in order.  The factor also runs part of the
 *     triangular inverse on the internal stream, forked from `stream` and
 *     joined back into it by events before the call's later work, so the
 *     call stays ordered on `stream` as a whole.  gptq_cholesky_inverse and
 *     gptq_quantize_layer (when it factors) enqueue all of a damping
 *     attempt's work, then synchronise `stream` once to read the
 *     positive-definiteness flag; a failed attempt is redone whole.
 *   - Matrices are row-major with an explicit leading dimension.
 *   - Every argument is validated before anything is enqueued; a call that
 *     fails validation returns a status and leaves outputs untouched (NOT_SPD
 *     is reported after the work ran; see the factor).  Nothing is thrown
 *     across the ABI.
 */
#ifndef GPTQ_MI355_H
#define GPTQ_MI355_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gptq_status {
  GPTQ_OK = 0,
  GPTQ_ERR_INVALID_ARG = 1, /* bad size, pointer, dtype or parameter           */
  GPTQ_ERR_NOT_SPD = 2,     /* damped Hessian not positive definite after the
                               retries ([derivation] section 10: raise the
                               damping and retry; here damp *= 10, 5 times)   */
  GPTQ_ERR_WORKSPACE = 3,   /* ws_bytes smaller than the matching *_bytes query */
  GPTQ_ERR_HIP = 4          /* a HIP launch or runtime call failed              */
} gptq_status;

typedef enum gptq_dtype { GPTQ_BF16 = 0, GPTQ_F32 = 1, GPTQ_F16 = 2 } gptq_dtype;

/* The quantization grid ([derivation] 1.1 fit, eq. (36) encoder). */
typedef enum gptq_grid {
  /* min-max over the group, widened to contain 0: Delta = (hi - lo) /
     (2^b - 1), z = round(-lo / Delta); unsigned codes 0 .. 2^b - 1.        */
  GPTQ_GRID_MINMAX = 0,
  /* symmetric ([derivation] 1.1 names it; 8.4 the signed code form): range
     [-a, a], a = max |w|, 2^b - 1 levels -h..h around an exact 0 (h =
     2^(b-1) - 1), Delta = a / h.  Codes are stored SIGNED, c - h as b-bit
     two's complement; zeros[] is written as 0; w_hat = Delta * code.  At
     bits = 2 this is the ternary grid {-1, 0, +1} * Delta of [teardown]
     "extreme quantization: 2-bit and ternary".                              */
  GPTQ_GRID_SYMMETRIC = 1,
  /* given by the caller (fixed_scales / fixed_zeros below), e.g. the fixed
     grid of the [derivation] section 11 example; unsigned codes as for
     MINMAX.  With group_size > 0 the grids are on the static layout.       */
  GPTQ_GRID_FIXED = 2
} gptq_grid;

/* Quantizer settings; names follow the GPTQConfig fields the pages mention
 * (bits, group_size, desc_act) plus the algorithm's block size and damping. */
typedef struct gptq_params {
  int32_t bits;       /* 2, 3, 4 or 8                                           */
  int32_t group_size; /* -1: one grid per row, fitted on the original row.
                         >0: groups of g columns: dynamic (refitted at each
                         group start, in processing order, on the
                         compensated working weights, [derivation] 8.3/8.4;
                         every group that starts inside a block must end
                         inside it) or static (see static_groups).          */
  int32_t blocksize;  /* lazy-update block, >= 1 (the pages use 128)           */
  float percdamp;     /* damp = max(percdamp * mean(diag H), 2^-23), >= 0       */
  int32_t act_order;  /* 0: natural order; 1: descending diag(H), stable       */
  int32_t grid;       /* gptq_grid                                              */
  int32_t static_groups; /* 0/1, with group_size > 0: groups fitted once, before
                         GPTQ, on the ORIGINAL contiguous columns
                         [G g, (G+1) g) of the original row; processing
                         position j uses group floor(perm[j] / g)
                         ([derivation] 8.3), so g_idx[c] = c / g.  Any
                         (g, blocksize) pair.  Implied by GPTQ_GRID_FIXED.  */
  const float* fixed_scales;  /* GPTQ_GRID_FIXED only (else NULL): DEVICE
                         [m, n_g] fp32, positive finite steps               */
  const uint8_t* fixed_zeros; /* GPTQ_GRID_FIXED only (else NULL): DEVICE
                         [m, n_g] zero points <= 2^bits - 1                   */
} gptq_params;

const char* gptq_status_string(gptq_status s);

/* ---------------------------------------------------------------------------
 * Hessian statistics ([derivation] eq. (5), (9); accumulable over chunks, 9.4)
 *
 *   S[d, d] += sum_t x_t x_t^T   over the n_tok rows x_t of X.
 *
 * X: token-major activations [n_tok, d], row stride ldx >= d elements, dtype
 *    GPTQ_BF16 (products exact in fp32, accumulated in fp32 on the matrix
 *    cores) or GPTQ_F32 (accumulated in fp64).
 * S: fp32 [d, d] row-major, dense and symmetric on return.  Zero it before the
 *    first chunk; the caller keeps the running token count N.
 * ws: device scratch of at least gptq_hessian_workspace_bytes(d, n_tok) bytes
 *    (may be 0 bytes, then ws may be NULL).
 * Errors: INVALID_ARG for d <= 0, d > 65535, n_tok < 0, ldx < d, NULL S/X
 * (X may be NULL when n_tok == 0), bad dtype; WORKSPACE; HIP.
 * ------------------------------------------------------------------------- */
size_t gptq_hessian_workspace_bytes(int64_t d, int64_t n_tok);
gptq_status gptq_hessian_accumulate(float* S, int64_t d, const void* X,
                                    gptq_dtype x_dtype, int64_t n_tok,
                                    int64_t ldx, void* ws, size_t ws_bytes,
                                    void* stream);

/* ---------------------------------------------------------------------------
 * Allocation-free variant of gptq_hessian_accumulate, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same operation, arguments and errors,
 * without ws: the token-split partial sums live in a static device array of
 * GPTQ_NOALLOC_SCRATCH_BYTES that the library owns (one per GPU it runs on,
 * held until the process ends).  The split plan is chosen to fit that array,
 * so larger problems run with fewer (longer) token splits than
 * gptq_hessian_accumulate may use: S agrees with it to fp32 summation
 * rounding, bit for bit when both plans coincide.  Every partial the call
 * reads it has written itself, so no clearing is needed between calls.  The
 * array is shared by every call on one GPU: calls that overlap on one GPU
 * (other streams, other host threads) race on it and must be serialised by
 * the caller.  Calls no hipMalloc/hipFree.
 * ------------------------------------------------------------------------- */
#define GPTQ_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
gptq_status gptq_hessian_accumulate_noalloc(float* S, int64_t d, const void* X,
                                            gptq_dtype x_dtype, int64_t n_tok,
                                            int64_t ldx, void* stream);

/* ---------------------------------------------------------------------------
 * Factor ([derivation] section 10 steps 5-6, eq. (37)-(40)).
 *
 * From S (fp32 [d, d], as accumulated above) and the token count n:
 *   H = (2/n) S; dead[j] = (S[j][j] == 0), H[j][j] = 1 for dead j;
 *   perm = identity, or the stable order of descending diag(H) (act_order);
 *   H' = H[perm][:, perm] + damp I, damp = max(percdamp * mean diag H, 2^-23);
 *   R  = upper Cholesky factor of H'^-1, i.e. R^T R = H'^-1.
 * Computed in fp64 as H' = U U^T (U upper) and R = U^-1.  On failure the
 * damping is multiplied by 10 and the factorisation retried, at most 5 times.
 *
 * Outputs: R fp32 [d, d] row-major, processing order, lower triangle 0;
 *          perm int32 [d] (perm[j] = original column processed j-th);
 *          dead uint8 [d] (original order); *damp_used [host] (may be NULL).
 * ws: at least gptq_factor_workspace_bytes(d).
 * A non-finite S (NaN or inf on the diagonal) is reported as NOT_SPD; perm
 * is still a permutation (NaN keys order after every number, by index).
 * Errors: INVALID_ARG (d <= 0, d > 65535, n <= 0, percdamp < 0 or NaN, NULL
 *         outputs); WORKSPACE; NOT_SPD (*damp_used = last damping tried; R,
 *         perm and dead then hold the last attempt's values, R meaningless);
 *         HIP.
 * ------------------------------------------------------------------------- */
size_t gptq_factor_workspace_bytes(int64_t d);
gptq_status gptq_cholesky_inverse(const float* S, int64_t n, int64_t d,
                                  float percdamp, int32_t act_order, float* R,
                                  int32_t* perm, uint8_t* dead,
                                  float* damp_used, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---------------------------------------------------------------------------
 * Quantize one layer ([teardown] Algorithm 1; [derivation] section 10 with
 * dynamic groups and act-order per 8.3-8.4).
 *
 * W: [m, d] row-major (row stride ldw >= d), GPTQ_BF16 or GPTQ_F32; read only.
 * Factor input, one of:
 *   - R, perm, dead all NULL: S (fp32 [d, d]) and n are used and the factor
 *     is computed internally exactly as gptq_cholesky_inverse does;
 *   - R, perm, dead all non-NULL: a factor from gptq_cholesky_inverse for the
 *     same S, percdamp and act_order (layers sharing one Hessian); S may be
 *     NULL and n is ignored.
 * Outputs (all in ORIGINAL column order, fully overwritten):
 *   qweight uint32 [m, ceil(d*bits/32)]: per row an LSB-first bit stream,
 *           column c's code in stream bits [c*bits, (c+1)*bits), stream bit p
 *           in bit p%32 of word p/32; unused trailing bits are 0;
 *   scales  fp32  [m, n_g]  step Delta of each (row, group): processing
 *           groups for dynamic groups, original contiguous groups for
 *           static ones;
 *   zeros   uint8 [m, n_g]  integer zero point z (0 for GPTQ_GRID_SYMMETRIC,
 *           whose codes are signed);
 *           n_g = 1 for group_size -1, else ceil(d / group_size);
 *   g_idx   int32 [d]       group of each original column (0 for -1);
 *   w_hat   fp32  [m, d]    dequantized Delta * (code - z); may be NULL.
 * Codes c = clip(round_half_even(w / Delta) + z, 0, maxq) (eq. (36)),
 * maxq = 2^bits - 1 (2^bits - 2 for the symmetric grid).
 * ws: at least gptq_workspace_bytes(m, d, p) (includes the factor workspace
 *     only when the factor is computed internally: pass factor_inside = 1).
 * Errors: INVALID_ARG (m, d <= 0, m or d > 65535, ldw < d, bad params --
 *         including grid / static_groups out of range, GPTQ_GRID_FIXED
 *         without both fixed arrays or with them for another grid --, mixed
 *         NULL-ness of R/perm/dead, NULL S when factoring, NULL outputs);
 *         WORKSPACE; NOT_SPD (the outputs then hold meaningless values); HIP.
 * ------------------------------------------------------------------------- */
size_t gptq_workspace_bytes(int64_t m, int64_t d, const gptq_params* p,
                            int32_t factor_inside);
gptq_status gptq_quantize_layer(const void* W, gptq_dtype w_dtype, int64_t m,
                                int64_t d, int64_t ldw, const float* S,
                                int64_t n, const gptq_params* p,
                                const float* R, const int32_t* perm,
                                const uint8_t* dead, uint32_t* qweight,
                                float* scales, uint8_t* zeros, int32_t* g_idx,
                                float* w_hat, void* ws, size_t ws_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------
 * Inference on the stored format: the fused dequantizing matmul
 * ([wiki] "inference": W4A16 -- 4-bit weights expanded inside the matmul
 * kernel -- and 3-/2-bit likewise; format of [derivation] 3.1 / 8.3).
 *
 *   Y[k][r] = sum_c X[k][c] * W_hat[r][c],
 *   W_hat[r][c] = scales[r][g] * (code[r][c] - zeros[r][g]),  g = g_idx[c]
 *   (signed_codes = 1: code sign-extended from `bits` bits, zeros ignored).
 *
 * X: bf16 activations [n, d] token-major, row stride ldx >= d (GPTQ_BF16
 *    only); 0 <= n <= 524280.  Up to 16 rows: the vector units, one weight
 *    pass per 8 rows; more: bf16 matrix cores on tiles of 128 rows.
 * qweight, scales, zeros, g_idx: as gptq_quantize_layer writes them
 *    (qweight [m, ceil(d*bits/32)] uint32, scales / zeros uint8 [m, n_g]
 *    with n_g from group_size, g_idx int32 [d], values < n_g).
 * scale_dtype: GPTQ_F32 (the scales as written) or GPTQ_F16 (the compact
 *    16-bit storage of the steps: fp16 scales [m, n_g], e.g. the fp32 ones
 *    rounded to nearest; each is widened exactly to fp32 in the kernel).
 * Y: fp32 [n, m], row stride ldy >= m; fully overwritten.
 * Sums in fp32, every product of an activation and a code exact: each
 * group's grid is factored out of the group's sums (Delta (sum x c - z sum x)),
 * the codes entering the products as exact small numbers, never as rounded
 * weights.
 * Errors: INVALID_ARG (bad sizes, dtype, scale_dtype, bits, group_size,
 *         NULL pointers when n > 0); HIP.  Allocates nothing; no workspace.
 * ------------------------------------------------------------------------- */
gptq_status gptq_dequant_matmul(const void* X, gptq_dtype x_dtype, int64_t n,
                                int64_t d, int64_t ldx, const uint32_t* qweight,
                                const void* scales, gptq_dtype scale_dtype,
                                const uint8_t* zeros,
                                const int32_t* g_idx, int64_t m, int32_t bits,
                                int32_t group_size, int32_t signed_codes,
                                float* Y, int64_t ldy, void* stream);

/* ---------------------------------------------------------------------------
 * The transposed dequantizing matmul: the gradient of gptq_dequant_matmul
 * with respect to its activations, through the frozen packed weights.
 *
 *   dX[k][c] = sum_r dY[k][r] * W_hat[r][c]
 *
 * dY: bf16 [n, m], row stride lddy >= m (GPTQ_BF16 only); 0 <= n <= 524280.
 * qweight .. signed_codes: the stored format, as in gptq_dequant_matmul; a
 * group id outside [0, n_g) counts as the nearest one.
 * dX: bf16 [n, d], row stride lddx >= d; fully overwritten.
 * W_hat is rounded to bf16 once (by at most 2^-8 of it, as dX itself is when
 * stored); products are exact, sums fp32, rounded to bf16 at the end.
 * ws: at least gptq_dequant_matmul_t_workspace_bytes(n, m, d) bytes, 16-byte
 * aligned (else WORKSPACE).
 * Errors: INVALID_ARG (bad sizes, m or d > 65535, dtype, bits, group_size,
 *         NULL pointers when n > 0); WORKSPACE; HIP.
 * ------------------------------------------------------------------------- */
size_t gptq_dequant_matmul_t_workspace_bytes(int64_t n, int64_t m, int64_t d);
gptq_status gptq_dequant_matmul_t(const void* dY, gptq_dtype dy_dtype, int64_t n,
                                  int64_t m, int64_t lddy, const uint32_t* qweight,
                                  const void* scales, gptq_dtype scale_dtype,
                                  const uint8_t* zeros, const int32_t* g_idx,
                                  int64_t d, int32_t bits, int32_t group_size,
                                  int32_t signed_codes, void* dX, int64_t lddx,
                                  void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters beside the packed weights, for activation rows of many
 * requests at once: row k goes through the shared product and through the
 * adapter a = row[k] of its own request,
 *
 *   H[k] = X[k] A_a^T                                    (rank values)
 *   Y[k] = X[k] W_hat^T + alpha_a H[k] B_a^T
 *
 * A row whose id is outside [0, n_adapters) (for instance -1) has none: its
 * H is 0 and its Y the shared product alone.  Rows may name adapters in any
 * order; rows of one adapter that follow each other share its loads.
 * Adapters of a smaller rank are stored with zeros up to `rank`.
 *
 * X: bf16 [n, d], row stride ldx >= d; 0 <= n <= 524280; qweight ..
 * signed_codes: as in gptq_dequant_matmul_t; H: fp32 [n, rank] contiguous, or
 * NULL (gptq_lora_backward needs it); Y: [n, m] of y_dtype GPTQ_F32 or
 * GPTQ_BF16 (rounded once, at the end), row stride ldy >= m.  Both are fully
 * overwritten.
 * The shared product is gptq_dequant_matmul's: exact codes and activations,
 * fp32 sums per group; H is summed and kept in fp32 and enters its product
 * with B as three bf16 parts, i.e. exactly.
 * An activation that is not finite makes its own row's Y not finite (NaN also
 * where inf times a weight has a sign), and no other row's.
 * ws: at least gptq_lora_workspace_bytes(n, m, d, group_size, rank) bytes,
 *     16-byte aligned (else WORKSPACE).
 * Errors: INVALID_ARG (bad sizes, m or d > 65535, rank outside 1 .. 128,
 *         n_adapters outside 1 .. 65535, dtype, bits, group_size, NULL
 *         pointers when n > 0); WORKSPACE; HIP.
 * ------------------------------------------------------------------------- */
typedef struct gptq_adapters {
  const void* A;        /* DEVICE bf16 [n_adapters, rank, d] contiguous  */
  const void* B;        /* DEVICE bf16 [n_adapters, m, rank] contiguous  */
  const float* alpha;   /* DEVICE fp32 [n_adapters]                       */
  const int32_t* row;   /* DEVICE int32 [n]: adapter of each row          */
  int32_t n_adapters;
  int32_t rank;
} gptq_adapters;

size_t gptq_lora_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t group_size,
                                 int32_t rank);
gptq_status gptq_lora_matmul(const void* X, gptq_dtype x_dtype, int64_t n, int64_t d,
                             int64_t ldx, const uint32_t* qweight, const void* scales,
                             gptq_dtype scale_dtype, const uint8_t* zeros,
                             const int32_t* g_idx, int64_t m, int32_t bits,
                             int32_t group_size, int32_t signed_codes,
                             const gptq_adapters* adapters /*[host]*/, float* H,
                             void* Y, gptq_dtype y_dtype, int64_t ldy, void* ws,
                             size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Gradients of gptq_lora_matmul, given dY = d loss / d Y.  With a = row[k],
 *
 *   G[k]  = alpha_a dY[k] B_a
 *   dX[k] = dY[k] W_hat + G[k] A_a
 *   dA_a  = sum over the rows k of a  G[k]^T X[k]
 *   dB_a  = alpha_a sum over the rows k of a  dY[k]^T H[k]
 *
 * dY: bf16 [n, m], row stride lddy >= m; X: bf16 [n, d], row stride ldx >= d;
 * H: fp32 [n, rank], as gptq_lora_matmul wrote it (read for dB only).
 * dX: bf16 [n, d], row stride lddx >= d, or NULL; rounded as in
 * gptq_dequant_matmul_t.  dA: fp32 [n_adapters, rank, d] or NULL; dB: fp32
 * [n_adapters, m, rank] or NULL.  accumulate = 1 adds to dA and dB (gradients
 * over several micro-batches) instead of overwriting them; adapters without a
 * row get 0 (nothing added).  G and H enter as three bf16 parts, i.e. exactly;
 * sums fp32, over rows in an order fixed by the sizes and ids alone.  With
 * n = 0 the outputs are written (zeros, unless accumulating).
 * ws: at least gptq_lora_backward_workspace_bytes(...) bytes, 16-byte aligned
 *     (else WORKSPACE).
 * Errors: as gptq_lora_matmul (a pointer that only an output left NULL would
 *         read may be NULL).
 * ------------------------------------------------------------------------- */
size_t gptq_lora_backward_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t rank,
                                          int32_t n_adapters);
gptq_status gptq_lora_backward(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                               int64_t lddy, const void* X, int64_t ldx, const float* H,
                               const uint32_t* qweight, const void* scales,
                               gptq_dtype scale_dtype, const uint8_t* zeros,
                               const int32_t* g_idx, int64_t d, int32_t bits,
                               int32_t group_size, int32_t signed_codes,
                               const gptq_adapters* adapters /*[host]*/, void* dX,
                               int64_t lddx, float* dA, float* dB, int32_t accumulate,
                               void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Distillation from a teacher's top logits: how far a student's logits are
 * from a teacher's of whom only the k largest logits of each row are known
 * (the unquantized model's, kept once), and the gradient that trains the
 * student's adapters towards it.  With z = logits / T, q = softmax(z) over the
 * vocabulary, S the row's known ids and t their logits,
 *
 *   t_lse NULL:  p = softmax of t / T over S
 *     loss = w T^2 sum_S p (log p - log q)
 *     d loss / d logits_v = w T (q_v - p_v)
 *   t_lse given (the teacher's log-sum-exp of its logits / T over the whole
 *   vocabulary): p = exp(t / T - t_lse), and what is left, p_r = max(0, 1 -
 *   sum_S p), is one more class against the student's q_r = 1 - sum_S q
 *     loss = w T^2 [sum_S p (log p - log q) + p_r (log p_r - log q_r)]
 *     d loss / d logits_v = w T (q_v - p_v) on S, w T q_v (1 - p_r / q_r)
 *     elsewhere.  Where p_r = 0, or the student has no mass outside S (every
 *     other logit -inf, or none), that class is left out: with P = sum_S p,
 *     d loss / d logits_v = w T (P q_v - p_v) on S, w T P q_v elsewhere.
 *
 * logits: [n, vocab] of dtype GPTQ_BF16, GPTQ_F16 or GPTQ_F32, row stride ldl
 *   >= vocab; 1 <= vocab <= 262144; n <= 2097152.
 * t_idx int32 [n, k], t_logits fp32 [n, k]: contiguous, 1 <= k <= 1024.  Ids
 *   outside [0, vocab) are padding.  The known ids of a row are meant to be
 *   distinct; one named twice counts both its entries' probabilities.  A row
 *   without any known id has loss 0 and (t_lse NULL or p_r = 1) gradient 0.
 * weight: fp32 [n] or NULL (1).  A row of weight 0 is not read: its loss,
 *   stats and gradient are 0 whatever its logits hold.
 * A logit of -inf has probability 0 (a masked token); one that the teacher
 *   gives probability makes the loss +inf.  NaN, +inf and a row of nothing
 *   but -inf give NaN; a row of nothing but the type's lowest value is a row
 *   of equal logits.
 * loss: fp32 [n].  stats: fp32 [n, 2] or NULL: the log-sum-exp of z over the
 *   vocabulary and over the ids outside S (t_lse NULL: the same), for
 *   gptq_distill_backward.  dlogits: d sum(loss) / d logits in the logits'
 *   dtype, row stride ldd >= vocab, or NULL; it may be the logits' own buffer
 *   (same pointer and stride).
 * Cells are exponentiated and summed in fp32 (fp64 across threads), all that
 * is per row or known id in fp64.  Allocates nothing; no workspace.
 * Errors: INVALID_ARG (bad sizes, dtype, temperature outside 1e-30 .. 1e30,
 *         NULL pointers when n > 0); HIP.
 * ------------------------------------------------------------------------- */
gptq_status gptq_distill_loss(const void* logits, gptq_dtype dtype, int64_t n,
                              int64_t vocab, int64_t ldl, const int32_t* t_idx,
                              const float* t_logits, int64_t k, float temperature,
                              const float* t_lse, const float* weight, float* loss,
                              float* stats, void* dlogits, int64_t ldd, void* stream);
/* The gradient by itself, from the stats that gptq_distill_loss wrote for the
 * same arguments: dlogits[k] = grad[k] d loss[k] / d logits[k], grad fp32 [n]
 * = the derivative of the caller's scalar with respect to loss[k].  Arguments
 * and errors otherwise as in gptq_distill_loss. */
gptq_status gptq_distill_backward(const void* logits, gptq_dtype dtype, int64_t n,
                                  int64_t vocab, int64_t ldl, const float* stats,
                                  const int32_t* t_idx, const float* t_logits, int64_t k,
                                  float temperature, const float* t_lse,
                                  const float* weight, const float* grad, void* dlogits,
                                  int64_t ldd, void* stream);

/* ---------------------------------------------------------------------------
 * What rows of logits say about given tokens: how likely each is, how spread
 * the row's distribution is, and the row's largest logits.  Scores a quantized
 * model, and makes from a teacher's logits what gptq_distill_loss reads
 * (top_idx as t_idx, top_logits as t_logits, lse as t_lse).  With z = logits /
 * T, q = softmax(z):
 *   logp = log q_token,  entropy = - sum q log q,  lse = log sum exp z,
 *   top: the k largest logits in descending order, equal ones by lower id.
 *
 * logits: [n, vocab] of dtype GPTQ_BF16, GPTQ_F16 or GPTQ_F32, row stride ldl
 *   >= vocab; 1 <= vocab <= 262144; n <= 2097152.
 * tokens: int32 [n]; an id outside [0, vocab) asks for none (logp 0); may be
 *   NULL where logp is.
 * logp, entropy, lse: fp32 [n], each may be NULL.  stats: fp32 [n, 3] or NULL,
 *   for the gradient: the row's largest logit r, the log of sum exp((x - r) / T),
 *   and the entropy.
 * top_logits fp32 [n, k] (the logits themselves, not over T), top_idx int32
 *   [n, k]: 0 <= k <= 512, k <= vocab; may be NULL where k = 0.
 * A logit of -inf has probability 0 and is chosen behind all others.  NaN and
 * +inf make logp, entropy and lse NaN, and so does a row of nothing but -inf
 * (lse: -inf); a row of nothing but the type's lowest value is a row of equal
 * logits.  NaN is never among the largest; where fewer than k logits are
 * numbers the rest of top_idx is -1, of top_logits -inf.
 * Cells are exponentiated in fp32 relative to the largest, summed in fp32 for 32
 * cells and in fp64 beyond, the largest itself in fp64: logp is never above 0, entropy never
 * below, and both keep their digits where one token has nearly all the
 * probability.  Results are the same bits from run to run.  Rows whose logits rise
 * all along the vocabulary take twelve (fp32) to some twenty-two times (bf16) as long
 * for their largest, and up to half as long again without.
 * ws: at least gptq_token_logprobs_workspace_bytes(n, vocab, k) bytes, 16-byte
 *   aligned (else WORKSPACE).
 * Errors: INVALID_ARG (bad sizes, dtype, k, temperature outside 1e-30 .. 1e30,
 *         NULL pointers when n > 0); WORKSPACE; HIP.
 * ------------------------------------------------------------------------- */
size_t gptq_token_logprobs_workspace_bytes(int64_t n, int64_t vocab, int64_t k);
gptq_status gptq_token_logprobs(const void* logits, gptq_dtype dtype, int64_t n, int64_t vocab,
                                int64_t ldl, const int32_t* tokens, float temperature,
                                int64_t k, float* logp, float* entropy, float* lse,
                                float* stats, float* top_logits, int32_t* top_idx, void* ws,
                                size_t ws_bytes, void* stream);
/* The gradient of sum(grad_logp logp + grad_entropy entropy) with respect to
 * the logits, from the stats of the forward call on the same arguments:
 *   dlogits_v = [g (1[v = token] - q_v) - h q_v (log q_v + entropy)] / T,
 * g = grad_logp fp32 [n] or NULL (0), h = grad_entropy fp32 [n] or NULL (0); g
 * is 0 for a row without a token.  A row whose g and h are both 0 is not read:
 * its gradient is 0 whatever its logits hold.  dlogits: in the logits' dtype,
 * row stride ldd >= vocab; it may be the logits' own buffer (same pointer and
 * stride).  Errors as above; no workspace. */
gptq_status gptq_token_logprobs_backward(const void* logits, gptq_dtype dtype, int64_t n,
                                         int64_t vocab, int64_t ldl, const float* stats,
                                         const int32_t* tokens, float temperature,
                                         const float* grad_logp, const float* grad_entropy,
                                         void* dlogits, int64_t ldd, void* stream);

/* ---------------------------------------------------------------------------
 * Layer by layer ([derivation] 3.2 steps 1-2 and 10: capture each layer's
 * inputs, quantize it, verify its reconstruction error, go on to the next;
 * [teardown] "layer-wise quantization").
 *
 * For l = 0 .. n_layers-1, with X_0 = X_in:
 *   S_l = X_l^T X_l (gptq_hessian_accumulate);
 *   layer l quantized from S_l and N = n_tok (gptq_quantize_layer, factor
 *   inside, layers[l].params) into layers[l]'s outputs;
 *   layer_err[l] = (1/N) ||(W_l - W_hat_l) X_l||_F^2 ([derivation] eq. (6),
 *   from S_l in fp32 products with fp64 partial sums);
 *   X_{l+1} = bf16(act(X_l W_hat_l^T)) (gptq_dequant_matmul's arithmetic,
 *   then the activation, rounded to nearest even bf16).
 * X_out receives X_{n_layers}: the inputs the next layer would see, so a
 * stack is resumed at any layer by calling again with the remaining layers
 * and that X as X_in (the result is the same bits as one call).
 *
 * layers [host]: n_layers >= 1 descriptors; layers[l].d == layers[l-1].m.
 * X_in: bf16 [n_tok, layers[0].d] contiguous; X_out: bf16 [n_tok,
 * layers[n-1].m] contiguous; 1 <= n_tok <= 524280.  activation: gptq_activation.
 * layer_err [host]: n_layers doubles, may be NULL.
 * ws: at least gptq_stack_workspace_bytes(layers, n_layers, n_tok).
 * Synchronises `stream` once per layer (the factor's flag) and at the end.
 * Errors: INVALID_ARG (any layer's arguments as for gptq_quantize_layer,
 *         mismatched dimensions, bad activation, NULL X_in / X_out);
 *         WORKSPACE; NOT_SPD (from the failing layer; earlier layers'
 *         outputs are final); HIP.
 * ------------------------------------------------------------------------- */
typedef enum gptq_activation {
  GPTQ_ACT_NONE = 0, GPTQ_ACT_RELU = 1, GPTQ_ACT_SILU = 2
} gptq_activation;

typedef struct gptq_stack_layer {
  const void* W;        /* [m, d] row-major, row stride ldw >= d; read only */
  gptq_dtype w_dtype;
  int64_t m, d, ldw;
  gptq_params params;
  uint32_t* qweight;    /* outputs, as gptq_quantize_layer writes them */
  float* scales;
  uint8_t* zeros;
  int32_t* g_idx;
} gptq_stack_layer;

size_t gptq_stack_workspace_bytes(const gptq_stack_layer* layers, int32_t n_layers,
                                  int64_t n_tok);
gptq_status gptq_quantize_stack(const gptq_stack_layer* layers, int32_t n_layers,
                                const void* X_in, int64_t n_tok, int32_t activation,
                                void* X_out, double* layer_err, void* ws,
                                size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Layers and activations in 4-bit floating point (MXFP4): values 0, 1/2, 1,
 * 3/2, 2, 3, 4, 6 and their negatives (e2m1) in blocks of 32 along a row, a
 * block's values times one power of two.  The format that the matrix cores
 * take directly, for layers that need no integer grid and for activations.
 *
 * Stored format of a matrix [rows, d], nb = ceil(d / 32):
 *   codes  uint8 [rows, 16 nb] contiguous, 16-byte aligned: the code (sign,
 *          two bits of exponent, one of mantissa) of column c in byte c / 2,
 *          even columns in the lower half; 0 past d;
 *   scales uint8 [rows, nb] contiguous: 127 + the power of two of each block;
 *          255: the block is NaN.
 *
 * gptq_mx_quantize rounds X [n, d] (bf16, fp16 or fp32, row stride ldx >=
 * d) to it.  The power of a block is floor(log2 max |x|) - 2, at least -127
 * (which a block of zeros gets), so that its largest value lies at 4 to 8;
 * values go to the nearest, halves to the even code, beyond 6 to 6.  A block
 * with a value that is not finite is NaN as a whole.  hat: the values that
 * the codes stand for, [n, d] in X's type (exact in it), row stride ldh >= d,
 * or NULL.  0 <= n <= 524280, d <= 65535.
 * Errors: INVALID_ARG (bad sizes, dtype, alignment, NULL pointers when n > 0);
 *         HIP.  Allocates nothing; no workspace.
 * ------------------------------------------------------------------------- */
gptq_status gptq_mx_quantize(const void* X, gptq_dtype dtype, int64_t n, int64_t d,
                                int64_t ldx, uint8_t* codes, uint8_t* scales, void* hat,
                                int64_t ldh, void* stream);

/* ---------------------------------------------------------------------------
 * The product with such a layer W [m, d]:  Y[k][r] = sum_c X[k][c] W[r][c].
 *
 * x_form: GPTQ_MX_BF16: X bf16 [n, d], row stride ldx >= d, as it is;
 *   GPTQ_MX_ROUND: the same, rounded as gptq_mx_quantize does (the result
 *   is that of the two calls); GPTQ_MX_CODES: X codes uint8 [n, 16 nb] and
 *   x_scales [n, nb], as gptq_mx_quantize writes them (ldx ignored), for
 *   activations that several products share.  x_scales is read only then.
 * Y: [n, m] of y_dtype GPTQ_F32 or GPTQ_BF16 (rounded once, at the end), row
 *   stride ldy >= m; fully overwritten.  Any n from 0 to 524280.
 * Every product is exact, sums are fp32.  Values beyond 2^127 (scale bytes
 * from 253 on, which no finite input gets) count as infinite with bf16
 * activations.  A block that is NaN, or an activation that is not finite, makes
 * its row's (its column's) results NaN or infinite and no others.
 * ws: at least gptq_mx_matmul_workspace_bytes(n, m, d, x_form) bytes,
 *   16-byte aligned (else WORKSPACE).
 * Errors: INVALID_ARG (bad sizes, m or d > 65535, x_form, dtype, alignment,
 *         NULL pointers when n > 0); WORKSPACE; HIP.
 * ------------------------------------------------------------------------- */
typedef enum gptq_mx_input {
  GPTQ_MX_BF16 = 0, GPTQ_MX_ROUND = 1, GPTQ_MX_CODES = 2
} gptq_mx_input;

size_t gptq_mx_matmul_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t x_form);
gptq_status gptq_mx_matmul(const void* X, int32_t x_form, const uint8_t* x_scales, int64_t n,
                              int64_t d, int64_t ldx, const uint8_t* codes,
                              const uint8_t* scales, int64_t m, void* Y, gptq_dtype y_dtype,
                              int64_t ldy, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Its gradient with respect to X as it is (through the frozen layer; for
 * rounded activations the one of the unrounded product):
 *   dX[k][c] = sum_r dY[k][r] W[r][c]
 * dY: bf16 [n, m], row stride lddy >= m; dX: bf16 [n, d], row stride lddx >= d,
 * fully overwritten.  Products are exact, sums fp32, rounded once at the end.
 * ws: at least gptq_mx_matmul_t_workspace_bytes(n, m, d) bytes, 16-byte
 * aligned (else WORKSPACE).  Errors as in gptq_mx_matmul.
 * ------------------------------------------------------------------------- */
size_t gptq_mx_matmul_t_workspace_bytes(int64_t n, int64_t m, int64_t d);
gptq_status gptq_mx_matmul_t(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                                int64_t lddy, const uint8_t* codes, const uint8_t* scales,
                                int64_t d, void* dX, int64_t lddx, void* ws, size_t ws_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------
 * The gated feed-forward block on two such layers [m, d],
 *   G = X W_gate^T,  U = X W_up^T,  Y = act(G) * U
 * with both products, the activation (gptq_activation) and the product of the
 * two in one pass; the block's third layer takes Y through gptq_mx_matmul.
 * X, x_form, x_scales, d, ldx: as in gptq_mx_matmul.  Y: bf16 [n, m], row
 * stride ldy >= m, from G and U in fp32.  G, U: bf16 [n, m] with row stride
 * ldg >= m for gptq_mx_gated_backward, or both NULL.
 * ws: at least gptq_mx_gated_workspace_bytes(n, m, d, x_form) bytes, 16-byte
 * aligned (else WORKSPACE).
 *
 * Its gradients, from dY bf16 [n, m] (row stride lddy >= m) and the G and U
 * that the forward call wrote:
 *   dU = dY act(G),  dG = dY U act'(G),  dX = dG W_gate + dU W_up
 * (ReLU's slope at 0 is 0; for rounded activations dX is that of the
 * unrounded product).  dGU: bf16 [n, 2 mp] contiguous, 16-byte aligned, mp =
 * m rounded up to 64: dG in columns [0, m), dU in [mp, mp + m), zeros between
 * and behind.  dX: bf16 [n, d], row stride lddx >= d, from dG and dU as rounded
 * to bf16 (off by 0.0023 of itself in the mean square, its own rounding being
 * 0.0017); or NULL (then neither the layers nor ws are read).
 * ws: at least gptq_mx_gated_backward_workspace_bytes(n, m, d) bytes,
 * 16-byte aligned (else WORKSPACE).
 * Errors: as in gptq_mx_matmul; INVALID_ARG also for a bad activation and
 *         for G without U.
 * ------------------------------------------------------------------------- */
size_t gptq_mx_gated_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t x_form);
gptq_status gptq_mx_gated(const void* X, int32_t x_form, const uint8_t* x_scales, int64_t n,
                             int64_t d, int64_t ldx, const uint8_t* gate_codes,
                             const uint8_t* gate_scales, const uint8_t* up_codes,
                             const uint8_t* up_scales, int64_t m, int32_t activation, void* Y,
                             int64_t ldy, void* G, void* U, int64_t ldg, void* ws,
                             size_t ws_bytes, void* stream);
size_t gptq_mx_gated_backward_workspace_bytes(int64_t n, int64_t m, int64_t d);
gptq_status gptq_mx_gated_backward(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                                      int64_t lddy, const void* G, const void* U, int64_t ldg,
                                      const uint8_t* gate_codes, const uint8_t* gate_scales,
                                      const uint8_t* up_codes, const uint8_t* up_scales,
                                      int64_t d, int32_t activation, void* dX, int64_t lddx,
                                      void* dGU, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Tracing: per-phase GPU time.  While enabled, each launch group of a phase
 * is bracketed by two hipEvents recorded on the caller's stream (a few
 * microseconds per group; leave it off when timing the whole path).
 * Phases: GPTQ_TRACE_STATS (the statistics kernels of one
 * gptq_hessian_accumulate call), GPTQ_TRACE_FACTOR (one damping attempt's
 * factorisation, H through R), GPTQ_TRACE_CHAIN (each in-block column-chain
 * launch), GPTQ_TRACE_LAZY (each lazy block update), GPTQ_TRACE_OTHER (grid
 * fits, working-copy set-up, output re-layout of a layer).
 * gptq_trace_read waits for the recorded events and writes the summed
 * milliseconds (and the number of launch groups) per phase since the last
 * reset; reset = 1 clears them.  Host-side state guarded by a mutex.
 * ------------------------------------------------------------------------- */
#define GPTQ_TRACE_PHASES 5
enum { GPTQ_TRACE_STATS = 0, GPTQ_TRACE_FACTOR = 1, GPTQ_TRACE_CHAIN = 2,
       GPTQ_TRACE_LAZY = 3, GPTQ_TRACE_OTHER = 4 };
gptq_status gptq_trace_enable(int32_t enable);
gptq_status gptq_trace_read(double* ms /*[host] 5*/, int64_t* launches /*[host] 5, may be NULL*/,
                            int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_MI355_H */
