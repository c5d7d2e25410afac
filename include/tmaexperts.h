/*
 * tmaexperts.h -- C ABI of the expert-layer operators that surround the fp16
 * GEMM of tmagemm.h in a mixture-of-experts feed-forward: tokens sorted by
 * expert and brought back, the experts' grouped products, both with their
 * gradients, and products with 4-bit weights for single tokens.
 *
 * Conventions are those of tmagemm.h: status codes of gemm_status, messages
 * through gemm_last_error(), DEVICE pointers owned by the caller and aligned to
 * 16 bytes, contiguous row-major matrices of fp16, sums in fp32 rounded once to
 * the output type, asynchronous launches on `cuda_stream` (a cudaStream_t;
 * NULL = legacy default stream), GEMM_ERR_NO_DEVICE without a GB300 and no
 * fallback of any kind.  Every kernel here is launched as a programmatic
 * dependent and touches global memory only after all earlier work on its
 * stream has completed, so stream order is kept.  All launches may be captured
 * into a CUDA graph (grouped plans: after one run outside the capture).
 * Results do not vary from run to run.
 *
 * Routing.  A layer sends each of `tokens` tokens to `topk` experts; slot
 * s = t * topk + j is choice j of token t.  A slot whose expert id is negative
 * or >= experts is dropped: it takes no part in any product, contributes
 * nothing to its token and has zero gradients.
 */
#ifndef TMAEXPERTS_H
#define TMAEXPERTS_H

#include "tmagemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- tokens sorted by expert and back ---------------------------------- */

/* Sort the slots by expert, keeping the order of slots within an expert:
 *   offsets[e]   first sorted row of expert e, e = 0..experts; offsets[0] = 0
 *                and offsets[experts] is the number of rows that are not dropped
 *   order[r]     slot at sorted row r
 *   position[s]  sorted row of slot s
 * Dropped slots take the rows from offsets[experts] on, in slot order, so
 * `order` and `position` are whole permutations.  expert_ids, order and
 * position hold tokens * topk int32, offsets experts + 1.  1 <= topk <= 256,
 * 1 <= experts <= 1024, tokens >= 0 and tokens * topk <= 2^30.  No workspace. */
TMAGEMM_API int gemm_expert_sort(int64_t tokens, int topk, int experts, const int32_t* expert_ids,
                                 int32_t* offsets, int32_t* order, int32_t* position,
                                 void* cuda_stream);

/* Xs[position[t * topk + j]] = X[t] for every slot that is not dropped; the
 * rows of dropped slots are set to zero.  X is tokens x width, Xs
 * tokens * topk x width, both fp16; width is a multiple of 8.  `offsets` and
 * `position` are those of gemm_expert_sort; X and Xs must not overlap. */
TMAGEMM_API int gemm_expert_gather(int64_t tokens, int topk, int experts, int64_t width,
                                   const void* X, const int32_t* offsets, const int32_t* position,
                                   void* Xs, void* cuda_stream);

/* Y[t] = sum_j weights[t * topk + j] * Ys[position[t * topk + j]] over the slots
 * that are not dropped, summed in fp32 in the order of j.  weights is fp32, or
 * NULL for a plain sum (the gradient of gemm_expert_gather with respect to X).
 * A token without any slot left gets a row of zeros.  The weight and the row of
 * a dropped slot are not used, so they may hold anything.  Ys is tokens * topk
 * x width fp16, Y tokens x width of dtype_out (a gemm_dtype).
 * With position = NULL the rows of Ys are in slot order and none is dropped
 * (offsets is then ignored and may be NULL). */
TMAGEMM_API int gemm_expert_combine(int64_t tokens, int topk, int experts, int64_t width,
                                    const void* Ys, const int32_t* offsets,
                                    const int32_t* position, const float* weights, int dtype_out,
                                    void* Y, void* cuda_stream);

/* As gemm_expert_combine for rows in slot order (row t * topk + j), as gemm_w4_run
 * leaves them; needs no sort.  A slot whose entry in `expert_ids` is negative or >=
 * experts is dropped, with the same meaning as there; expert_ids = NULL: none is. */
TMAGEMM_API int gemm_expert_combine_slots(int64_t tokens, int topk, int experts, int64_t width,
                                          const void* Ys, const int32_t* expert_ids,
                                          const float* weights, int dtype_out, void* Y,
                                          void* cuda_stream);

/* Gradients of the weighted gemm_expert_combine, given dY (tokens x width fp16):
 *   dYs[position[s]] = weights[s] * dY[t]               (fp16, every row written)
 *   dweights[s]      = sum_c dY[t][c] * Ys[position[s]][c]   (fp32)
 * with zeros for dropped slots.  dYs may be Ys itself (in place). */
TMAGEMM_API int gemm_expert_combine_grad(int64_t tokens, int topk, int experts, int64_t width,
                                         const void* dY, const void* Ys, const int32_t* offsets,
                                         const int32_t* position, const float* weights, void* dYs,
                                         float* dweights, void* cuda_stream);

/* ---- grouped products ---------------------------------------------------- */

typedef struct gemm_grouped_plan gemm_grouped_plan; /* opaque; owned by the library */

/* Rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1] - 1.
 *   GEMM_GROUPED_FORWARD      C[r]  = A[r] . B[e]^T     P = A (rows x K), Q = B
 *                             (experts x N x K), out = C (rows x N)
 *   GEMM_GROUPED_GRAD_INPUT   dA[r] = dC[r] . B[e]      P = dC (rows x N), Q = B,
 *                             out = dA (rows x K)
 *   GEMM_GROUPED_GRAD_WEIGHT  dB[e] = dC_e^T . A_e      P = dC (rows x N), Q = A
 *                             (rows x K), out = dB (experts x N x K)
 * Rows from offsets[experts] on belong to no expert: their C or dA is zero and
 * they add nothing to dB.  An expert without rows gets dB = 0.
 * The whole contraction is one sum in the tensor cores' fp32, which truncate where an
 * fp32 adder rounds: as with the GEMM, fp32 outputs are off by about 2e-6 of their
 * norm after 1000 to 2000 products, three times what a chain of rounded sums is. */
typedef enum {
    GEMM_GROUPED_FORWARD = 0,
    GEMM_GROUPED_GRAD_INPUT = 1,
    GEMM_GROUPED_GRAD_WEIGHT = 2
} gemm_grouped_op;

/* Plan for `rows` rows (an upper bound is fixed by the tensors, the split over
 * experts is read from `offsets` on the device at every run).  rows >= 0,
 * 1 <= experts <= 1024, N and K multiples of 8, all at most 2^31 - 65536 (and
 * experts * N too).  Returns NULL on error.  The plan owns a device record of 32
 * bytes, its status.  The counters from which runs hand out their tiles are the
 * device's (512 KB, allocated with its first plan and kept), one for every stream and
 * every captured launch: so runs of one plan may overlap on the GPU, on several
 * streams, from several threads, and with replays of graphs that hold runs of it. */
TMAGEMM_API gemm_grouped_plan* gemm_grouped_create_plan(int64_t rows, int64_t N, int64_t K,
                                                        int experts, int op, int dtype_out);

/* Same with an explicit output tile: 128 x 128 or 128 x 256 on single CTAs, 256 x
 * 256 on CTA pairs (up to about 200 experts).  GEMM_GROUPED_TILE_AUTO chooses by
 * the number of tiles and the rows per expert. */
typedef enum {
    GEMM_GROUPED_TILE_AUTO = 0,
    GEMM_GROUPED_TILE_128X128 = 1,
    GEMM_GROUPED_TILE_128X256 = 2,
    GEMM_GROUPED_TILE_256X256 = 3
} gemm_grouped_tile;

TMAGEMM_API gemm_grouped_plan* gemm_grouped_create_plan_ex(int64_t rows, int64_t N, int64_t K,
                                                           int experts, int op, int dtype_out,
                                                           int tile);

/* Enqueue the product.  `offsets` (experts + 1 int32, device memory) is as
 * gemm_expert_sort writes it: ascending from 0 to at most rows.  Values outside
 * [0, rows] are taken as the nearest bound, so a bad table gives wrong rows but
 * no access out of range; with one that descends no row belongs to an expert in
 * FORWARD and GRAD_INPUT. */
TMAGEMM_API int gemm_grouped_run(gemm_grouped_plan* plan, const void* P, const void* Q,
                                 const int32_t* offsets, void* out, void* cuda_stream);

/* Later runs: the bound on any single wait inside the kernel in milliseconds (0: the
 * default, 2000), and for tests of it `debug_stall` (0: none): 1 makes the producer of
 * the copies, 2 the reader of the sums first wait on a barrier that nothing completes.
 * Such a run ends with GEMM_ERR_TIMEOUT in the status; its output is not whole. */
TMAGEMM_API int gemm_grouped_set_wait(gemm_grouped_plan* plan, int wait_budget_ms,
                                      int debug_stall);

/* As gemm_get_device_status, gemm_destroy and gemm_plan_describe. */
TMAGEMM_API int gemm_grouped_get_device_status(gemm_grouped_plan* plan);
TMAGEMM_API void gemm_grouped_destroy(gemm_grouped_plan* plan);
TMAGEMM_API const char* gemm_grouped_describe(const gemm_grouped_plan* plan);

/* ---- products with 4-bit weights ----------------------------------------- */

typedef struct gemm_w4_plan gemm_w4_plan; /* opaque; owned by the library */

/* Y[m][n] = sum_k X[m][k] * scales[n][k / group] * (q[n][k] - zeros[n][k / group])
 *
 *   packed : N x K/2 bytes; byte b of a row holds q[2b] in its low and
 *            q[2b + 1] in its high four bits, q in 0..15
 *   scales : N x K/group fp16
 *   zeros  : N x K/group uint8 zero points, or NULL for 8 everywhere
 *   X      : M x K fp16      Y : M x N of dtype_out
 *
 * group is 32, 64 or 128, K a multiple of group, N of 8 (fp16) or 4 (fp32); all are at
 * most 2^31 - 65536, and experts * N too.
 * No weight is rounded, whatever the number of rows.  Up to 64 rows, and above where
 * that is expected to be faster, q - zero enters the tensor cores as the integer
 * it is, each group is summed in fp32 and scaled there ("rows" in gemm_w4_describe).
 * For more rows of an fp16 output, or of a short length, each weight is written out
 * once per run as the sum of two fp16 numbers and the GEMM of tmagemm.h multiplies them
 * over twice the length ("expand"); where a weight is beyond 65504 or an entry of X is
 * not finite, which that form does not cover, the kernel of "rows" computes Y.  The
 * plan then owns workspaces of N * K * 4 and M * K * 4 bytes.  An fp32 output is off by
 * about 1.5e-7 of its norm, by up to 3e-6 (the GEMM's sum) with more than 1024 rows and
 * K <= 1280.
 *
 * experts > 0: packed, scales and zeros are stacked (experts x N x ...), and row
 * m of Y is the product of X[m / share] with the weights of expert
 * expert_ids[m]; X has ceil(M / share) rows.  M <= 1024 then.  A row whose id is
 * negative or >= experts is set to zero.  experts = 0: one matrix, share = 1.
 *
 * Returns NULL on error.  Runs of one plan must not overlap on the GPU when it
 * expands the weights (they share the workspace). */
TMAGEMM_API gemm_w4_plan* gemm_w4_create_plan(int64_t M, int64_t N, int64_t K, int group,
                                              int experts, int share, int dtype_out);

/* Same with the caller's choice for many rows: GEMM_W4_WEIGHTS_ROUNDED lets a plan that
 * expands round each weight to fp16 (nearest even; beyond 65504 to an infinity), which
 * halves the GEMM and needs a workspace of N * K * 2 bytes only.  Y is then off by up
 * to half a unit in the last place of each weight. */
typedef enum { GEMM_W4_WEIGHTS_EXACT = 0, GEMM_W4_WEIGHTS_ROUNDED = 1 } gemm_w4_weights;

TMAGEMM_API gemm_w4_plan* gemm_w4_create_plan_ex(int64_t M, int64_t N, int64_t K, int group,
                                                 int experts, int share, int dtype_out,
                                                 int weights);

/* Enqueue the product.  expert_ids (M int32) must be given exactly when the
 * plan has experts. */
TMAGEMM_API int gemm_w4_run(gemm_w4_plan* plan, const void* X, const void* packed,
                            const void* scales, const void* zeros, const int32_t* expert_ids,
                            void* Y, void* cuda_stream);

/* As gemm_grouped_set_wait, for the kernel of "rows" (the GEMM of "expand" keeps its
 * default). */
TMAGEMM_API int gemm_w4_set_wait(gemm_w4_plan* plan, int wait_budget_ms, int debug_stall);

/* As gemm_get_device_status, gemm_destroy and gemm_plan_describe. */
TMAGEMM_API int gemm_w4_get_device_status(gemm_w4_plan* plan);
TMAGEMM_API void gemm_w4_destroy(gemm_w4_plan* plan);
TMAGEMM_API const char* gemm_w4_describe(const gemm_w4_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* TMAEXPERTS_H */
