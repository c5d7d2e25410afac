/*
 * tmamicro.h -- C ABI of the block-scaled ("microscaled") operators beside the fp16
 * GEMM of tmagemm.h: quantisation of fp16 matrices to 8- and 4-bit floating point
 * with scales, and the products of such matrices on the tensor cores' block-scaled
 * path.
 *
 * Conventions are those of tmagemm.h and tmaexperts.h: status codes of gemm_status,
 * messages through gemm_last_error(), DEVICE pointers owned by the caller and aligned
 * to 16 bytes, asynchronous launches on `cuda_stream`, GEMM_ERR_NO_DEVICE without a
 * GB300, no fallback, launches that may be captured into a CUDA graph, results that do
 * not vary from run to run.
 *
 * Formats (q is what is stored for a value, s the scale of its block; blocks run along
 * a row, and a row's last block may be short):
 *
 *   GEMM_MXFP8   q e4m3 (largest 448), s a power of two (e8m0) for every 32 values
 *   GEMM_MXFP4   q e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), s a power of two for every 32
 *   GEMM_NVFP4   q e2m1, s e4m3 for every 16, and one fp32, the tensor scale t, for the
 *                whole matrix: a value is q * s * t
 *
 * Quantisation of a block whose largest magnitude is a:
 *   MXFP8, MXFP4   s is the least power of two (of those from 2^-127) with a <= largest *
 *                  s, so that no value is cut off; q = round(x / s)
 *   NVFP4          t is the least power of two with max|X| <= 6 * 448 * t (1 for a matrix
 *                  of zeros) unless it is given, s = max(round_e4m3(a / (6 t)), 2^-9), at most
 *                  448, q = round(x / (s t)), at most 6 in magnitude
 * Every rounding is to the nearest, ties to even; with a given t that is no power of two,
 * of quotients that fp32 arithmetic leaves off by up to 2^-22 of themselves.  A block that
 * holds an infinity or a NaN gets the scale NaN: all its values are NaN.  Such values do not
 * enter t.
 *
 * Storage.  A matrix of `rows` x `K` is kept in the order in which the tensor cores read
 * it, in blocks of 128 rows:
 *   codes   [row / 128][chunk][row % 128][16 bytes]; a chunk is 16 bytes of a row (16
 *           values of MXFP8, 32 of the others, the first of two in the low four bits);
 *           a row has 2 * ceil(K / 32) chunks of MXFP8, 3 * ceil(K / 96) of MXFP4 and
 *           2 * ceil(K / 64) of NVFP4
 *   scales  [row / 128][group][row % 32][row % 128 / 32][4 bytes]; a group is four
 *           consecutive blocks of a row, of MXFP4 three (its fourth byte is not used)
 * Behind a row's K values there are codes of zero with scales that are numbers.  The
 * rows that fill up the last block of 128 may hold anything.
 */
#ifndef TMAMICRO_H
#define TMAMICRO_H

#include "tmagemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_MXFP8 = 0, GEMM_MXFP4 = 1, GEMM_NVFP4 = 2 } gemm_mx_format;

/* Bytes of the codes and of the scales of a rows x K matrix.  rows >= 0, K >= 1, both at
 * most 2^31 - 65536, and as many chunks over all blocks of rows and one more. */
TMAGEMM_API int gemm_mx_sizes(int64_t rows, int64_t K, int format, int64_t* codes_bytes,
                              int64_t* scales_bytes);

/* Workspace that gemm_mx_quantize needs to find a tensor scale itself. */
#define GEMM_MX_WORKSPACE_BYTES 4096

/* Quantise X (fp16, contiguous).  transpose = 0: X is rows x K, K a multiple of 8.
 * transpose = 1: X is K x rows, rows a multiple of 8, and the quantised matrix is its
 * transpose: blocks run along the columns of X.
 * tensor_scale (GEMM_NVFP4 only, else NULL): one fp32 in device memory.  With a workspace
 * (GEMM_MX_WORKSPACE_BYTES, for this call alone until it has run) it is found from X and
 * written; with workspace = NULL the number that it holds is used as it is: values beyond
 * 2688 times it are cut off.  With a negative number or a NaN all values are NaN. */
TMAGEMM_API int gemm_mx_quantize(int64_t rows, int64_t K, int format, int transpose, const void* X,
                                 void* codes, void* scales, float* tensor_scale, void* workspace,
                                 void* cuda_stream);

/* values[r][k] = q * s * t, rows x K of dtype_out (a gemm_dtype), contiguous, rounded once to
 * fp32, which holds every value where t is a power of two (but products under 2^-149), and
 * from there to fp16. */
TMAGEMM_API int gemm_mx_values(int64_t rows, int64_t K, int format, const void* codes,
                               const void* scales, const float* tensor_scale, int dtype_out,
                               void* values, void* cuda_stream);

/* ---- products ------------------------------------------------------------ */

typedef struct gemm_mx_plan gemm_mx_plan; /* opaque; owned by the library */

/* C[m][n] = sum_k A[m][k] * B[n][k] over the values of two quantised matrices of the same
 * format, A of M x K and B of N x K; C is M x N of dtype_out, row-major.  N * sizeof(C
 * element) is a multiple of 16; M, N, K >= 1 and at most 2^31 - 65536.  The products
 * are exact and summed in the tensor cores' fp32.  A plan owns a status record of
 * 32 bytes and no workspace: its runs may overlap.  A graph that captured a run must not be
 * replayed once the record is gone. */
TMAGEMM_API gemm_mx_plan* gemm_mx_create_plan(int64_t M, int64_t N, int64_t K, int format,
                                              int dtype_out);

/* Same with an explicit kernel: tiles of 256 x 256 on CTA pairs, or 128 rows of one operand
 * and up to 128 of the other on single CTAs, with `split` (1, 2, 4 or 8; 0: automatic) CTAs
 * of a cluster sharing a tile's length. */
typedef enum { GEMM_MX_AUTO = 0, GEMM_MX_PAIR = 1, GEMM_MX_SINGLE = 2 } gemm_mx_kernel;

TMAGEMM_API gemm_mx_plan* gemm_mx_create_plan_ex(int64_t M, int64_t N, int64_t K, int format,
                                                 int dtype_out, int kernel, int split);

/* A plan of other sizes in `plan`'s format, for products whose sizes change from call to call:
 * it has no device memory of its own and is made without a call that waits, also while a
 * stream is being captured.  Both use one status record, which reports a timeout in a run of
 * either and stays until the last of its plans is destroyed. */
TMAGEMM_API gemm_mx_plan* gemm_mx_create_plan_beside(const gemm_mx_plan* plan, int64_t M,
                                                     int64_t N, int64_t K, int dtype_out,
                                                     int kernel, int split);

/* Enqueue the product.  No scale may have its sign bit set (gemm_mx_quantize sets none).
 * scale_a, scale_b: the tensor scales of GEMM_NVFP4 (one fp32 each, whose product is a
 * finite fp32), or NULL for 1. */
TMAGEMM_API int gemm_mx_run(gemm_mx_plan* plan, const void* codes_a, const void* scales_a,
                            const float* scale_a, const void* codes_b, const void* scales_b,
                            const float* scale_b, void* C, void* cuda_stream);

/* As for grouped plans (tmaexperts.h). */
TMAGEMM_API int gemm_mx_set_wait(gemm_mx_plan* plan, int wait_budget_ms, int debug_stall);
TMAGEMM_API int gemm_mx_get_device_status(gemm_mx_plan* plan);
TMAGEMM_API void gemm_mx_destroy(gemm_mx_plan* plan);
TMAGEMM_API const char* gemm_mx_describe(const gemm_mx_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* TMAMICRO_H */
