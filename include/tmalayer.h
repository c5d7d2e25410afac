/*
 * tmalayer.h -- C ABI of what surrounds the products in a layer and in its training step:
 * the root-mean-square norm with the residual's addition and quantised rows, its
 * gradient, and the global norm of many gradients with clipping.
 *
 * Conventions are those of tmagemm.h, tmaexperts.h and tmamicro.h.
 */
#ifndef TMALAYER_H
#define TMALAYER_H

#include "tmamicro.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- root-mean-square norm ----------------------------------------------- */

/* For every row (token) of `width` values, with h = X + residual (h = X without):
 *   z = h / sqrt(mean(h^2) + eps) * weight
 * in fp32 from the unrounded sum h.  Written as asked for (NULL: not):
 *   total   h, fp16; may be X or residual itself
 *   Z       z, fp16; may be X (residual) itself, unless total is
 *   codes, scales   z as a matrix of `tokens` rows in `format` (tmamicro.h), rounded once;
 *           for GEMM_NVFP4 with the tensor scale 1, which suits values of this size:
 *           blocks of magnitudes from 0.1 to 2688 keep all bits of their scale
 * X, residual, weight (width values) are fp16.  width is a multiple of 8, 8 <= width <=
 * 32768; tokens >= 0; eps >= 0.  A row of zeros gives zeros (with eps = 0: NaN).  A row's
 * results do not depend on the other rows, nor on how many there are. */
TMAGEMM_API int gemm_rms_norm(int64_t tokens, int64_t width, const void* X, const void* residual,
                              const void* weight, float eps, void* total, void* Z, int format,
                              void* codes, void* scales, void* cuda_stream);

/* Gradients of gemm_rms_norm, given dZ, the h that it wrote (X without residual) and, if
 * not NULL, dH, the gradient that reaches h by its other uses:
 *   dX = dH + rstd * (u - n * mean(u n)),  rstd = 1 / sqrt(mean(h^2) + eps), n = h rstd,
 *                                          u = dZ weight
 * (fp16; the gradient of X and of residual alike; may be dZ or dH itself) and
 *   dweight = sum over the tokens of dZ n      (fp32).
 * The quantised rows count as z.  A row of dX does not depend on the other rows.  The
 * workspace is this call's alone until it has run. */
TMAGEMM_API int64_t gemm_rms_norm_grad_workspace(int64_t tokens, int64_t width); /* bytes */
TMAGEMM_API int gemm_rms_norm_grad(int64_t tokens, int64_t width, const void* dZ, const void* H,
                                   const void* weight, const void* dH, float eps, void* dX,
                                   float* dweight, void* workspace, void* cuda_stream);

/* ---- global gradient norm and clipping ------------------------------------ */

typedef struct gemm_clip_plan gemm_clip_plan; /* opaque; owned by the library */

/* For `count` tensors of sizes[i] >= 0 values of dtypes[i] (a gemm_dtype) at grads[i], and
 * outs[i] where the clipped values go: grads[i] itself, or memory that overlaps none of
 * the tensors.  The tensors are
 * aligned to their values' size (to 16 bytes they are faster).  The plan keeps a table of
 * the addresses in device memory (32 bytes for every 16384 values or part of a tensor), which
 * a graph that captured a run reads: it must not be replayed once the plan is destroyed. */
TMAGEMM_API gemm_clip_plan* gemm_clip_create_plan(int64_t count, const void* const* grads,
                                                  void* const* outs, const int64_t* sizes,
                                                  const int* dtypes);

/* Enqueue
 *   *norm = sqrt(sum of squares over all tensors)                    (fp32)
 *   outs[i] = grads[i] * min(1, max_norm / (*norm + eps))           (* 1 where the norm is 0)
 * Sums are held in fp32 over a few values and in fp64 over those, so that magnitudes
 * from the smallest to the largest fp32 neither vanish nor overflow (a norm beyond fp32 is
 * written as infinity, but the factor is that of the norm).  Infinite gradients
 * give an infinite norm and the factor 0 (infinities become NaN), NaN a factor NaN.
 * max_norm >= 0, eps >= 0.  The workspace (GEMM_CLIP_WORKSPACE_BYTES) is this call's alone
 * until it has run. */
#define GEMM_CLIP_WORKSPACE_BYTES 16384
TMAGEMM_API int gemm_clip_run(gemm_clip_plan* plan, float max_norm, float eps, float* norm,
                              void* workspace, void* cuda_stream);
/* The norm alone. */
TMAGEMM_API int gemm_clip_norm(gemm_clip_plan* plan, float* norm, void* workspace,
                               void* cuda_stream);
TMAGEMM_API void gemm_clip_destroy(gemm_clip_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* TMALAYER_H */
