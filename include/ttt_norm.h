/*
 * ttt_norm.h -- C ABI of the root-mean-square norm between two blocks (B200, sm_100a).
 *
 * For every row of D numbers, in fp32,
 *
 *     s = x + residual           (s = x without a residual)
 *     y = s / sqrt(mean(s^2) + eps) * weight
 *
 * s goes out in the residual stream's type, y (from the unrounded s) as fp32,
 * bf16, or 8 bits (e4m3) with fp32 scales: for each row, or for each 128 columns
 * of it, scale = max |y| / 448 (at least the smallest normal fp32, so that it can be
 * divided by; NaN with a NaN among them) and code = e4m3(y / scale), the fp32 quotient to nearest. The 8-bit form is
 * what the projections behind the norm take in serving.
 *
 * Status codes are those of ttt_scan.h. Every call only enqueues work on
 * `cuda_stream`, allocates no device memory, and reports argument errors before
 * anything is launched.
 */
#ifndef TTT_NORM_H
#define TTT_NORM_H

#include <stddef.h>

#include "ttt_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Mode bits: TTT_IN_BF16 (x is bf16, else fp32), TTT_OUT_BF16 (y is bf16, else fp32), and */
enum {
  TTT_NORM_SUM_BF16 = 1u << 18, /* residual and s (and, backward, s, ds, dx) are bf16, else fp32 */
  TTT_NORM_Y_E4M3 = 1u << 19    /* y is e4m3 codes with scales; excludes TTT_OUT_BF16 */
};

/*
 * All pointers are device pointers, aligned to their element size:
 *   x        [M, D]; residual [M, D], or NULL (then s is not written and must be NULL)
 *   weight   [D] fp32
 *   y        [M, D] out
 *   s        [M, D] out; NULL = not wanted; may equal residual, or x where x has its type (same
 *            row stride)
 *   scale    [M, groups] fp32 out, contiguous, with TTT_NORM_Y_E4M3 (else NULL); groups = 1 with
 *            group = 0 and ceil(D / 128) with group = 128
 *   strides  NULL = contiguous, or 4 element counts between rows, at least D: x, residual, y, s
 * Sizes: M >= 0, 1 <= D <= 16384, eps >= 0 (finite). Outputs overlap nothing else.
 */
int ttt_norm_forward(const void* x, const void* residual, const float* weight, int M, int D,
                     float eps, unsigned mode, int group, const long long* strides, void* y,
                     void* s, float* scale, void* cuda_stream);

/*
 * Backward: with s as the forward wrote it (x itself without a residual), r = 1 / sqrt(mean(s^2) +
 * eps), and ds the gradient that reaches s from elsewhere (NULL = none),
 *     dx      = r (weight dy - s r mean(weight dy s r)) + ds     the gradient of x and of residual
 *     dweight = sum over rows of dy s r, in a fixed order (repeated calls agree bit for bit)
 *   dy [M, D] fp32, or bf16 with TTT_OUT_BF16; s, ds, dx [M, D] fp32, or bf16 with
 *   TTT_NORM_SUM_BF16; dx may equal ds (same row stride); dweight [D] fp32
 *   strides    NULL or 4 element counts between rows: dy, s, ds, dx
 *   workspace  ttt_norm_backward_workspace_bytes(M, D) bytes of device memory, 16-byte aligned;
 *              calls that share one must not overlap
 */
size_t ttt_norm_backward_workspace_bytes(int M, int D);
int ttt_norm_backward(const void* dy, const void* s, const float* weight, const void* ds, int M,
                      int D, float eps, unsigned mode, const long long* strides, void* dx,
                      float* dweight, void* workspace, size_t workspace_bytes,
                      void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_NORM_H */
