/*
 * ttt_conv.h -- C ABI of the short causal convolution (B200, sm_100a).
 *
 * A depthwise convolution over the last K tokens of every channel, the one that
 * stands in front of a recurrence: on the queries and keys of the TTT scan
 * ("causal convolutions", PonderTTT, "Technical Architecture") and on the input
 * of the selective state space scan (ttt_ssm.h). For every batch row and channel
 *
 *     pre_t = bias + sum_{j < K} weight[j] * x_{t - (K-1) + j}
 *     y_t   = SiLU(pre_t) with TTT_CONV_SILU, else pre_t        (SiLU(x) = x sigmoid(x))
 *
 * where x_{-1}, x_{-2}, ... come from `state`, the K - 1 inputs before the first
 * token (zeros when NULL), and state_T is the K - 1 inputs before the position
 * that follows the last token, so that a prompt can be continued by another
 * prompt or by single tokens. Arithmetic is fp32.
 *
 * Channels are laid out as heads, [B, H, T, d] (H = 1: [B, T, d]), as in
 * ttt_scan.h. Every token-indexed tensor may have strides of its own between
 * batch rows, heads and tokens (a row of d channels is always contiguous), so
 * that a token-major projection [B, T, H*d] can be read in place and written as
 * the contiguous [B, H, T, d] that ttt_scan_forward takes.
 *
 * Status codes are those of ttt_scan.h. Every call only enqueues work on
 * `cuda_stream`, allocates no device memory, and reports argument errors before
 * anything is launched.
 */
#ifndef TTT_CONV_H
#define TTT_CONV_H

#include <stddef.h>

#include "ttt_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Mode bits, beside TTT_IN_BF16 (x, state, dx, dstate are bf16, else fp32) and
 * TTT_OUT_BF16 (y and dy are bf16, else fp32). */
enum {
  TTT_CONV_SILU = 1u << 16,    /* y = SiLU(pre) */
  TTT_CONV_PAD_ZERO = 1u << 20 /* y is set to 0 behind a row's length and in rows that are not
                                  active, else left as it was there (ignored by the backward) */
};

/*
 * A prompt. All pointers are device pointers, aligned to their element size (weight: 16 bytes):
 *   x        [B, H, T, d]     fp32, or bf16 with TTT_IN_BF16
 *   weight   [H, d, K]        fp32, contiguous, 16-byte aligned; K in {2, 3, 4}
 *   bias     [H, d]           fp32, contiguous; NULL = 0
 *   state    [B, H, K-1, d]   type of x, oldest first; NULL = zeros
 *   lengths  [B]              int32 tokens of each row, clipped to [0, T]; NULL = T.
 *                             Tokens at or past the length are not read, and y is left as it
 *                             was there (or 0 with TTT_CONV_PAD_ZERO).
 *   y        [B, H, T, d]     out: fp32, or bf16 with TTT_OUT_BF16
 *   state_T  [B, H, K-1, d]   out, or NULL; may be `state` itself (same strides)
 *   strides  NULL = all contiguous, or 12 element counts: between batch rows, heads and
 *            tokens (entries) of x, of y, of state and of state_T; none negative
 * Sizes: B, H, T >= 0, d >= 1, B <= 2^30, T <= 2^30 (backward: 2^22).
 * The extent of an output (from its first to its last element) may not meet
 * that of an input or of another output.
 */
int ttt_conv_forward(const void* x, const float* weight, const float* bias, const void* state,
                     const int* lengths, int B, int H, int T, int d, int K, unsigned mode,
                     const long long* strides, void* y, void* state_T, void* cuda_stream);

/*
 * Backward of a prompt: the gradients of <dy, y> + <dstate_T, state_T>.
 *   dy         as y of the forward (type and strides); dstate_T [B, H, K-1, d]
 *              contiguous, type of x; NULL = zero
 *   dx         [B, H, T, d] contiguous, type of x; 0 at and past a row's length
 *   dweight    [H, d, K] fp32, dbias [H, d] fp32 (NULL only with bias NULL): sums over rows
 *              and tokens in a fixed order, so that repeated calls agree bit for bit
 *   dstate     [B, H, K-1, d] contiguous, type of x; NULL = not wanted
 *   strides    NULL or 9 element counts: those of x, of dy and of state
 *   workspace  ttt_conv_backward_workspace_bytes(B, H, T, d, K) bytes of device memory, 16-byte
 *              aligned; calls that share one must not overlap
 */
size_t ttt_conv_backward_workspace_bytes(int B, int H, int T, int d, int K);
int ttt_conv_backward(const void* x, const float* weight, const float* bias, const void* state,
                      const int* lengths, int B, int H, int T, int d, int K, unsigned mode,
                      const long long* strides, const void* dy, const void* dstate_T, void* dx,
                      float* dweight, float* dbias, void* dstate, void* workspace,
                      size_t workspace_bytes, void* cuda_stream);

/*
 * One token of every row: x, y [B, H, d]; state [B, H, K-1, d] is read and moved
 * on by one IN PLACE. active [B] bytes or NULL: 0 = the row's state is left bit for bit, and its
 * y as it was (or 0 with TTT_CONV_PAD_ZERO). strides: NULL or 7 element counts, between rows and heads of x and of y, and
 * between rows, heads and entries of state. A chain of steps equals the prompt.
 */
int ttt_conv_step(const void* x, const float* weight, const float* bias, void* state,
                  const unsigned char* active, int B, int H, int d, int K, unsigned mode,
                  const long long* strides, void* y, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_CONV_H */
