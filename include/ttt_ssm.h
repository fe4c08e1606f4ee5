/*
 * ttt_ssm.h -- C ABI of the selective state space scan (B200, sm_100a).
 *
 * The diagonal recurrence with input-dependent step size and vectors, a sibling
 * of the TTT scan whose state is N numbers for each channel. For every batch row b,
 * channel c (of group g(c) = c / (D / G)) and token t
 *
 *     dt_t   = softplus(delta_t + delta_bias[c])     (delta_t + delta_bias[c] without TTT_SSM_SOFTPLUS)
 *     h_t[n] = exp(dt_t A[c, n]) h_{t-1}[n] + dt_t u_t Bm_t[g, n]
 *     r_t    = sum_n Cm_t[g, n] h_t[n] + skip[c] u_t
 *     y_t    = r_t SiLU(z_t)                         (r_t without z)
 *
 * States, parameters and arithmetic are fp32.
 *
 * Status codes are those of ttt_scan.h. Every call only enqueues work on
 * `cuda_stream`, allocates no device memory, and reports argument errors before
 * anything is launched.
 */
#ifndef TTT_SSM_H
#define TTT_SSM_H

#include <stddef.h>

#include "ttt_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Mode bits, beside TTT_IN_BF16 (u, delta, z, Bm, Cm and their gradients are bf16, else
 * fp32) and TTT_OUT_BF16 (y and dy are bf16, else fp32). */
enum {
  TTT_SSM_SOFTPLUS = 1u << 17, /* dt = softplus(delta + delta_bias) */
  TTT_SSM_PAD_ZERO = 1u << 20  /* y is set to 0 behind a row's length and in rows that are not
                                  active, else left as it was there (ignored by the backward) */
};

/* Tokens between two snapshots of the state (h_chunks). */
enum { TTT_SSM_CHUNK = 16 };

/*
 * A prompt. All pointers are device pointers, aligned to their element size except
 * where noted:
 *   u, delta, z [B, T, D]   fp32, or bf16 with TTT_IN_BF16; z NULL = no output gate
 *   Bm, Cm      [B, T, G, N] same type
 *   A           [D, N]      fp32, contiguous, 16-byte aligned; finite (beyond 2.35e38 it counts as
 *                           that), and A dt <= 0 for a state that decays (a growing one may leave
 *                           fp32's range)
 *   skip, delta_bias [D]    fp32; NULL = 0
 *   h0          [B, D, N]   fp32, contiguous, 16-byte aligned; NULL = zeros
 *   lengths     [B]         int32 tokens of each row, clipped to [0, T]; NULL = T. Tokens at or
 *                           past the length are not read, and y is left as it was there
 *                           (or 0 with TTT_SSM_PAD_ZERO)
 *   y           [B, T, D]   out: fp32, or bf16 with TTT_OUT_BF16
 *   h_T         [B, D, N]   out, fp32, contiguous, 16-byte aligned: the state after each row's
 *                           last token; may equal h0
 *   h_chunks    NULL, or out [B, ceil(T/16), D, N] fp32, 16-byte aligned: the state before every 16th
 *               token, for the backward (slots of chunks past a row's length are left as they were)
 *   strides     NULL = all contiguous, or 14 element counts, none negative: between rows and tokens of
 *               u, of delta, of z; between rows, tokens and groups of Bm, of Cm; between rows and
 *               tokens of y; at most 2^24 between tokens (any with T <= 1). The D channels, and
 *               the N entries, are always contiguous.
 * Sizes: B, T >= 0, B <= 2^30, T <= 2^30, 1 <= D <= 2^24, G >= 1 dividing D, N in {8, 16, 32, 64}.
 * The extent of an output may not meet that of an input (except h_T = h0) or of another
 * output.
 */
int ttt_ssm_forward(const void* u, const void* delta, const float* A, const void* Bm,
                    const void* Cm, const float* skip, const void* z, const float* delta_bias,
                    const float* h0, const int* lengths, int B, int T, int D, int G, int N,
                    unsigned mode, const long long* strides, void* y, float* h_T,
                    float* h_chunks, void* cuda_stream);

/*
 * Backward of a prompt: the gradients of <dy, y> + <dh_T, h_T> with respect to every
 * input of a ttt_ssm_forward call with the same arguments.
 *   h_chunks    the snapshots that call wrote
 *   dy          [B, T, D] type of y; dh_T [B, D, N] fp32, 16-byte aligned; NULL = zero
 *   du, ddelta, dz [B, T, D], dBm, dCm [B, T, G, N]: contiguous, type of u; 0 at and past a
 *               row's length (dz NULL exactly when z is)
 *   dA [D, N], dskip, d_delta_bias [D]  fp32: sums over rows and tokens in a fixed order, so that
 *               repeated calls agree bit for bit (dskip / d_delta_bias may be NULL: not wanted)
 *   dh0         [B, D, N] fp32, 16-byte aligned; NULL = not wanted
 *   strides     NULL or 14 element counts: as for the forward, with dy's in the place of y's
 *   workspace   ttt_ssm_backward_workspace_bytes(B, T, D, G, N) bytes of device memory, 16-byte
 *               aligned; calls that share one must not overlap
 */
size_t ttt_ssm_backward_workspace_bytes(int B, int T, int D, int G, int N);
int ttt_ssm_backward(const void* u, const void* delta, const float* A, const void* Bm,
                     const void* Cm, const float* skip, const void* z, const float* delta_bias,
                     const int* lengths, int B, int T, int D, int G, int N, unsigned mode,
                     const long long* strides, const float* h_chunks, const void* dy,
                     const float* dh_T, void* du, void* ddelta, float* dA, void* dBm, void* dCm,
                     float* dskip, void* dz, float* d_delta_bias, float* dh0, void* workspace,
                     size_t workspace_bytes, void* cuda_stream);

/*
 * One token of every row: u, delta, z, y [B, D]; Bm, Cm [B, G, N]; h [B, D, N] fp32, contiguous,
 * 16-byte aligned, is read and updated IN PLACE. active [B] bytes or NULL: 0 = the row's h is left bit for
 * bit, and its y as it was (or 0 with TTT_SSM_PAD_ZERO). strides: NULL or 8 element counts, between rows of u, delta, z; between rows and
 * groups of Bm, of Cm; between rows of y. A chain of steps equals the prompt.
 */
int ttt_ssm_step(const void* u, const void* delta, const float* A, const void* Bm,
                 const void* Cm, const float* skip, const void* z, const float* delta_bias,
                 float* h, const unsigned char* active, int B, int D, int G, int N,
                 unsigned mode, const long long* strides, void* y, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_SSM_H */
