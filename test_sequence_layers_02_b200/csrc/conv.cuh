// Short causal convolution, depthwise over K = 2..4 tokens: prompt, backward and
// one-token step (include/ttt_conv.h has the formulas).
//
// Every kernel is one pass over the tokens: K multiply-adds and one SiLU per
// element against one read and one write, so HBM bounds it. A thread owns VEC
// neighbouring channels and walks a run of tokens with the last K - 1 inputs in
// registers, so an input is read from memory once (and K - 1 tokens again at the
// start of a run, from cache); a warp reads 32 VEC neighbouring channels.
#pragma once

#include "seq_common.cuh"

namespace ttt {

struct RowStrides {
  long long b, h, t;  // elements between batch rows, heads, tokens
};

struct ConvParams {
  const void* x;
  const float* weight;  // [H, d, K]
  const float* bias;    // [H, d] or null
  const void* state;    // [B, H, K-1, d] or null
  const int* lengths;   // [B] or null
  void* y;              // forward out, backward dy (read only)
  void* state_T;        // forward out or null
  const void* dstate_T;  // backward, contiguous, or null
  void* dx;             // backward, contiguous
  void* dstate;         // backward, contiguous, or null
  float* part;          // backward: [B * tiles][D K + D] partial sums
  const unsigned char* active;  // step: [B] or null
  RowStrides xs, ys, ss, so;
  int B, H, T, d;
  int vecs;             // vectors of VEC channels over all heads: H * d / VEC
  int tiles;            // runs of tokens (forward), blocks along the tokens (backward)
  int silu;
  int pad_zero;         // y = 0 behind a length and in rows that are not active
};

template <typename T>
__device__ __forceinline__ const T* row_ptr(const void* p, const RowStrides& s, int b, int h,
                                            long long t, int c) {
  return static_cast<const T*>(p) + b * s.b + h * s.h + t * s.t + c;
}
template <typename T>
__device__ __forceinline__ T* row_ptr(void* p, const RowStrides& s, int b, int h, long long t,
                                      int c) {
  return static_cast<T*>(p) + b * s.b + h * s.h + t * s.t + c;
}

// The VEC channels' weights, w[i][j] = weight[c + i][j]. The VEC K floats are one
// contiguous run that starts on 16 bytes when VEC is a multiple of 4.
template <int VEC, int K>
__device__ __forceinline__ void load_weights(const float* weight, int c, float (&w)[VEC][K]) {
  const float* p = weight + (size_t)c * K;
  if constexpr (VEC % 4 == 0) {
    float f[VEC * K];
#pragma unroll
    for (int i = 0; i < VEC * K; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < K; ++j) w[i][j] = f[i * K + j];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < K; ++j) w[i][j] = __ldg(p + i * K + j);
  }
}

__device__ __forceinline__ int row_length(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

constexpr int kConvRun = 16;     // tokens per thread (forward)

// Linear thread index over (run, vector) in x, batch rows in y.
template <typename InT, typename OutT, int VEC, int K>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const ConvParams p) {
  const long long idx = (long long)blockIdx.x * 128 + threadIdx.x;
  const int run = (int)(idx / p.vecs);
  if (run >= p.tiles) return;
  const int cc = (int)(idx - (long long)run * p.vecs) * VEC;  // channel over all heads
  const int h = cc / p.d, c = cc - h * p.d;
  const int t0 = run * kConvRun;
  float w[VEC][K], bias[VEC];
  load_weights<VEC, K>(p.weight, cc, w);
#pragma unroll
  for (int i = 0; i < VEC; ++i) bias[i] = p.bias ? __ldg(p.bias + cc + i) : 0.f;

  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int len = row_length(p.lengths, b, p.T);
    float win[K][VEC];  // inputs t-K+1 .. t
    const InT* xp = row_ptr<InT>(p.x, p.xs, b, h, 0, c);
    if (run == 0) {
      // The first run alone reads the old state and writes the new one, so the two
      // may be the same memory.
      float old[K - 1][VEC];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        if (p.state)
          load_vec<InT, VEC>(row_ptr<InT>(p.state, p.ss, b, h, j, c), old[j]);
        else
#pragma unroll
          for (int i = 0; i < VEC; ++i) old[j][i] = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) win[j + 1][i] = old[j][i];
      }
      if (p.state_T) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          const int e = len + j;  // entry of [state, x]
          float v[VEC];
          if (e >= K - 1) {
            load_vec<InT, VEC>(xp + (long long)(e - (K - 1)) * p.xs.t, v);
          } else {
#pragma unroll
            for (int q = 0; q < K - 1; ++q)
              if (q == e)
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = old[q][i];
          }
          store_vec<InT, VEC>(row_ptr<InT>(p.state_T, p.so, b, h, j, c), v);
        }
      }
    } else {
      if (t0 < len)
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          load_vec<InT, VEC>(xp + (long long)(t0 - (K - 1) + j) * p.xs.t, win[j + 1]);
    }
    OutT* yp = row_ptr<OutT>(p.y, p.ys, b, h, 0, c);
    if (p.pad_zero) {
      const float none[VEC] = {};
      const int end = t0 + kConvRun < p.T ? t0 + kConvRun : p.T;
      for (int t = len > t0 ? len : t0; t < end; ++t)
        store_vec<OutT, VEC>(yp + (long long)t * p.ys.t, none);
    }
    constexpr int NB = VEC == 8 ? 4 : 8;  // tokens loaded at a time
    for (int s = 0; s < kConvRun; s += NB) {
      const int ts = t0 + s;
      if (ts >= len) break;
      float in[NB][VEC];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        // behind the length: the last token again, unused
        const int t = ts + j < len ? ts + j : len - 1;
        load_vec<InT, VEC>(xp + (long long)t * p.xs.t, in[j]);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float out[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int q = 0; q < K - 1; ++q) win[q][i] = win[q + 1][i];
          win[K - 1][i] = in[j][i];
          float a = bias[i];
#pragma unroll
          for (int q = 0; q < K; ++q) a = fmaf(w[i][q], win[q][i], a);
          out[i] = p.silu ? a * sigmoid_fast(a) : a;
        }
        if (ts + j < len) store_vec<OutT, VEC>(yp + (long long)(ts + j) * p.ys.t, out);
      }
    }
  }
}

// ---- backward ----
// A thread walks a segment of kConvSeg tokens and K - 1 beyond it: the gradient
// before the activation at token t reaches dx at t - K + 1 .. t, so dx comes out
// K - 1 tokens late from a second window. A block is 32 vectors by 8 segments; the
// weight sums stay in registers along a segment and are added over the 8
// segments in shared memory, one partial sum per block in global memory, added in
// block order by reduce_parts_kernel (no atomics: the same bits on every call).
constexpr int kConvSeg = 32;
constexpr int kConvSegs = 8;

template <typename InT, typename OutT, int VEC, int K>
__global__ void __launch_bounds__(32 * kConvSegs) conv_bwd_kernel(const ConvParams p) {
  __shared__ float red[kConvSegs][32][VEC * (K + 1) + 1];
  const int lane = threadIdx.x, seg = threadIdx.y;
  const int vec = blockIdx.x * 32 + lane;
  const bool on = vec < p.vecs;
  const int cc = (on ? vec : 0) * VEC;
  const int h = cc / p.d, c = cc - h * p.d;
  const int tile = blockIdx.y;
  const int t0 = (tile * kConvSegs + seg) * kConvSeg;
  const long long D = (long long)p.H * p.d;
  float w[VEC][K], bias[VEC];
  load_weights<VEC, K>(p.weight, cc, w);
#pragma unroll
  for (int i = 0; i < VEC; ++i) bias[i] = p.bias ? __ldg(p.bias + cc + i) : 0.f;
  const RowStrides dxs = {(long long)p.H * p.T * p.d, (long long)p.T * p.d, p.d};
  const RowStrides dss = {(long long)p.H * (K - 1) * p.d, (long long)(K - 1) * p.d, p.d};

  for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
    const int len = row_length(p.lengths, b, p.T);
    float dw[VEC][K], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      db[i] = 0.f;
#pragma unroll
      for (int q = 0; q < K; ++q) dw[i][q] = 0.f;
    }
    if (on && (t0 < p.T || (tile == 0 && seg == 0))) {
      const InT* xp = row_ptr<InT>(p.x, p.xs, b, h, 0, c);
      const OutT* gp = row_ptr<OutT>(const_cast<const void*>(p.y), p.ys, b, h, 0, c);
      InT* dxp = row_ptr<InT>(p.dx, dxs, b, h, 0, c);
      const int end = t0 + kConvSeg < p.T ? t0 + kConvSeg : p.T;  // dx written up to here
      const bool first = t0 == 0;
      // inputs t0-K+1 .. t0-1 (0 behind the length, where nothing uses them)
      float win[K][VEC], dwin[K][VEC];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        if (t >= 0 && t < len) {
          load_vec<InT, VEC>(xp + (long long)t * p.xs.t, win[j + 1]);
        } else if (t < 0 && p.state) {
          load_vec<InT, VEC>(row_ptr<InT>(p.state, p.ss, b, h, t + K - 1, c), win[j + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) win[j + 1][i] = 0.f;
        }
      }
#pragma unroll
      for (int q = 0; q < K; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dwin[q][i] = 0.f;

      // one token: d(pre_t) into dwin (0 behind the length), its weight sums, and
      // dx at t - K + 1
      auto token = [&](int t, const float (&xin)[VEC], const float (&gin)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int q = 0; q < K - 1; ++q) {
            win[q][i] = win[q + 1][i];
            dwin[q][i] = dwin[q + 1][i];
          }
          win[K - 1][i] = xin[i];
          float g = gin[i];
          if (p.silu) {
            float a = bias[i];
#pragma unroll
            for (int q = 0; q < K; ++q) a = fmaf(w[i][q], win[q][i], a);
            const float sg = sigmoid_fast(a);
            g *= sg * fmaf(a, 1.f - sg, 1.f);
          }
          if (t >= len) g = 0.f;
          dwin[K - 1][i] = g;
          if (t >= end) g = 0.f;  // a later segment's token: its sums are there
          db[i] += g;
#pragma unroll
          for (int q = 0; q < K; ++q) dw[i][q] = fmaf(g, win[q][i], dw[i][q]);
        }
        const int e = t - (K - 1);  // the input whose gradient is complete now
        if (e >= end || (e < t0 && !(first && e < 0))) return;
        float out[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          out[i] = 0.f;
#pragma unroll
          for (int q = 0; q < K; ++q) out[i] = fmaf(w[i][K - 1 - q], dwin[q][i], out[i]);
        }
        const int js = e + (K - 1) - len;  // its place in state_T, if it has one
        if (p.dstate_T && js >= 0 && js < K - 1 && e < len) {
          float ds[VEC];
          load_vec<InT, VEC>(row_ptr<InT>(p.dstate_T, dss, b, h, js, c), ds);
#pragma unroll
          for (int i = 0; i < VEC; ++i) out[i] += ds[i];
        }
        if (e >= 0) {
          if (e >= len)
#pragma unroll
            for (int i = 0; i < VEC; ++i) out[i] = 0.f;
          store_vec<InT, VEC>(dxp + (long long)e * p.d, out);
        } else if (p.dstate) {
          store_vec<InT, VEC>(row_ptr<InT>(p.dstate, dss, b, h, e + K - 1, c), out);
        }
      };

      const int stop = end + K - 1;
      constexpr int NB = 4;  // tokens loaded at a time
      for (int ts = t0; ts < stop; ts += NB) {
        float xin[NB][VEC], gin[NB][VEC];
        if (ts < len) {
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int t = ts + j < len ? ts + j : len - 1;  // behind the length: unused
            load_vec<InT, VEC>(xp + (long long)t * p.xs.t, xin[j]);
            load_vec<OutT, VEC>(gp + (long long)t * p.ys.t, gin[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) xin[j][i] = gin[j][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) token(ts + j, xin[j], gin[j]);
      }
    }
    // partial sums of the block: over its segments in order
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int q = 0; q < K; ++q) red[seg][lane][i * K + q] = dw[i][q];
      red[seg][lane][VEC * K + i] = db[i];
    }
    __syncthreads();
    float* part = p.part + ((long long)b * p.tiles + tile) * (D * (K + 1));
    for (int i = seg * 32 + lane; i < 32 * VEC * (K + 1); i += 32 * kConvSegs) {
      // outputs ordered as in the partial sums: 32 VEC K weights, then 32 VEC biases
      const bool is_w = i < 32 * VEC * K;
      const int k = is_w ? i : i - 32 * VEC * K;
      const int per = is_w ? VEC * K : VEC;
      const int v = k / per, r = k - v * per;
      if (blockIdx.x * 32 + v < p.vecs) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kConvSegs; ++q) s += red[q][v][is_w ? r : VEC * K + r];
        part[(is_w ? 0 : D * K) + (long long)blockIdx.x * 32 * per + k] = s;
      }
    }
    __syncthreads();
  }
}

// ---- one token ----
template <typename InT, typename OutT, int VEC, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
  const int vec = blockIdx.x * 128 + threadIdx.x;
  if (vec >= p.vecs) return;
  const int cc = vec * VEC;
  const int h = cc / p.d, c = cc - h * p.d;
  float w[VEC][K];
  load_weights<VEC, K>(p.weight, cc, w);
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    float win[K][VEC], out[VEC];
    if (p.active && !p.active[b]) {
      if (p.pad_zero) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[i] = 0.f;
        store_vec<OutT, VEC>(row_ptr<OutT>(p.y, p.ys, b, h, 0, c), out);
      }
      continue;
    }
    InT* st = row_ptr<InT>(p.state_T, p.ss, b, h, 0, c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_vec<InT, VEC>(st + j * p.ss.t, win[j]);
    load_vec<InT, VEC>(row_ptr<InT>(p.x, p.xs, b, h, 0, c), win[K - 1]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float a = p.bias ? __ldg(p.bias + cc + i) : 0.f;
#pragma unroll
      for (int q = 0; q < K; ++q) a = fmaf(w[i][q], win[q][i], a);
      out[i] = p.silu ? a * sigmoid_fast(a) : a;
    }
    store_vec<OutT, VEC>(row_ptr<OutT>(p.y, p.ys, b, h, 0, c), out);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_vec<InT, VEC>(st + j * p.ss.t, win[j + 1]);
  }
}

}  // namespace ttt
