// Short causal convolution, depthwise over K = 2..4 tokens: prompt, backward and
// one-token step (include/ttt_conv.h has the formulas).
//
// Every kernel is one pass over the tokens: K multiply-adds and one SiLU per element
// against one read and one write, so HBM bounds it. A thread owns four neighbouring channels
// (one where rows do not allow packs), in fp32 pairs, and walks a run of tokens with the last inputs in
// registers, so an input is read from memory once (and K - 1 tokens again at the
// start of a run, from cache), while the next batch of loads is under way.
//
// Measured, K = 4: 2 x 32768 tokens by 2048 channels into heads in bf16 105 us (537 MB: 78 % of the copy
// bandwidth; with batches of 4 tokens 110 us), in fp32 203 us (1074 MB: 81 %; two batches of 8 packs of fp32 do not fit
// 96 registers, up to 192 bytes a thread are spilled); forward and backward of 8 x 4096 tokens by 768 channels, ragged,
// bf16, 71 us, of which the backward's kernel 48 us: its windows, weights and weight sums take 128
// registers (and spill 16 bytes, in fp32 208), so 16 warps an SM, and latency is what is left (in fp32 the
// backward takes 99 us for 302 MB); one token for 512 rows of 2048 channels 5.5 us, 6.3 us with inputs and states out of HBM.
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
  int run;              // tokens per run (forward)
  int seg;              // tokens per segment (backward)
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

// The VEC channels' weights, w[j] of tap j. The VEC K floats are one contiguous run that starts
// on 16 bytes when VEC is 4.
template <int VEC, int K>
__device__ __forceinline__ void load_weights(const float* weight, int c, Lanes<VEC> (&w)[K]) {
  const float* p = weight + (size_t)c * K;
  float f[VEC * K];
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < VEC * K; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC * K; ++i) f[i] = __ldg(p + i);
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float t[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] = f[i * K + j];
    w[j].set(t);
  }
}

template <int VEC>
__device__ __forceinline__ Lanes<VEC> load_bias(const float* bias, int c) {
  float t[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) t[i] = bias ? __ldg(bias + c + i) : 0.f;
  Lanes<VEC> r;
  r.set(t);
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ Lanes<VEC> widened(const Pack<T, VEC>& x) {
  float t[VEC];
  x.widen(t);
  Lanes<VEC> r;
  r.set(t);
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ Lanes<VEC> load_lanes(const T* p) {
  float t[VEC];
  load_vec<T, VEC>(p, t);
  Lanes<VEC> r;
  r.set(t);
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_lanes(T* p, const Lanes<VEC>& x) {
  float t[VEC];
  x.get(t);
  store_vec<T, VEC>(p, t);
}

__device__ __forceinline__ int row_length(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

constexpr int kConvBatch = 8;  // tokens loaded at a time (forward)

// Linear thread index over (run, vector) in x, batch rows in y. p.run tokens a thread: 32 where
// that leaves 16 warps for every SM, else 8 (short prompts, few channels).
template <typename InT, typename OutT, int VEC, int K>
__global__ void __launch_bounds__(128, 5) conv_fwd_kernel(const ConvParams p) {
  using V = Lanes<VEC>;
  const long long idx = (long long)blockIdx.x * 128 + threadIdx.x;
  const int run = (int)(idx / p.vecs);
  if (run >= p.tiles) return;
  const int cc = (int)(idx - (long long)run * p.vecs) * VEC;  // channel over all heads
  const int h = cc / p.d, c = cc - h * p.d;
  const int t0 = run * p.run;
  V w[K];
  load_weights<VEC, K>(p.weight, cc, w);
  const V bias = load_bias<VEC>(p.bias, cc);
  V zero;
  zero.set(0.f);

  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int len = row_length(p.lengths, b, p.T);
    const int end = t0 + p.run < len ? t0 + p.run : len;
    V win[4];  // the last inputs, that of token t at (t - t0) & 3: the batches turn it in place
    const InT* xp = row_ptr<InT>(p.x, p.xs, b, h, t0, c);
    OutT* yp = row_ptr<OutT>(p.y, p.ys, b, h, t0, c);
    if (run == 0) {
      // The first run alone reads the old state and writes the new one, so the two
      // may be the same memory.
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        win[(j - (K - 1)) & 3] =
            p.state ? load_lanes<InT, VEC>(row_ptr<InT>(p.state, p.ss, b, h, j, c)) : zero;
      if (p.state_T) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          const int e = len + j;  // entry of [state, x]
          V v = zero;
          if (e >= K - 1) {
            v = load_lanes<InT, VEC>(xp + (long long)(e - (K - 1)) * p.xs.t);
          } else {
#pragma unroll
            for (int q = 0; q < K - 1; ++q)
              if (q == e) v = win[(q - (K - 1)) & 3];
          }
          store_lanes<InT, VEC>(row_ptr<InT>(p.state_T, p.so, b, h, j, c), v);
        }
      }
    } else if (t0 < len) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        win[(j - (K - 1)) & 3] = load_lanes<InT, VEC>(xp + (long long)(j - (K - 1)) * p.xs.t);
    }
    if (p.pad_zero) {
      const int stop = t0 + p.run < p.T ? t0 + p.run : p.T;
      for (int t = len > t0 ? len : t0; t < stop; ++t)
        store_lanes<OutT, VEC>(yp + (long long)(t - t0) * p.ys.t, zero);
    }
    // the next batch is on its way while this one is worked on
    Pack<InT, VEC> next[kConvBatch];
    auto fetch = [&](int left) {
#pragma unroll
      for (int j = 0; j < kConvBatch; ++j)
        if (j < left) next[j] = *reinterpret_cast<const Pack<InT, VEC>*>(xp + (long long)j * p.xs.t);
      xp += kConvBatch * p.xs.t;
    };
    fetch(end - t0);
    for (int t = t0; t < end; t += kConvBatch) {
      const int left = end - t;
      Pack<InT, VEC> in[kConvBatch];
#pragma unroll
      for (int j = 0; j < kConvBatch; ++j) in[j] = next[j];
      fetch(left - kConvBatch);
#pragma unroll
      for (int j = 0; j < kConvBatch; ++j) {
        win[j & 3] = widened<InT, VEC>(in[j]);
        V a = bias;
#pragma unroll
        for (int q = 0; q < K; ++q) a.fma(w[q], win[(j - (K - 1) + q) & 3]);
        if (p.silu) a.mul(a.sigmoid());
        if (j < left) store_lanes<OutT, VEC>(yp + (long long)j * p.ys.t, a);
      }
      yp += kConvBatch * p.ys.t;
    }
  }
}

// ---- backward ----
// A thread walks a segment of p.seg tokens and K - 1 beyond it: the gradient
// before the activation at token t reaches dx at t - K + 1 .. t, so dx comes out
// K - 1 tokens late from a second window. A block is 32 vectors by 8 segments; the
// weight sums stay in registers along a segment and are added over the 8
// segments in shared memory, one partial sum per block in global memory, added in
// block order by reduce_parts_kernel (no atomics: the same bits on every call).
constexpr int kConvSegs = 8;

template <typename InT, typename OutT, int VEC, int K>
__global__ void __launch_bounds__(32 * kConvSegs, 2) conv_bwd_kernel(const ConvParams p) {
  using V = Lanes<VEC>;
  __shared__ float red[kConvSegs][32][VEC * (K + 1) + 1];
  const int lane = threadIdx.x, seg = threadIdx.y;
  const int vec = blockIdx.x * 32 + lane;
  const bool on = vec < p.vecs;
  const int cc = (on ? vec : 0) * VEC;
  const int h = cc / p.d, c = cc - h * p.d;
  const int tile = blockIdx.y;
  const int t0 = (tile * kConvSegs + seg) * p.seg;
  const long long D = (long long)p.H * p.d;
  V w[K], zero;
  load_weights<VEC, K>(p.weight, cc, w);
  const V bias = load_bias<VEC>(p.bias, cc);
  zero.set(0.f);
  const RowStrides dxs = {(long long)p.H * p.T * p.d, (long long)p.T * p.d, p.d};
  const RowStrides dss = {(long long)p.H * (K - 1) * p.d, (long long)(K - 1) * p.d, p.d};

  for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
    const int len = row_length(p.lengths, b, p.T);
    V dw[K], db = zero;
#pragma unroll
    for (int q = 0; q < K; ++q) dw[q] = zero;
    if (on && (t0 < p.T || (tile == 0 && seg == 0))) {
      const InT* xp = row_ptr<InT>(p.x, p.xs, b, h, t0, c);
      const OutT* gp = row_ptr<OutT>(const_cast<const void*>(p.y), p.ys, b, h, t0, c);
      InT* dxp = row_ptr<InT>(p.dx, dxs, b, h, t0, c);
      const int end = t0 + p.seg < p.T ? t0 + p.seg : p.T;  // dx written up to here
      const bool first = t0 == 0;
      // inputs t0-K+1 .. t0-1 (0 behind the length, where nothing uses them)
      V win[4], dwin[4];  // of token t at (t - t0) & 3
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        if (t >= 0 && t < len)
          win[(j - (K - 1)) & 3] = load_lanes<InT, VEC>(xp + (long long)(j - (K - 1)) * p.xs.t);
        else if (t < 0 && p.state)
          win[(j - (K - 1)) & 3] =
              load_lanes<InT, VEC>(row_ptr<InT>(p.state, p.ss, b, h, t + K - 1, c));
        else
          win[(j - (K - 1)) & 3] = zero;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) dwin[q] = zero;

      // Token t = ts + j: d(pre_t) into dwin, its weight sums, and dx at t - K + 1. `inner`: t lies
      // in the segment and in the length, and t - K + 1 in the segment; else what lies
      // behind the length is 0, and a later segment's token leaves its sums to it.
      auto token = [&](int t, int j, const V& xin, V g, bool inner) {
        win[j & 3] = xin;
        if (p.silu) {
          V a = bias;
#pragma unroll
          for (int q = 0; q < K; ++q) a.fma(w[q], win[(j - (K - 1) + q) & 3]);
          const V sg = a.sigmoid();
          // SiLU'(a) = s (1 + a (1 - s)): 1 - s is exact where a is large, and s + a s - a s s is not
          V rest, d;
          rest.set(1.f);
          d.set(1.f);
          rest.fma_minus(sg, d);
          d.fma(a, rest);
          d.mul(sg);
          g.mul(d);
        }
        if (!inner && t >= len) g = zero;
        dwin[j & 3] = g;
        // (not as a product with 0: the window may hold an infinite input)
        if (inner || (t < len && t < end)) {
          db.add(g);
#pragma unroll
          for (int q = 0; q < K; ++q) dw[q].fma(g, win[(j - (K - 1) + q) & 3]);
        }
        const int e = t - (K - 1);  // the input whose gradient is complete now
        if (!inner && (e >= end || (e < t0 && !(first && e < 0)))) return;
        V out = w[K - 1];
        out.mul(dwin[(j - (K - 1)) & 3]);
#pragma unroll
        for (int q = 1; q < K; ++q) out.fma(w[K - 1 - q], dwin[(j - (K - 1) + q) & 3]);
        if (inner) {
          store_lanes<InT, VEC>(dxp + (long long)(e - t0) * p.d, out);
          return;
        }
        const int js = e + (K - 1) - len;  // its place in state_T, if it has one
        if (p.dstate_T && js >= 0 && js < K - 1 && e < len)
          out.add(load_lanes<InT, VEC>(row_ptr<InT>(p.dstate_T, dss, b, h, js, c)));
        if (e >= 0) {
          if (e >= len) out = zero;
          store_lanes<InT, VEC>(dxp + (long long)(e - t0) * p.d, out);
        } else if (p.dstate) {
          store_lanes<InT, VEC>(row_ptr<InT>(p.dstate, dss, b, h, e + K - 1, c), out);
        }
      };

      const int stop = end + K - 1;
      constexpr int NB = 4;  // tokens loaded at a time; the next ones while these are worked on
      Pack<InT, VEC> xnext[NB];
      Pack<OutT, VEC> gnext[NB];
      auto fetch = [&](int left) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (j < left) {
            xnext[j] = *reinterpret_cast<const Pack<InT, VEC>*>(xp + (long long)j * p.xs.t);
            gnext[j] = *reinterpret_cast<const Pack<OutT, VEC>*>(gp + (long long)j * p.ys.t);
          } else {
            xnext[j] = {};
            gnext[j] = {};
          }
        }
        xp += NB * p.xs.t;
        gp += NB * p.ys.t;
      };
      const int seen = stop < len ? stop : len;   // no token is needed from here on
      const int inner = end < len ? end : len;
      fetch(seen - t0);
      for (int ts = t0; ts < stop; ts += NB) {
        Pack<InT, VEC> xin[NB];
        Pack<OutT, VEC> gin[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          xin[j] = xnext[j];
          gin[j] = gnext[j];
        }
        fetch(seen - ts - NB);
        if (ts > t0 && ts + NB <= inner) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
            token(ts + j, j, widened<InT, VEC>(xin[j]), widened<OutT, VEC>(gin[j]), true);
        } else {
#pragma unroll
          for (int j = 0; j < NB; ++j)
            token(ts + j, j, widened<InT, VEC>(xin[j]), widened<OutT, VEC>(gin[j]), false);
        }
      }
    }
    // partial sums of the block: over its segments in order
#pragma unroll
    for (int q = 0; q < K; ++q) {
      float f[VEC];
      dw[q].get(f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) red[seg][lane][i * K + q] = f[i];
    }
    {
      float f[VEC];
      db.get(f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) red[seg][lane][VEC * K + i] = f[i];
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
  using V = Lanes<VEC>;
  const int vec = blockIdx.x * 128 + threadIdx.x;
  if (vec >= p.vecs) return;
  const int cc = vec * VEC;
  const int h = cc / p.d, c = cc - h * p.d;
  V w[K];
  load_weights<VEC, K>(p.weight, cc, w);
  const V bias = load_bias<VEC>(p.bias, cc);
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    OutT* yp = row_ptr<OutT>(p.y, p.ys, b, h, 0, c);
    if (p.active && !p.active[b]) {
      if (p.pad_zero) {
        V zero;
        zero.set(0.f);
        store_lanes<OutT, VEC>(yp, zero);
      }
      continue;
    }
    V win[K], a = bias;
    InT* st = row_ptr<InT>(p.state_T, p.ss, b, h, 0, c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j] = load_lanes<InT, VEC>(st + j * p.ss.t);
    win[K - 1] = load_lanes<InT, VEC>(row_ptr<InT>(p.x, p.xs, b, h, 0, c));
#pragma unroll
    for (int q = 0; q < K; ++q) a.fma(w[q], win[q]);
    if (p.silu) a.mul(a.sigmoid());
    store_lanes<OutT, VEC>(yp, a);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_lanes<InT, VEC>(st + j * p.ss.t, win[j + 1]);
  }
}

}  // namespace ttt
