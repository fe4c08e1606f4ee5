// Root-mean-square norm with the residual's addition (include/ttt_norm.h).
//
// One read of x and the residual, one write of s and y: HBM bounds it. A row stays in
// registers between its sum of squares and its output. In the vector form a
// lane holds VPT groups of 8 neighbouring columns and a row takes W warps; rows of
// up to 1024 columns fit one warp, which then needs no barrier at all, and four
// such rows share a CTA. Rows whose pointers or strides are off 16 bytes, or
// with D not a multiple of 8, take the same kernel with single columns, at about half the speed in bf16.
//
// Measured, bf16: 65536 rows of 2048 in 8 bits, a scale for each 128 columns, 150 us (944 MB: 96 % of the copy
// bandwidth; 164 in a long run of calls); 32768 rows of 1536 forward 61 us (403 MB: 101 %, part of it still in L2) and
// backward 72 us and 8 us for the sum of the weight gradients' parts; the same with 1535 columns 115 us, in 8 bits 158
// (69 at 1536), backward 133. fp32, 32768 rows of 1536: 121 and 124 us. 64 rows of 2048 in 8 bits 3.9 us. The backward
// spills where a row takes more registers than its CTA leaves: 104 bytes a thread in fp32 beyond 2048 columns, 112 in
// single columns, 376 to 840 beyond 8192, where 1024 threads have 64 registers (4096 rows of 16384, bf16: 371 us,
// 82 for its bytes).
#pragma once

#include <cuda_fp8.h>
#include <type_traits>

#include "seq_common.cuh"

namespace ttt {

struct NormParams {
  const void* x;
  const void* residual;  // or null
  const float* weight;
  void* y;
  void* s;               // or null
  float* scale;          // 8-bit output
  long long x_ld, r_ld, y_ld, s_ld;
  int M, D;
  int W;                 // warps per row
  int groups;            // scales per row
  int group128;          // a scale for each 128 columns, else one for the row
  float eps;
};

struct NormBwdParams {
  const void* dy;
  const void* s;
  const float* weight;
  const void* ds;        // or null
  void* dx;
  float* part;           // [CTAs][D] partial sums of dweight
  long long dy_ld, s_ld, ds_ld, dx_ld;
  int M, D;
  int W;
  float eps;
};

struct E4M3 {};  // 8-bit output

// The larger number; NaN where one of them is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// x / scale, rounded once, for many x and one scale. The product with 1 / scale alone is an fp32 rounding
// off and takes two codes in a million to the other side of the middle between two; corrected
// by its exact remainder it is the quotient (P. Markstein, IBM J. Res. Dev. 34, 1990: y = 1 / scale correctly
// rounded, q = x y, q - (q scale - x) y) for two more paired multiply-adds: 65536 rows of 2048 take 150 us, with the
// product alone 148, with divisions 164 (single columns divide). The remainder of small numbers is not
// exact, so scales below 2^-80, and those that are no numbers, divide.
struct Quotients {
  float scale, y;
  bool plain;
  __device__ __forceinline__ explicit Quotients(float s)
      : scale(s), y(1.0f / s), plain(s >= 0x1p-80f && s <= 3.402823466e38f) {}
  __device__ __forceinline__ float2 operator()(float2 x) const {
    if (!plain) return make_float2(x.x / scale, x.y / scale);
    const float2 y2 = make_float2(y, y), q = __fmul2_rn(x, y2);
    const float2 over = __ffma2_rn(q, make_float2(scale, scale), make_float2(-x.x, -x.y));
    return __ffma2_rn(over, make_float2(-y, -y), q);  // (in these signs, -0 stays -0)
  }
};

// Columns of a lane: VEC neighbouring ones at column(v), v = 0 .. VPT - 1. The VPT
// vectors of a warp are neighbours, so that 128 columns are either 16 lanes of
// one vector (VEC = 8) or 4 vectors of all lanes (VEC = 1).
template <int VEC, int VPT>
__device__ __forceinline__ int norm_column(int warp, int lane, int v) {
  return ((warp * VPT + v) * 32 + lane) * VEC;
}

template <typename XT, typename RT, typename YT, int VEC, int VPT>
__device__ __forceinline__ void norm_fwd(const NormParams& p) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31;
  const int warp = (threadIdx.x >> 5) % p.W, sub = (threadIdx.x >> 5) / p.W;
  const int rows_per_cta = (blockDim.x >> 5) / p.W;  // more than one only with W = 1
  const long long row = (long long)blockIdx.x * rows_per_cta + sub;
  if (row >= p.M) return;                            // whole warps; W > 1 has one row a CTA
  const XT* xp = static_cast<const XT*>(p.x) + row * p.x_ld;
  const RT* rp = static_cast<const RT*>(p.residual) + row * p.r_ld;
  float s[VPT][VEC];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = norm_column<VEC, VPT>(warp, lane, v);
    if (c < p.D) {
      load_vec<XT, VEC>(xp + c, s[v]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[v][i] = 0.f;
    }
  }
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
      float r[VEC];
      if (c < p.D) {
        load_vec<RT, VEC>(rp + c, r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[v][i] += r[i];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(s[v][i], s[v][i], ss);
  ss = warp_sum(ss);
  if (p.W > 1) {
    if (lane == 0) red[0][warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < p.W; ++w) ss += red[0][w];
  }
  const float rs = rsqrtf(ss / (float)p.D + p.eps);
  if (p.s) {
    RT* sp = static_cast<RT*>(p.s) + row * p.s_ld;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
      if (c < p.D) store_vec<RT, VEC>(sp + c, s[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = norm_column<VEC, VPT>(warp, lane, v);
    if (c < p.D) {
      float w[VEC];
      load_vec<float, VEC>(p.weight + c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[v][i] = s[v][i] * rs * w[i];
    }
  }

  if constexpr (!std::is_same<YT, E4M3>::value) {
    YT* yp = static_cast<YT*>(p.y) + row * p.y_ld;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
      if (c < p.D) store_vec<YT, VEC>(yp + c, s[v]);
    }
  } else {
    float amax[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      amax[v] = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) amax[v] = max_nan(amax[v], fabsf(s[v][i]));
    }
    if (!p.group128) {
      float m = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) m = max_nan(m, amax[v]);
      m = warp_max(m);
      if (p.W > 1) {
        if (lane == 0) red[1][warp] = m;
        __syncthreads();
        m = 0.f;
        for (int w = 0; w < p.W; ++w) m = max_nan(m, red[1][w]);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) amax[v] = m;
    } else if constexpr (VEC == 8) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
          amax[v] = max_nan(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], off));
    } else {
      static_assert(VEC == 8 || VPT % 4 == 0, "whole groups of 128 columns");
#pragma unroll
      for (int v = 0; v < VPT; v += 4) {
        const float m = warp_max(max_nan(max_nan(amax[v], amax[v + 1]), max_nan(amax[v + 2], amax[v + 3])));
        amax[v] = amax[v + 1] = amax[v + 2] = amax[v + 3] = m;
      }
    }
    unsigned char* yp = static_cast<unsigned char*>(p.y) + row * p.y_ld;
    float* sc = p.scale + row * p.groups;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
      if (c >= p.D) continue;
      // At least the smallest normal number: a row of zeros stays dividable. NaN stays NaN.
      const float scale = max_nan(amax[v] / 448.f, 1.17549435e-38f);
      if (p.group128 ? c % 128 == 0 : c == 0) sc[p.group128 ? c / 128 : 0] = scale;
      if constexpr (VEC == 8) {
        const Quotients by(scale);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = __nv_cvt_float2_to_fp8x2(by(make_float2(s[v][2 * i], s[v][2 * i + 1])), __NV_SATFINITE,
                                          __NV_E4M3);
        *reinterpret_cast<uint2*>(yp + c) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
      } else {
        yp[c] = __nv_cvt_float_to_fp8(s[v][0] / scale, __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

// The entries hold the registers to what the largest launch may have: a row of 16384 columns takes 16 warps of
// four vectors a lane, or 32 warps of single columns.
// Four vectors a lane otherwise take a few registers more than 64 (65536 rows of 2048: bf16 183 us, so 157;
// in 8 bits 158, so 150). Single columns are at most 48: 32768 rows of 1535 in bf16 115 us and in 8 bits 158; with 64,
// loads are brought forward at the price of warps, 122 and 165.
template <typename XT, typename RT, typename YT, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 256, VPT == 4 ? 2 : 0) norm_fwd_kernel(const NormParams p) {
  norm_fwd<XT, RT, YT, 8, VPT>(p);
}
template <typename XT, typename RT, typename YT>
__global__ void __maxnreg__(48) norm_fwd_single_kernel(const NormParams p) {
  norm_fwd<XT, RT, YT, 1, 16>(p);
}

// Backward. A CTA of W warps walks rows blockIdx.x, blockIdx.x + gridDim.x, ..., one at
// a time, with the weight gradients of its columns in registers; they go out as one
// row of partial sums per CTA and are added by reduce_parts_kernel. MAXT bounds the
// CTA (a row of 16384 columns takes 1024 threads, which leaves 64 registers each).
template <typename GT, typename ST, int VEC, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) norm_bwd_kernel(const NormBwdParams p) {
  __shared__ float2 red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[VPT][VEC], dw[VPT][VEC];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = norm_column<VEC, VPT>(warp, lane, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[v][i] = dw[v][i] = 0.f;
    if (c < p.D) load_vec<float, VEC>(p.weight + c, w[v]);
  }
  // The next row's numbers are on their way while this one's are worked on.
  Pack<GT, VEC> gn[VPT];
  Pack<ST, VEC> sn[VPT], en[VPT];
  auto fetch = [&](long long row) {
    const GT* gp = static_cast<const GT*>(p.dy) + row * p.dy_ld;
    const ST* sp = static_cast<const ST*>(p.s) + row * p.s_ld;
    const ST* ep = static_cast<const ST*>(p.ds) + row * p.ds_ld;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
      gn[v] = {};
      sn[v] = en[v] = {};
      if (c < p.D) {
        gn[v] = *reinterpret_cast<const Pack<GT, VEC>*>(gp + c);
        sn[v] = *reinterpret_cast<const Pack<ST, VEC>*>(sp + c);
        if (p.ds) en[v] = *reinterpret_cast<const Pack<ST, VEC>*>(ep + c);
      }
    }
  };
  int buf = 0;
  if (blockIdx.x < p.M) fetch(blockIdx.x);
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
    ST* op = static_cast<ST*>(p.dx) + row * p.dx_ld;
    float g[VPT][VEC], s[VPT][VEC], e[VPT][VEC];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      gn[v].widen(g[v]);
      sn[v].widen(s[v]);
      en[v].widen(e[v]);
    }
    if (row + gridDim.x < p.M) fetch(row + gridDim.x);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(s[v][i], s[v][i], ss);
        dot = fmaf(w[v][i] * g[v][i], s[v][i], dot);
      }
    ss = warp_sum(ss);
    dot = warp_sum(dot);
    if (p.W > 1) {
      if (lane == 0) red[buf][warp] = make_float2(ss, dot);
      __syncthreads();  // two buffers: the next row's sums cannot meet a reader of these
      ss = dot = 0.f;
      for (int k = 0; k < p.W; ++k) {
        ss += red[buf][k].x;
        dot += red[buf][k].y;
      }
    }
    const float rs = rsqrtf(ss / (float)p.D + p.eps);
    const float k = dot / (float)p.D * rs * rs;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = norm_column<VEC, VPT>(warp, lane, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[v][i] = fmaf(g[v][i], s[v][i] * rs, dw[v][i]);
        e[v][i] = fmaf(rs, fmaf(w[v][i], g[v][i], -s[v][i] * k), e[v][i]);
      }
      if (c < p.D) store_vec<ST, VEC>(op + c, e[v]);
    }
  }
  float* part = p.part + (size_t)blockIdx.x * p.D;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = norm_column<VEC, VPT>(warp, lane, v);
    if (c < p.D) store_vec<float, VEC>(part + c, dw[v]);
  }
}

}  // namespace ttt
