// Device helpers shared by the operators around the scan (convolution, selective
// scan, norm), and the launch of their fixed-order reductions.
#pragma once

#include "common.cuh"

namespace ttt {

// 2^x on the special-function unit: relative error at most 2^-22, denormal results are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Added to the exponent of a decay. For results in (0.7, 1) ex2 is low by 0.2 to 0.35 units of 2^-24
// on average (measured, 16384 decays in each of six ranges), which a state that lives for
// hundreds of tokens multiplies by their number: 1.5e-6 of it after 81 tokens, measured.
// With this the mean is within 0.11 units there, for the price of a multiply-add in the place of a
// multiplication; an exponent of 0 still gives 1.
constexpr float kDecayBias = 2.0e-8f;

// 1 / x on the special-function unit (2^-23); 1 / inf = 0, a denormal x counts as 0.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + exp(-x)) from one ex2 and one reciprocal; exp(-x) = inf gives 0. Off by up to 2^-21 of itself, and for
// x < 0, where exp(-x) counts in full, by |x| 2^-23 more: the exponent is a rounded product.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return rcp(1.0f + ex2(-kLog2e * x));
}

// log(1 + exp(x)), accurate in the relative sense also where it is small (a step size of
// 1e-3 needs log1p: 1 + e would keep 4 of its digits): off by 2^-21 of itself, and for x < 0 by |x| 2^-23
// more, from e's exponent, a rounded product. With e = exp(-|x|) it is
// max(x, 0) + log1p(e), and log1p(e) = 2 atanh(s) with s = e / (2 + e) <= 1/3:
// 2 s P(s^2), P the degree-4 polynomial through atanh(s) / s at the Chebyshev nodes of
// [0, 1/9] (7.6e-9 off in these constants). A third of log1pf's instructions.
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(-kLog2e * fabsf(x));
  const float s = e * rcp(2.0f + e), z = s * s;
  float p = fmaf(0.140788892f, z, 0.139825789f);
  p = fmaf(p, z, 0.200122976f);
  p = fmaf(p, z, 0.333331608f);
  p = fmaf(p, z, 1.0f);
  return fmaf(2.0f * s, p, fmaxf(x, 0.0f));
}

// Load VEC consecutive elements, widened to fp32. VEC > 1 needs the address
// aligned to VEC elements (16 bytes at most per access).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[VEC]) {
  if constexpr (VEC == 1) {
    out[0] = to_f32(p[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      out[i] = x.x; out[i + 1] = x.y; out[i + 2] = x.z; out[i + 3] = x.w;
    }
  } else {
    static_assert(VEC == 4 || VEC == 8, "bf16 vectors of 4 or 8");
    uint32_t w[VEC / 2];
    if constexpr (VEC == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
    static_assert(VEC == 4, "bf16 vectors of 4 or 8");
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
}

// VEC neighbouring elements of a row as they are in memory, in as few registers.
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 1> {
  float v;
  __device__ __forceinline__ void widen(float (&o)[1]) const { o[0] = v; }
};
template <>
struct Pack<float, 4> {
  float4 v;
  __device__ __forceinline__ void widen(float (&o)[4]) const {
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
  }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void widen(float (&o)[1]) const { o[0] = __uint_as_float((uint32_t)v << 16); }
};
template <>
struct Pack<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void widen(float (&o)[4]) const {
    o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xffff0000u);
    o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void widen(float (&o)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Pack<float, 8> {
  float4 v, w;
  __device__ __forceinline__ void widen(float (&o)[8]) const {
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    o[4] = w.x; o[5] = w.y; o[6] = w.z; o[7] = w.w;
  }
};

// VEC neighbouring channels in fp32, in pairs for the paired instructions where there are
// pairs (half the issue slots).
template <int VEC>
struct Lanes {
  float2 v[VEC / 2];
  __device__ __forceinline__ void set(float x) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = make_float2(x, x);
  }
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) { x[2 * i] = v[i].x; x[2 * i + 1] = v[i].y; }
  }
  // this += a b
  __device__ __forceinline__ void fma(const Lanes& a, const Lanes& b) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = __ffma2_rn(a.v[i], b.v[i], v[i]);
  }
  __device__ __forceinline__ void mul(const Lanes& a) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = __fmul2_rn(v[i], a.v[i]);
  }
  __device__ __forceinline__ void add(const Lanes& a) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = __fadd2_rn(v[i], a.v[i]);
  }
  // this -= a b
  __device__ __forceinline__ void fma_minus(const Lanes& a, const Lanes& b) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      v[i] = __ffma2_rn(make_float2(-a.v[i].x, -a.v[i].y), b.v[i], v[i]);
  }
  // 1 / (1 + exp(-this)), as sigmoid_fast
  __device__ __forceinline__ Lanes sigmoid() const {
    Lanes r;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 x = __fmul2_rn(v[i], make_float2(-kLog2e, -kLog2e));
      const float2 d = __fadd2_rn(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
      r.v[i] = make_float2(rcp(d.x), rcp(d.y));
    }
    return r;
  }
};
template <>
struct Lanes<1> {
  float v;
  __device__ __forceinline__ void set(float x) { v = x; }
  __device__ __forceinline__ void set(const float (&x)[1]) { v = x[0]; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = v; }
  __device__ __forceinline__ void fma(const Lanes& a, const Lanes& b) { v = fmaf(a.v, b.v, v); }
  __device__ __forceinline__ void fma_minus(const Lanes& a, const Lanes& b) { v = fmaf(-a.v, b.v, v); }
  __device__ __forceinline__ void mul(const Lanes& a) { v *= a.v; }
  __device__ __forceinline__ void add(const Lanes& a) { v += a.v; }
  __device__ __forceinline__ Lanes sigmoid() const { return {sigmoid_fast(v)}; }
};

// Sum of `parts` rows of n floats in an order that `parts` and n fix: the same bits on every
// call. Column i goes to the segment that holds it (up to three outputs laid end to end); a
// null output is skipped.
struct ReduceOut {
  float* p[3];
  long long n[3];
};

// Defined in conv.cu.
int launch_reduce_parts(const float* part, int parts, long long n, const ReduceOut& out,
                        cudaStream_t stream);

}  // namespace ttt
