// C-ABI entry points of the root-mean-square norm (include/ttt_norm.h): argument
// checks, how a row is spread over warps, launches.
#include <cmath>
#include <type_traits>

#include "ttt_norm.h"
#include "abi_util.h"
#include "launch.h"
#include "norm.cuh"

namespace {

using ttt::NormBwdParams;
using ttt::NormParams;
using ttt::abi::misaligned;
using ttt::abi::misaligned_to;
using ttt::abi::Span;
using ttt::abi::Strided;

constexpr unsigned kKnownModes = TTT_IN_BF16 | TTT_OUT_BF16 | TTT_NORM_SUM_BF16 | TTT_NORM_Y_E4M3;
constexpr int kMaxD = 16384;
constexpr int kRowsPerCta = 4;     // rows of one warp each
constexpr int kBwdCtasMax = 1184;  // CTAs of the backward, at most (8 per SM of 148)

bool finite_eps(float eps) { return eps >= 0.0f && std::isfinite(eps); }

// Vectors of 8 columns: every pointer on 16 bytes (8 bytes of codes for the 8-bit
// output), every row stride a multiple of 8.
bool vec_ok(const void* p, size_t elt, long long ld, int M) {
  return !p || (!misaligned_to(p, elt * 8 < 16 ? elt * 8 : 16) && (M <= 1 || ld % 8 == 0));
}

template <typename XT, typename RT, typename YT, int VEC, int VPT>
int launch_fwd(NormParams p, cudaStream_t s) {
  const int per_warp = VEC * VPT * 32;
  p.W = (p.D + per_warp - 1) / per_warp;
  const int rows = p.W == 1 ? kRowsPerCta : 1;
  const unsigned blocks = (unsigned)(((long long)p.M + rows - 1) / rows);
  if constexpr (VEC == 1)
    ttt::norm_fwd_single_kernel<XT, RT, YT><<<blocks, 32 * p.W * rows, 0, s>>>(p);
  else
    ttt::norm_fwd_kernel<XT, RT, YT, VPT><<<blocks, 32 * p.W * rows, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename XT, typename RT, typename YT>
int dispatch_shape(const NormParams& p, bool vec, cudaStream_t s) {
  if (!vec) return launch_fwd<XT, RT, YT, 1, 16>(p, s);
  if (p.D <= 256) return launch_fwd<XT, RT, YT, 8, 1>(p, s);
  if (p.D <= 512) return launch_fwd<XT, RT, YT, 8, 2>(p, s);
  if (p.D <= 1024) return launch_fwd<XT, RT, YT, 8, 4>(p, s);
  // Longer rows take several warps: of 512 columns where that leaves fewer lanes idle than 1024 (1536
  // columns, 32768 rows of bf16: 60.6 against 61.4 us, in 8 bits 67.8 against 69.6), else of 1024 (2048 columns in 8
  // bits, 65536 rows: 150 against 169 us).
  const int w512 = (p.D + 511) / 512, w1024 = (p.D + 1023) / 1024;
  if (w512 < 2 * w1024 && w512 <= 8) return launch_fwd<XT, RT, YT, 8, 2>(p, s);
  return launch_fwd<XT, RT, YT, 8, 4>(p, s);
}

template <typename XT, typename RT>
int dispatch_y(const NormParams& p, unsigned mode, bool vec, cudaStream_t s) {
  if (mode & TTT_NORM_Y_E4M3) return dispatch_shape<XT, RT, ttt::E4M3>(p, vec, s);
  if (mode & TTT_OUT_BF16) return dispatch_shape<XT, RT, __nv_bfloat16>(p, vec, s);
  return dispatch_shape<XT, RT, float>(p, vec, s);
}

template <typename XT>
int dispatch_r(const NormParams& p, unsigned mode, bool vec, cudaStream_t s) {
  return (mode & TTT_NORM_SUM_BF16) ? dispatch_y<XT, __nv_bfloat16>(p, mode, vec, s)
                                    : dispatch_y<XT, float>(p, mode, vec, s);
}

int bwd_ctas(int M) { return M < kBwdCtasMax ? M : kBwdCtasMax; }

template <typename GT, typename ST, int VEC, int VPT, int MAXT>
int launch_bwd(NormBwdParams p, cudaStream_t s) {
  const int per_warp = VEC * VPT * 32;
  p.W = (p.D + per_warp - 1) / per_warp;
  ttt::norm_bwd_kernel<GT, ST, VEC, VPT, MAXT><<<bwd_ctas(p.M), 32 * p.W, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename GT, typename ST>
int dispatch_bwd_shape(const NormBwdParams& p, bool vec, cudaStream_t s) {
  if (!vec)
    return p.D <= 8192 ? launch_bwd<GT, ST, 1, 16, 512>(p, s) : launch_bwd<GT, ST, 1, 16, 1024>(p, s);
  if (p.D <= 2048) return launch_bwd<GT, ST, 8, 1, 256>(p, s);
  return p.D <= 8192 ? launch_bwd<GT, ST, 8, 2, 512>(p, s) : launch_bwd<GT, ST, 8, 2, 1024>(p, s);
}

template <typename GT>
int dispatch_bwd(const NormBwdParams& p, unsigned mode, bool vec, cudaStream_t s) {
  return (mode & TTT_NORM_SUM_BF16) ? dispatch_bwd_shape<GT, __nv_bfloat16>(p, vec, s)
                                    : dispatch_bwd_shape<GT, float>(p, vec, s);
}

Strided rows(int M, long long ld, int D, size_t elt) { return {{M, 1, 1}, {ld, 0, 0}, D, elt}; }

bool short_rows(const long long* strides, int M, int D) {
  if (!strides || M <= 1) return false;
  for (int i = 0; i < 4; ++i)
    if (strides[i] < D) return true;
  return false;
}

}  // namespace

extern "C" {

int ttt_norm_forward(const void* x, const void* residual, const float* weight, int M, int D,
                     float eps, unsigned mode, int group, const long long* strides, void* y,
                     void* s, float* scale, void* cuda_stream) {
  if (mode & ~kKnownModes) return TTT_ERR_INVALID_ARG;
  const bool e4m3 = mode & TTT_NORM_Y_E4M3;
  if (e4m3 && (mode & TTT_OUT_BF16)) return TTT_ERR_INVALID_ARG;
  if (M < 0 || D < 1 || !finite_eps(eps)) return TTT_ERR_INVALID_ARG;
  if ((group != 0 && group != 128) || (group && !e4m3)) return TTT_ERR_INVALID_ARG;
  if (M > 0 && (!x || !weight || !y || (e4m3 && !scale))) return TTT_ERR_INVALID_ARG;
  if ((scale && !e4m3) || (s && !residual)) return TTT_ERR_INVALID_ARG;
  if (short_rows(strides, M, D)) return TTT_ERR_INVALID_ARG;
  const size_t xe = (mode & TTT_IN_BF16) ? 2 : 4, re = (mode & TTT_NORM_SUM_BF16) ? 2 : 4;
  const size_t ye = e4m3 ? 1 : (mode & TTT_OUT_BF16) ? 2 : 4;
  if (misaligned_to(x, xe) || misaligned_to(residual, re) || misaligned_to(s, re) ||
      misaligned_to(y, ye) || misaligned_to(weight, 4) || misaligned_to(scale, 4))
    return TTT_ERR_INVALID_ARG;
  if (D > kMaxD) return TTT_ERR_UNSUPPORTED;
  NormParams p{};
  p.x_ld = strides ? strides[0] : D;
  p.r_ld = strides ? strides[1] : D;
  p.y_ld = strides ? strides[2] : D;
  p.s_ld = strides ? strides[3] : D;
  // s over the residual, or over x where both have its type, row for row
  const bool over_r = s && s == residual, over_x = s && s == x;
  if ((over_r && p.s_ld != p.r_ld) || (over_x && (p.s_ld != p.x_ld || xe != re)))
    return TTT_ERR_INVALID_ARG;
  const int groups = group ? (D + 127) / 128 : 1;
  const Span in[] = {{over_x ? nullptr : x, rows(M, p.x_ld, D, xe).extent()},
                     {over_r ? nullptr : residual, rows(M, p.r_ld, D, re).extent()},
                     {weight, (size_t)D * 4}};
  const Span out[] = {{y, rows(M, p.y_ld, D, ye).extent()}, {s, rows(M, p.s_ld, D, re).extent()},
                      {scale, (size_t)M * groups * 4}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  // y is written while other rows' inputs are read, also where s takes their place
  if (ttt::abi::overlaps(y, out[0].n, x, rows(M, p.x_ld, D, xe).extent()) ||
      ttt::abi::overlaps(y, out[0].n, residual, rows(M, p.r_ld, D, re).extent()))
    return TTT_ERR_INVALID_ARG;
  if (M == 0) return TTT_OK;

  p.x = x; p.residual = residual; p.weight = weight; p.y = y; p.s = s; p.scale = scale;
  p.M = M; p.D = D; p.eps = eps;
  p.groups = groups;
  p.group128 = group ? 1 : 0;
  const bool vec = D % 8 == 0 && vec_ok(x, xe, p.x_ld, M) && vec_ok(residual, re, p.r_ld, M) &&
                   vec_ok(y, ye, p.y_ld, M) && vec_ok(s, re, p.s_ld, M) && !misaligned(weight);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return (mode & TTT_IN_BF16) ? dispatch_r<__nv_bfloat16>(p, mode, vec, st)
                              : dispatch_r<float>(p, mode, vec, st);
}

size_t ttt_norm_backward_workspace_bytes(int M, int D) {
  if (M <= 0 || D <= 0) return 0;
  return (size_t)bwd_ctas(M) * D * sizeof(float);
}

int ttt_norm_backward(const void* dy, const void* s, const float* weight, const void* ds, int M,
                      int D, float eps, unsigned mode, const long long* strides, void* dx,
                      float* dweight, void* workspace, size_t workspace_bytes,
                      void* cuda_stream) {
  if ((mode & ~kKnownModes) || (mode & TTT_NORM_Y_E4M3)) return TTT_ERR_INVALID_ARG;
  if (M < 0 || D < 1 || !finite_eps(eps)) return TTT_ERR_INVALID_ARG;
  if (!dweight || (M > 0 && (!dy || !s || !weight || !dx || !workspace))) return TTT_ERR_INVALID_ARG;
  if (short_rows(strides, M, D)) return TTT_ERR_INVALID_ARG;
  const size_t ge = (mode & TTT_OUT_BF16) ? 2 : 4, se = (mode & TTT_NORM_SUM_BF16) ? 2 : 4;
  if (misaligned_to(dy, ge) || misaligned_to(s, se) || misaligned_to(ds, se) ||
      misaligned_to(dx, se) || misaligned_to(weight, 4) || misaligned_to(dweight, 4) ||
      misaligned(workspace))
    return TTT_ERR_INVALID_ARG;
  const size_t need = ttt_norm_backward_workspace_bytes(M, D);
  if (workspace_bytes < need) return TTT_ERR_INVALID_ARG;
  if (D > kMaxD) return TTT_ERR_UNSUPPORTED;
  NormBwdParams p{};
  p.dy_ld = strides ? strides[0] : D;
  p.s_ld = strides ? strides[1] : D;
  p.ds_ld = strides ? strides[2] : D;
  p.dx_ld = strides ? strides[3] : D;
  const bool in_place = ds && dx == ds;
  if (in_place && p.ds_ld != p.dx_ld) return TTT_ERR_INVALID_ARG;
  const Span in[] = {{dy, rows(M, p.dy_ld, D, ge).extent()}, {s, rows(M, p.s_ld, D, se).extent()},
                     {in_place ? nullptr : ds, rows(M, p.ds_ld, D, se).extent()},
                     {weight, (size_t)D * 4}};
  const Span out[] = {{dx, rows(M, p.dx_ld, D, se).extent()}, {dweight, (size_t)D * 4},
                      {workspace, need}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (M == 0)
    return cudaMemsetAsync(dweight, 0, (size_t)D * 4, st) == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;

  p.dy = dy; p.s = s; p.weight = weight; p.ds = ds; p.dx = dx;
  p.part = static_cast<float*>(workspace);
  p.M = M; p.D = D; p.eps = eps;
  const bool vec = D % 8 == 0 && vec_ok(dy, ge, p.dy_ld, M) && vec_ok(s, se, p.s_ld, M) &&
                   vec_ok(ds, se, p.ds_ld, M) && vec_ok(dx, se, p.dx_ld, M) && !misaligned(weight);
  const int rc = (mode & TTT_OUT_BF16) ? dispatch_bwd<__nv_bfloat16>(p, mode, vec, st)
                                       : dispatch_bwd<float>(p, mode, vec, st);
  if (rc != TTT_OK) return rc;
  return ttt::launch_reduce_parts(p.part, bwd_ctas(M), D, {{dweight, nullptr, nullptr}, {D, 0, 0}},
                                  st);
}

}  // extern "C"
