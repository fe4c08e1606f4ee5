// C-ABI entry points of the short causal convolution (include/ttt_conv.h):
// argument checks, choice of the vector width, launches; and the reduction of
// partial sums that the other operators' backward passes share.
#include "ttt_conv.h"
#include "abi_util.h"
#include "conv.cuh"

namespace ttt {

// COLS columns by 1024 / COLS strands of rows a block.
template <int COLS>
__global__ void __launch_bounds__(1024) reduce_parts_kernel(const float* part, int parts,
                                                            long long n, ReduceOut out) {
  constexpr int STRANDS = 1024 / COLS;
  __shared__ float red[STRANDS][COLS + 1];
  const int col = threadIdx.x % COLS, strand = threadIdx.x / COLS;
  const long long i = (long long)blockIdx.x * COLS + col;
  float s = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int k = strand; k < parts; k += STRANDS) s += part[(long long)k * n + i];
  }
  red[strand][col] = s;
#pragma unroll
  for (int half = STRANDS / 2; half > 0; half /= 2) {
    __syncthreads();
    if (strand < half) red[strand][col] += red[strand + half][col];
  }
  if (strand != 0 || i >= n) return;
  long long o = i;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (o < out.n[k]) {
      if (out.p[k]) out.p[k][o] = red[0][col];
      return;
    }
    o -= out.n[k];
  }
}

// 8 columns a block (one sector of 32 bytes a row) where 32 would leave most SMs idle and a
// strand long: 1184 rows of 1536, 48 blocks, took 20 us.
int launch_reduce_parts(const float* part, int parts, long long n, const ReduceOut& out,
                        cudaStream_t stream) {
  if (n <= 0) return TTT_OK;
  if (n >= 32 * 296)
    reduce_parts_kernel<32><<<(unsigned)((n + 31) / 32), 1024, 0, stream>>>(part, parts, n, out);
  else
    reduce_parts_kernel<8><<<(unsigned)((n + 7) / 8), 1024, 0, stream>>>(part, parts, n, out);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

}  // namespace ttt

namespace {

using ttt::ConvParams;
using ttt::RowStrides;
using ttt::abi::misaligned;
using ttt::abi::misaligned_to;
using ttt::abi::Span;
using ttt::abi::Strided;

constexpr unsigned kKnownModes = TTT_IN_BF16 | TTT_OUT_BF16 | TTT_CONV_SILU | TTT_CONV_PAD_ZERO;
constexpr int kMaxGridY = 65535;
constexpr int kMaxT = 1 << 30;  // token numbers and a run beyond them fit an int
constexpr int kMaxB = 1 << 30;  // row numbers and a grid's height beyond them fit an int

enum Which { kForward, kBackward, kStep };

template <Which W, typename InT, typename OutT, int VEC, int K>
int launch(ConvParams p, cudaStream_t s) {
  p.vecs = (int)((long long)p.H * p.d / VEC);
  const unsigned rows = p.B < kMaxGridY ? p.B : kMaxGridY;
  if constexpr (W == kForward) {
    const long long enough = 148LL * 16 * 32 * 32;
    p.run = (long long)p.vecs * p.B * p.T >= enough ? 32 : 8;
    p.tiles = p.T > 0 ? (int)(((long long)p.T + p.run - 1) / p.run) : 1;
    const long long blocks = ((long long)p.tiles * p.vecs + 127) / 128;
    if (blocks > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
    ttt::conv_fwd_kernel<InT, OutT, VEC, K><<<dim3((unsigned)blocks, rows), 128, 0, s>>>(p);
  } else if constexpr (W == kBackward) {
    ttt::conv_bwd_kernel<InT, OutT, VEC, K>
        <<<dim3((p.vecs + 31) / 32, p.tiles, rows), dim3(32, ttt::kConvSegs), 0, s>>>(p);
  } else {
    ttt::conv_step_kernel<InT, OutT, VEC, K><<<dim3((p.vecs + 127) / 128, rows), 128, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <Which W, typename InT, typename OutT, int VEC>
int dispatch_k(const ConvParams& p, int K, cudaStream_t s) {
  if (K == 2) return launch<W, InT, OutT, VEC, 2>(p, s);
  if (K == 3) return launch<W, InT, OutT, VEC, 3>(p, s);
  return launch<W, InT, OutT, VEC, 4>(p, s);
}

// `vec`: every pointer and stride allows vectors of the type's width.
template <Which W, typename InT, int VEC>
int dispatch_out(const ConvParams& p, int K, unsigned mode, bool vec, cudaStream_t s) {
  if (mode & TTT_OUT_BF16)
    return vec ? dispatch_k<W, InT, __nv_bfloat16, VEC>(p, K, s)
               : dispatch_k<W, InT, __nv_bfloat16, 1>(p, K, s);
  return vec ? dispatch_k<W, InT, float, VEC>(p, K, s) : dispatch_k<W, InT, float, 1>(p, K, s);
}

template <Which W>
int dispatch(const ConvParams& p, int K, unsigned mode, bool vec, cudaStream_t s) {
  return (mode & TTT_IN_BF16) ? dispatch_out<W, __nv_bfloat16, 4>(p, K, mode, vec, s)
                              : dispatch_out<W, float, 4>(p, K, mode, vec, s);
}

// Can every row be read and written four channels at a time? (8 bytes of bf16: with 16, eight
// channels a thread, the windows and weights leave too few warps, 170 against 108 us for
// 2 x 32768 tokens by 2048 channels.)
bool can_vec(int d, const Strided* ts, const void* const* ptrs, int n) {
  const int v = 4;
  if (d % v != 0) return false;
  for (int i = 0; i < n; ++i) {
    const size_t bytes = v * ts[i].elt < 16 ? v * ts[i].elt : 16;
    if (misaligned_to(ptrs[i], bytes) || (ptrs[i] && !ts[i].multiple_of(v))) return false;
  }
  return true;
}

RowStrides rs(const long long* s) { return {s[0], s[1], s[2]}; }

Strided tensor(const RowStrides& s, int B, int H, int n, int d, size_t elt) {
  return {{B, H, n}, {s.b, s.h, s.t}, d, elt};
}

RowStrides contiguous(int H, int n, int d) {
  return {(long long)H * n * d, (long long)n * d, d};
}

// What every entry point checks first.
int check_sizes(int B, int H, int T, int d, int K, unsigned mode) {
  if (mode & ~kKnownModes) return TTT_ERR_INVALID_ARG;
  if (B < 0 || H < 0 || T < 0 || d < 1 || K < 1) return TTT_ERR_INVALID_ARG;
  if (K < 2 || K > 4) return TTT_ERR_UNSUPPORTED;
  if ((long long)H * d * K > 0x7fffffffLL || T > kMaxT || B > kMaxB) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// Tokens per segment of the backward: what costs least when the blocks go over 148 SMs two at a
// time in whole rounds and a segment has 9 tokens' worth of start beside its own (8 x 4096 tokens by 768
// channels: 43, two rounds, 59 us; 32, 2.6 rounds, 65 us). By the sizes alone, so that the
// workspace and the order of the sums follow from them.
int bwd_seg(int B, int H, int T, int d) {
  const long long vecs = (long long)H * d / (d % 4 == 0 ? 4 : 1);
  const long long columns = (vecs + 31) / 32 * B;
  int best = 8;
  long long least = 0;
  for (int seg = 8; seg <= 64; ++seg) {
    const long long tiles = ((long long)T + seg * ttt::kConvSegs - 1) / (seg * ttt::kConvSegs);
    const long long cost = (columns * tiles + 295) / 296 * (seg + 9);
    if (seg == 8 || cost <= least) {
      best = seg;
      least = cost;
    }
  }
  return best;
}

// Blocks of the backward along the tokens.
int bwd_tiles(int B, int H, int T, int d) {
  const int per = bwd_seg(B, H, T, d) * ttt::kConvSegs;
  const int n = (int)(((long long)T + per - 1) / per);
  return n > 0 ? n : 1;
}

}  // namespace

extern "C" {

int ttt_conv_forward(const void* x, const float* weight, const float* bias, const void* state,
                     const int* lengths, int B, int H, int T, int d, int K, unsigned mode,
                     const long long* strides, void* y, void* state_T, void* cuda_stream) {
  if (const int rc = check_sizes(B, H, T, d, K, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  const bool rows = (long long)B * H > 0;
  if (rows && (!weight || (T > 0 && (!x || !y)))) return TTT_ERR_INVALID_ARG;
  if (misaligned(weight) || misaligned_to(bias, 4) || misaligned_to(lengths, 4) ||
      misaligned_to(x, ie) || misaligned_to(state, ie) || misaligned_to(state_T, ie) ||
      misaligned_to(y, oe))
    return TTT_ERR_INVALID_ARG;
  ConvParams p{};
  p.xs = strides ? rs(strides) : contiguous(H, T, d);
  p.ys = strides ? rs(strides + 3) : contiguous(H, T, d);
  p.ss = strides ? rs(strides + 6) : contiguous(H, K - 1, d);
  p.so = strides ? rs(strides + 9) : contiguous(H, K - 1, d);
  const Strided ts[] = {tensor(p.xs, B, H, T, d, ie), tensor(p.ys, B, H, T, d, oe),
                        tensor(p.ss, B, H, K - 1, d, ie), tensor(p.so, B, H, K - 1, d, ie)};
  const void* const ptrs[] = {x, y, state, state_T};
  for (const Strided& t : ts)
    if (t.negative()) return TTT_ERR_INVALID_ARG;
  if (ts[1].self_overlap() || (state_T && ts[3].self_overlap())) return TTT_ERR_INVALID_ARG;
  const bool in_place = state_T && state_T == state;
  if (in_place && (p.ss.b != p.so.b || p.ss.h != p.so.h || p.ss.t != p.so.t))
    return TTT_ERR_INVALID_ARG;
  const size_t we = (size_t)H * d * 4;
  const Span in[] = {{x, ts[0].extent()}, {weight, we * K}, {bias, we},
                     {in_place ? nullptr : state, ts[2].extent()}, {lengths, (size_t)B * 4}};
  const Span out[] = {{y, ts[1].extent()}, {state_T, ts[3].extent()}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  if (!rows || (T == 0 && !state_T)) return TTT_OK;

  p.x = x; p.weight = weight; p.bias = bias; p.state = state; p.lengths = lengths;
  p.y = y; p.state_T = state_T;
  p.B = B; p.H = H; p.T = T; p.d = d;
  p.silu = (mode & TTT_CONV_SILU) ? 1 : 0;
  p.pad_zero = (mode & TTT_CONV_PAD_ZERO) ? 1 : 0;
  return dispatch<kForward>(p, K, mode, can_vec(d, ts, ptrs, 4),
                            static_cast<cudaStream_t>(cuda_stream));
}

size_t ttt_conv_backward_workspace_bytes(int B, int H, int T, int d, int K) {
  if (B <= 0 || H <= 0 || T < 0 || d <= 0 || K <= 0) return 0;
  return (size_t)B * bwd_tiles(B, H, T, d) * ((size_t)H * d) * (K + 1) * sizeof(float);
}

int ttt_conv_backward(const void* x, const float* weight, const float* bias, const void* state,
                      const int* lengths, int B, int H, int T, int d, int K, unsigned mode,
                      const long long* strides, const void* dy, const void* dstate_T, void* dx,
                      float* dweight, float* dbias, void* dstate, void* workspace,
                      size_t workspace_bytes, void* cuda_stream) {
  if (const int rc = check_sizes(B, H, T, d, K, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  const bool rows = (long long)B * H > 0;
  if (rows && (!weight || !workspace || (T > 0 && (!x || !dy || !dx)))) return TTT_ERR_INVALID_ARG;
  if (H > 0 && (!dweight || (bias && !dbias))) return TTT_ERR_INVALID_ARG;
  if (misaligned(weight) || misaligned(workspace) || misaligned_to(bias, 4) ||
      misaligned_to(lengths, 4) || misaligned_to(dweight, 4) || misaligned_to(dbias, 4) ||
      misaligned_to(x, ie) || misaligned_to(state, ie) || misaligned_to(dstate_T, ie) ||
      misaligned_to(dx, ie) || misaligned_to(dstate, ie) || misaligned_to(dy, oe))
    return TTT_ERR_INVALID_ARG;
  const size_t need = ttt_conv_backward_workspace_bytes(B, H, T, d, K);
  if (workspace_bytes < need) return TTT_ERR_INVALID_ARG;
  ConvParams p{};
  p.xs = strides ? rs(strides) : contiguous(H, T, d);
  p.ys = strides ? rs(strides + 3) : contiguous(H, T, d);
  p.ss = strides ? rs(strides + 6) : contiguous(H, K - 1, d);
  const RowStrides xc = contiguous(H, T, d), sc = contiguous(H, K - 1, d);
  const Strided ts[] = {tensor(p.xs, B, H, T, d, ie),     tensor(p.ys, B, H, T, d, oe),
                        tensor(p.ss, B, H, K - 1, d, ie), tensor(sc, B, H, K - 1, d, ie),
                        tensor(xc, B, H, T, d, ie),       tensor(sc, B, H, K - 1, d, ie)};
  const void* const ptrs[] = {x, dy, state, dstate_T, dx, dstate};
  for (const Strided& t : ts)
    if (t.negative()) return TTT_ERR_INVALID_ARG;
  const size_t we = (size_t)H * d * 4;
  const Span in[] = {{x, ts[0].extent()}, {dy, ts[1].extent()}, {state, ts[2].extent()},
                     {dstate_T, ts[3].extent()}, {weight, we * K}, {bias, we},
                     {lengths, (size_t)B * 4}};
  const Span out[] = {{dx, ts[4].extent()}, {dstate, ts[5].extent()}, {dweight, we * K},
                      {dbias, we}, {workspace, need}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  p.seg = bwd_seg(B, H, T, d);
  p.tiles = bwd_tiles(B, H, T, d);
  if (p.tiles > kMaxGridY) return TTT_ERR_UNSUPPORTED;
  if ((long long)B * p.tiles > kMaxB) return TTT_ERR_UNSUPPORTED;  // rows of partial sums
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const long long D = (long long)H * d;
  if (!rows) {
    if (D > 0 && (cudaMemsetAsync(dweight, 0, we * K, s) != cudaSuccess ||
                  (dbias && cudaMemsetAsync(dbias, 0, we, s) != cudaSuccess)))
      return TTT_ERR_CUDA;
    return TTT_OK;
  }

  p.x = x; p.weight = weight; p.bias = bias; p.state = state; p.lengths = lengths;
  p.y = const_cast<void*>(dy); p.dstate_T = dstate_T; p.dx = dx; p.dstate = dstate;
  p.part = static_cast<float*>(workspace);
  p.B = B; p.H = H; p.T = T; p.d = d;
  p.silu = (mode & TTT_CONV_SILU) ? 1 : 0;
  p.pad_zero = (mode & TTT_CONV_PAD_ZERO) ? 1 : 0;
  const int rc =
      dispatch<kBackward>(p, K, mode, can_vec(d, ts, ptrs, 6), s);
  if (rc != TTT_OK) return rc;
  return ttt::launch_reduce_parts(p.part, B * p.tiles, D * (K + 1),
                                  {{dweight, dbias, nullptr}, {D * K, D, 0}}, s);
}

int ttt_conv_step(const void* x, const float* weight, const float* bias, void* state,
                  const unsigned char* active, int B, int H, int d, int K, unsigned mode,
                  const long long* strides, void* y, void* cuda_stream) {
  if (const int rc = check_sizes(B, H, 1, d, K, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  const bool rows = (long long)B * H > 0;
  if (rows && (!x || !weight || !state || !y)) return TTT_ERR_INVALID_ARG;
  if (misaligned(weight) || misaligned_to(bias, 4) || misaligned_to(x, ie) ||
      misaligned_to(state, ie) || misaligned_to(y, oe))
    return TTT_ERR_INVALID_ARG;
  ConvParams p{};
  p.xs = strides ? RowStrides{strides[0], strides[1], 0} : contiguous(H, 1, d);
  p.ys = strides ? RowStrides{strides[2], strides[3], 0} : contiguous(H, 1, d);
  p.ss = strides ? rs(strides + 4) : contiguous(H, K - 1, d);
  const Strided ts[] = {tensor(p.xs, B, H, 1, d, ie), tensor(p.ys, B, H, 1, d, oe),
                        tensor(p.ss, B, H, K - 1, d, ie)};
  const void* const ptrs[] = {x, y, state};
  for (const Strided& t : ts)
    if (t.negative()) return TTT_ERR_INVALID_ARG;
  if (ts[1].self_overlap() || ts[2].self_overlap()) return TTT_ERR_INVALID_ARG;
  const size_t we = (size_t)H * d * 4;
  const Span in[] = {{x, ts[0].extent()}, {weight, we * K}, {bias, we}, {active, (size_t)B}};
  const Span out[] = {{y, ts[1].extent()}, {state, ts[2].extent()}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  if (!rows) return TTT_OK;

  p.x = x; p.weight = weight; p.bias = bias; p.active = active; p.y = y; p.state_T = state;
  p.B = B; p.H = H; p.T = 1; p.d = d;
  p.silu = (mode & TTT_CONV_SILU) ? 1 : 0;
  p.pad_zero = (mode & TTT_CONV_PAD_ZERO) ? 1 : 0;
  return dispatch<kStep>(p, K, mode, can_vec(d, ts, ptrs, 3),
                         static_cast<cudaStream_t>(cuda_stream));
}

}  // extern "C"
