// C-ABI entry points of the selective state space scan (include/ttt_ssm.h):
// argument checks, how far a prompt's tokens are split over CTAs, launches.
#include <initializer_list>

#include "ttt_ssm.h"
#include "abi_util.h"
#include "launch.h"
#include "ssm_bwd.cuh"

static_assert(ttt::kSsmTile == TTT_SSM_CHUNK, "a snapshot for every tile");

namespace {

using ttt::SsmParams;
using ttt::abi::misaligned;
using ttt::abi::misaligned_to;
using ttt::abi::Span;
using ttt::abi::Strided;

constexpr unsigned kKnownModes = TTT_IN_BF16 | TTT_OUT_BF16 | TTT_SSM_SOFTPLUS | TTT_SSM_PAD_ZERO;
constexpr int kMaxGridY = 65535;
constexpr int kMaxT = 1 << 30;  // token numbers and a tile beyond them fit an int
constexpr int kMaxB = 1 << 30;  // row numbers and a grid's height beyond them fit an int
constexpr long long kMaxTokenStride = 1 << 24;  // 16 tokens of 4 bytes and a row of channels: 32 bits

int check_sizes(int B, int T, int D, int G, int N, unsigned mode) {
  if (mode & ~kKnownModes) return TTT_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || D < 1 || G < 1 || N < 1 || D % G != 0) return TTT_ERR_INVALID_ARG;
  if (N != 8 && N != 16 && N != 32 && N != 64) return TTT_ERR_UNSUPPORTED;
  if (T > kMaxT || B > kMaxB || D > kMaxTokenStride || (long long)G * N > kMaxTokenStride || (long long)D * N > 0x7fffffffLL)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// Blocks of 32 channels in a group: each has its partial sums of dBm and dCm.
int channel_blocks(int D, int G) { return (D / G + 31) / 32; }

// CTAs along the tokens for `ctas` pairs of a row and a channel tile. Each CTA of a split runs its
// span nearly twice, so a split has to bring at least twice the SMs into play: none with
// more than half an SM's worth of pairs (128 pairs, 4096 tokens, forward: 172 us whole, 248 us
// in two), then up to two CTAs per SM (32 pairs: 174 us whole, 154 in two, 82 in four, 74 in
// eight; backward, 2048 tokens, 291, 201, 111 and 92). A span keeps 4 tiles (777 tokens, 24 pairs,
// backward: 121 us in four, 76 in eight).
int split_for(long long ctas, int T, int sms) {
  if (2 * ctas > sms) return 1;
  const int tiles = (T + ttt::kSsmTile - 1) / ttt::kSsmTile;
  int s = 1;
  while (s < ttt::kSsmMaxSplit && ctas * s <= sms && tiles >= 8 * s) s *= 2;
  return s;
}

int sm_count() {
  const int n = ttt::device_sm_count();
  return n > 0 ? n : 148;
}

template <typename Kernel>
int launch_kernel(Kernel kernel, long long blocks, int split, int B, int threads, size_t smem,
                  const SsmParams& p, cudaStream_t s) {
  if (blocks * split > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
  // (with a split's exchange on top, static)
  if (smem > 24 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * split), B < kMaxGridY ? B : kMaxGridY);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

// Forward: P states a thread (N = 16: 4; with 2, more warps and more parts to add, 1.38 against 1.33 ms
// for two prompts of 32768 tokens by 2048 channels).
template <int N, int P, typename InT, int VEC>
int launch_fwd_as(SsmParams p, cudaStream_t s) {
  using S = ttt::SsmFwdShape<N, P, InT, VEC>;
  p.tiles = (p.per_group + S::CH - 1) / S::CH;
  const long long blocks = (long long)p.tiles * p.G;
  p.split = split_for(blocks * p.B, p.T, sm_count());
  constexpr size_t smem = sizeof(typename S::Smem);
  return p.split > 1
             ? launch_kernel(ttt::ssm_fwd_kernel<N, P, InT, VEC, true>, blocks, p.split, p.B, S::NT, smem, p, s)
             : launch_kernel(ttt::ssm_fwd_kernel<N, P, InT, VEC, false>, blocks, 1, p.B, S::NT, smem, p, s);
}

template <int L, typename InT>
int launch_fwd(const SsmParams& p, cudaStream_t s) {
  constexpr int N = 4 * L;
  constexpr int P = N <= 16 ? 4 : 8;
  return p.vec ? launch_fwd_as<N, P, InT, 4>(p, s) : launch_fwd_as<N, P, InT, 1>(p, s);
}

template <int N, int P, typename InT, typename OutT, int VEC>
int launch_bwd_as(SsmParams p, cudaStream_t s) {
  using S = ttt::SsmBwdShape<N, P, InT, OutT, VEC>;
  const long long blocks = (long long)((p.per_group + S::CH - 1) / S::CH) * p.G;
  constexpr size_t smem = sizeof(typename S::Smem);
  return p.split > 1
             ? launch_kernel(ttt::ssm_bwd_kernel<N, P, InT, OutT, VEC, true>, blocks, p.split, p.B, S::NT, smem, p, s)
             : launch_kernel(ttt::ssm_bwd_kernel<N, P, InT, OutT, VEC, false>, blocks, 1, p.B, S::NT, smem, p, s);
}

template <int L, typename InT>
int launch_bwd(const SsmParams& p, cudaStream_t s) {
  constexpr int N = 4 * L;
  constexpr int P = N <= 16 ? 4 : 8;
  if (p.out_bf16)
    return p.vec ? launch_bwd_as<N, P, InT, __nv_bfloat16, 4>(p, s)
                 : launch_bwd_as<N, P, InT, __nv_bfloat16, 1>(p, s);
  return p.vec ? launch_bwd_as<N, P, InT, float, 4>(p, s) : launch_bwd_as<N, P, InT, float, 1>(p, s);
}

// Several batch rows a thread once that still leaves 16 warps for every SM.
template <int L, typename InT, int VEC>
int launch_step_as(const SsmParams& p, cudaStream_t s) {
  constexpr int R = L < 4 ? L : 4;  // (of 2048 channels, 512 rows: 22 us; two rows 28 us)
  const long long blocks = ((long long)p.D * L + 255) / 256;
  const bool several = blocks * (p.B / R) >= 2LL * sm_count();
  const int rows = several ? (p.B + R - 1) / R : p.B;
  const dim3 grid((unsigned)blocks, rows < kMaxGridY ? rows : kMaxGridY);
  if (several)
    ttt::ssm_step_kernel<L, InT, VEC, R><<<grid, 256, 0, s>>>(p);
  else
    ttt::ssm_step_kernel<L, InT, VEC, 1><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <int L, typename InT>
int launch_step(const SsmParams& p, cudaStream_t s) {
  return p.vec ? launch_step_as<L, InT, 4>(p, s) : launch_step_as<L, InT, 1>(p, s);
}

enum Which { kForward, kBackward, kStep };

template <Which W, int L, typename InT>
int launch_one(const SsmParams& p, cudaStream_t s) {
  if constexpr (W == kForward) return launch_fwd<L, InT>(p, s);
  if constexpr (W == kBackward) return launch_bwd<L, InT>(p, s);
  return launch_step<L, InT>(p, s);
}

template <Which W, typename InT>
int dispatch_n(const SsmParams& p, int N, cudaStream_t s) {
  switch (N) {
    case 8: return launch_one<W, 2, InT>(p, s);
    case 16: return launch_one<W, 4, InT>(p, s);
    case 32: return launch_one<W, 8, InT>(p, s);
    default: return launch_one<W, 16, InT>(p, s);
  }
}

template <Which W>
int dispatch(const SsmParams& p, int N, unsigned mode, cudaStream_t s) {
  return (mode & TTT_IN_BF16) ? dispatch_n<W, __nv_bfloat16>(p, N, s) : dispatch_n<W, float>(p, N, s);
}

// Strides of a prompt's tensors into p (null: contiguous). False: a token stride that is
// negative or too long for the kernels' arithmetic within a tile, where there are two tokens.
bool set_strides(SsmParams& p, int T, int D, int G, int N, const long long* s) {
  const long long tok = (long long)T * D, vec = (long long)T * G * N, gn = (long long)G * N;
  const long long whole[14] = {tok, D, tok, D, tok, D, vec, gn, N, vec, gn, N, tok, D};
  if (!s) s = whole;
  p.u_b = s[0]; p.d_b = s[2]; p.z_b = s[4]; p.Bm_b = s[6]; p.Bm_g = s[8]; p.Cm_b = s[9];
  p.Cm_g = s[11]; p.y_b = s[12];
  const long long t[6] = {s[1], s[3], s[5], s[7], s[10], s[13]};
  int* to[6] = {&p.u_t, &p.d_t, &p.z_t, &p.Bm_t, &p.Cm_t, &p.y_t};
  for (int i = 0; i < 6; ++i) {
    if (T <= 1) { *to[i] = 0; continue; }  // (no distance to go)
    if (t[i] < 0 || t[i] > kMaxTokenStride) return false;
    *to[i] = (int)t[i];
  }
  return true;
}

struct Tensors {
  Strided u, delta, z, Bm, Cm, y;
  bool negative() const {
    return u.negative() || delta.negative() || z.negative() || Bm.negative() || Cm.negative() ||
           y.negative();
  }
};

Tensors tensors(const SsmParams& p, int B, int T, int D, int G, int N, size_t ie, size_t oe) {
  return {{{B, T, 1}, {p.u_b, p.u_t, 0}, D, ie},          {{B, T, 1}, {p.d_b, p.d_t, 0}, D, ie},
          {{B, T, 1}, {p.z_b, p.z_t, 0}, D, ie},          {{B, T, G}, {p.Bm_b, p.Bm_t, p.Bm_g}, N, ie},
          {{B, T, G}, {p.Cm_b, p.Cm_t, p.Cm_g}, N, ie},   {{B, T, 1}, {p.y_b, p.y_t, 0}, D, oe}};
}

// Can every row of channels and of Bm and Cm be read and written in packs of 4?
bool packs_of_4(const SsmParams& p, std::initializer_list<const void*> in, size_t ie, const void* y,
                size_t oe) {
  for (const void* q : in)
    if (misaligned_to(q, 4 * ie)) return false;
  long long all = p.u_b | p.u_t | p.d_b | p.d_t | p.Bm_b | p.Bm_t | p.Bm_g | p.Cm_b | p.Cm_t |
                  p.Cm_g | p.y_b | p.y_t | p.per_group;
  if (p.z) all |= p.z_b | p.z_t;
  return !misaligned_to(y, 4 * oe) && all % 4 == 0;
}

size_t par_floats(int B, int D, int N) { return (size_t)B * ttt::kSsmMaxSplit * D * (N + 2); }
size_t bc_floats(int B, int T, int D, int G, int N) {
  return (size_t)channel_blocks(D, G) * B * T * G * 2 * N;
}

}  // namespace

extern "C" {

int ttt_ssm_forward(const void* u, const void* delta, const float* A, const void* Bm,
                    const void* Cm, const float* skip, const void* z, const float* delta_bias,
                    const float* h0, const int* lengths, int B, int T, int D, int G, int N,
                    unsigned mode, const long long* strides, void* y, float* h_T,
                    float* h_chunks, void* cuda_stream) {
  if (const int rc = check_sizes(B, T, D, G, N, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  if (B > 0 && (!A || !h_T || (T > 0 && (!u || !delta || !Bm || !Cm || !y))))
    return TTT_ERR_INVALID_ARG;
  if (misaligned(A) || misaligned(h0) || misaligned(h_T) || misaligned(h_chunks) ||
      misaligned_to(skip, 4) || misaligned_to(delta_bias, 4) || misaligned_to(lengths, 4) ||
      misaligned_to(u, ie) || misaligned_to(delta, ie) || misaligned_to(z, ie) ||
      misaligned_to(Bm, ie) || misaligned_to(Cm, ie) || misaligned_to(y, oe))
    return TTT_ERR_INVALID_ARG;
  SsmParams p{};
  if (!set_strides(p, T, D, G, N, strides)) return TTT_ERR_INVALID_ARG;
  const Tensors ts = tensors(p, B, T, D, G, N, ie, oe);
  if (ts.negative() || ts.y.self_overlap()) return TTT_ERR_INVALID_ARG;
  const size_t state = (size_t)B * D * N * 4;
  const size_t n_chunks = ((size_t)T + ttt::kSsmTile - 1) / ttt::kSsmTile;
  const Span in[] = {{u, ts.u.extent()}, {delta, ts.delta.extent()}, {z, ts.z.extent()},
                     {Bm, ts.Bm.extent()}, {Cm, ts.Cm.extent()}, {A, (size_t)D * N * 4},
                     {skip, (size_t)D * 4}, {delta_bias, (size_t)D * 4},
                     {h0 == h_T ? nullptr : h0, state}, {lengths, (size_t)B * 4}};
  const Span out[] = {{y, ts.y.extent()}, {h_T, state}, {h_chunks, state * n_chunks}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  if (B == 0) return TTT_OK;

  p.u = u; p.delta = delta; p.z = z; p.Bm = Bm; p.Cm = Cm;
  p.A = A; p.skip = skip; p.delta_bias = delta_bias; p.h0 = h0; p.lengths = lengths;
  p.y = y; p.h_T = h_T; p.h_chunks = h_chunks;
  p.B = B; p.T = T; p.D = D; p.G = G;
  p.per_group = D / G;
  p.softplus = (mode & TTT_SSM_SOFTPLUS) ? 1 : 0;
  p.out_bf16 = (mode & TTT_OUT_BF16) ? 1 : 0;
  p.pad_zero = (mode & TTT_SSM_PAD_ZERO) ? 1 : 0;
  p.vec = packs_of_4(p, {u, delta, z, Bm, Cm}, ie, y, oe);
  return dispatch<kForward>(p, N, mode, static_cast<cudaStream_t>(cuda_stream));
}

size_t ttt_ssm_backward_workspace_bytes(int B, int T, int D, int G, int N) {
  if (B <= 0 || T < 0 || D < 1 || G < 1 || D % G != 0) return 0;
  if (N != 8 && N != 16 && N != 32 && N != 64) return 0;
  return (bc_floats(B, T, D, G, N) + par_floats(B, D, N)) * sizeof(float);
}

int ttt_ssm_backward(const void* u, const void* delta, const float* A, const void* Bm,
                     const void* Cm, const float* skip, const void* z, const float* delta_bias,
                     const int* lengths, int B, int T, int D, int G, int N, unsigned mode,
                     const long long* strides, const float* h_chunks, const void* dy,
                     const float* dh_T, void* du, void* ddelta, float* dA, void* dBm, void* dCm,
                     float* dskip, void* dz, float* d_delta_bias, float* dh0, void* workspace,
                     size_t workspace_bytes, void* cuda_stream) {
  if (const int rc = check_sizes(B, T, D, G, N, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  const bool toks = B > 0 && T > 0;
  if (!dA || (B > 0 && (!A || !workspace))) return TTT_ERR_INVALID_ARG;
  if (toks && (!u || !delta || !Bm || !Cm || !h_chunks || !dy || !du || !ddelta || !dBm || !dCm))
    return TTT_ERR_INVALID_ARG;
  if (toks && ((z != nullptr) != (dz != nullptr))) return TTT_ERR_INVALID_ARG;
  if (misaligned(A) || misaligned(h_chunks) || misaligned(dh_T) || misaligned(dh0) ||
      misaligned(workspace) || misaligned_to(dA, 4) || misaligned_to(skip, 4) ||
      misaligned_to(delta_bias, 4) || misaligned_to(lengths, 4) || misaligned_to(dskip, 4) ||
      misaligned_to(d_delta_bias, 4) || misaligned_to(u, ie) || misaligned_to(delta, ie) ||
      misaligned_to(z, ie) || misaligned_to(Bm, ie) || misaligned_to(Cm, ie) ||
      misaligned_to(dy, oe) || misaligned_to(du, ie) || misaligned_to(ddelta, ie) ||
      misaligned_to(dz, ie) || misaligned_to(dBm, ie) || misaligned_to(dCm, ie))
    return TTT_ERR_INVALID_ARG;
  const size_t need = ttt_ssm_backward_workspace_bytes(B, T, D, G, N);
  if (workspace_bytes < need) return TTT_ERR_INVALID_ARG;
  SsmParams p{};
  if (!set_strides(p, T, D, G, N, strides)) return TTT_ERR_INVALID_ARG;
  const Tensors ts = tensors(p, B, T, D, G, N, ie, oe);
  if (ts.negative()) return TTT_ERR_INVALID_ARG;
  const size_t state = (size_t)B * D * N * 4, par = (size_t)D * N * 4;
  const size_t n_chunks = ((size_t)T + ttt::kSsmTile - 1) / ttt::kSsmTile;
  const size_t tok = (size_t)B * T * D * ie, vec = (size_t)B * T * G * N * ie;
  const Span in[] = {{u, ts.u.extent()}, {delta, ts.delta.extent()}, {z, ts.z.extent()},
                     {Bm, ts.Bm.extent()}, {Cm, ts.Cm.extent()}, {A, par},
                     {skip, (size_t)D * 4}, {delta_bias, (size_t)D * 4},
                     {lengths, (size_t)B * 4}, {h_chunks, state * n_chunks},
                     {dy, ts.y.extent()}, {dh_T, state}};
  const Span out[] = {{du, tok}, {ddelta, tok}, {dz, tok}, {dBm, vec}, {dCm, vec}, {dA, par},
                      {dskip, (size_t)D * 4}, {d_delta_bias, (size_t)D * 4}, {dh0, state},
                      {workspace, need}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (B == 0) {
    if (cudaMemsetAsync(dA, 0, par, s) != cudaSuccess ||
        (dskip && cudaMemsetAsync(dskip, 0, (size_t)D * 4, s) != cudaSuccess) ||
        (d_delta_bias && cudaMemsetAsync(d_delta_bias, 0, (size_t)D * 4, s) != cudaSuccess))
      return TTT_ERR_CUDA;
    return TTT_OK;
  }

  p.u = u; p.delta = delta; p.z = z; p.Bm = Bm; p.Cm = Cm;
  p.A = A; p.skip = skip; p.delta_bias = delta_bias; p.lengths = lengths;
  p.h_chunks = const_cast<float*>(h_chunks);
  p.dy = dy; p.dh_T = dh_T; p.du = du; p.ddelta = ddelta; p.dz = dz; p.dh0 = dh0;
  p.part_bc = static_cast<float*>(workspace);
  p.part_par = p.part_bc + bc_floats(B, T, D, G, N);
  p.B = B; p.T = T; p.D = D; p.G = G;
  p.per_group = D / G;
  p.tiles = channel_blocks(D, G);
  p.split = split_for((long long)p.tiles * G * B, T, sm_count());
  p.softplus = (mode & TTT_SSM_SOFTPLUS) ? 1 : 0;
  p.out_bf16 = (mode & TTT_OUT_BF16) ? 1 : 0;
  p.vec = packs_of_4(p, {u, delta, z, Bm, Cm, du, ddelta, dz}, ie, dy, oe) && D % 4 == 0;
  const size_t bc = (size_t)B * T * G * 2 * N;
  const size_t bc_blocks = (bc / 4 + 255) / 256;
  if (bc_blocks > 0x7fffffffULL || (long long)B * p.split > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
  int rc = dispatch<kBackward>(p, N, mode, s);
  if (rc != TTT_OK) return rc;
  if (bc_blocks > 0) {
    if (mode & TTT_IN_BF16)
      ttt::ssm_sum_bc_kernel<<<(unsigned)bc_blocks, 256, 0, s>>>(
          p.part_bc, p.tiles, B, T, G, N, lengths, static_cast<__nv_bfloat16*>(dBm),
          static_cast<__nv_bfloat16*>(dCm));
    else
      ttt::ssm_sum_bc_kernel<<<(unsigned)bc_blocks, 256, 0, s>>>(
          p.part_bc, p.tiles, B, T, G, N, lengths, static_cast<float*>(dBm),
          static_cast<float*>(dCm));
    if (cudaGetLastError() != cudaSuccess) return TTT_ERR_CUDA;
  }
  const long long dn = (long long)D * N;
  return ttt::launch_reduce_parts(p.part_par, B * p.split, dn + 2LL * D,
                                  {{dA, dskip, d_delta_bias}, {dn, D, D}}, s);
}

int ttt_ssm_step(const void* u, const void* delta, const float* A, const void* Bm,
                 const void* Cm, const float* skip, const void* z, const float* delta_bias,
                 float* h, const unsigned char* active, int B, int D, int G, int N,
                 unsigned mode, const long long* strides, void* y, void* cuda_stream) {
  if (const int rc = check_sizes(B, 1, D, G, N, mode)) return rc;
  const size_t ie = (mode & TTT_IN_BF16) ? 2 : 4, oe = (mode & TTT_OUT_BF16) ? 2 : 4;
  if (B > 0 && (!u || !delta || !A || !Bm || !Cm || !h || !y)) return TTT_ERR_INVALID_ARG;
  if (misaligned(A) || misaligned(h) || misaligned_to(skip, 4) || misaligned_to(delta_bias, 4) ||
      misaligned_to(u, ie) || misaligned_to(delta, ie) || misaligned_to(z, ie) ||
      misaligned_to(Bm, ie) || misaligned_to(Cm, ie) || misaligned_to(y, oe))
    return TTT_ERR_INVALID_ARG;
  SsmParams p{};
  if (strides) {
    const long long full[14] = {strides[0], 0, strides[1], 0, strides[2], 0, strides[3], 0,
                                strides[4], strides[5], 0, strides[6], strides[7], 0};
    if (!set_strides(p, 1, D, G, N, full)) return TTT_ERR_INVALID_ARG;
  } else {
    if (!set_strides(p, 1, D, G, N, nullptr)) return TTT_ERR_INVALID_ARG;
  }
  const Tensors ts = tensors(p, B, 1, D, G, N, ie, oe);
  if (ts.negative() || ts.y.self_overlap()) return TTT_ERR_INVALID_ARG;
  const Span in[] = {{u, ts.u.extent()}, {delta, ts.delta.extent()}, {z, ts.z.extent()},
                     {Bm, ts.Bm.extent()}, {Cm, ts.Cm.extent()}, {A, (size_t)D * N * 4},
                     {skip, (size_t)D * 4}, {delta_bias, (size_t)D * 4}, {active, (size_t)B}};
  const Span out[] = {{y, ts.y.extent()}, {h, (size_t)B * D * N * 4}};
  if (ttt::abi::any_overlap(in, out)) return TTT_ERR_INVALID_ARG;
  if (B == 0) return TTT_OK;

  p.u = u; p.delta = delta; p.z = z; p.Bm = Bm; p.Cm = Cm;
  p.A = A; p.skip = skip; p.delta_bias = delta_bias; p.active = active; p.h_T = h; p.y = y;
  p.B = B; p.T = 1; p.D = D; p.G = G;
  p.per_group = D / G;
  p.softplus = (mode & TTT_SSM_SOFTPLUS) ? 1 : 0;
  p.out_bf16 = (mode & TTT_OUT_BF16) ? 1 : 0;
  p.pad_zero = (mode & TTT_SSM_PAD_ZERO) ? 1 : 0;
  p.vec = !misaligned_to(Bm, 4 * ie) && !misaligned_to(Cm, 4 * ie) &&
          (p.Bm_b | p.Bm_g | p.Cm_b | p.Cm_g) % 4 == 0;
  return dispatch<kStep>(p, N, mode, static_cast<cudaStream_t>(cuda_stream));
}

}  // extern "C"

