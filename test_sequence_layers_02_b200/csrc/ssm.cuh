// Selective state space scan, forward and one-token step (include/ttt_ssm.h has the
// formulas). The backward is in ssm_bwd.cuh.
//
// Work: one exponential, one multiply and two multiply-adds for each of the N
// states of every (token, channel), against four 2- or 4-byte elements of
// traffic. At N = 16 the special-function units (16 lanes per clock and SM) bind:
// (N + 4) / 16 clocks per (token, channel) with the softplus and the gate counted,
// where HBM would take a quarter of that in bf16.
#pragma once

#include <cooperative_groups.h>

#include "seq_common.cuh"

namespace ttt {

struct SsmParams {
  const void *u, *delta, *z, *Bm, *Cm;  // z may be null
  const float* A;           // [D, N]
  const float* skip;        // [D] or null
  const float* delta_bias;  // [D] or null
  const float* h0;          // [B, D, N] or null
  const int* lengths;       // [B] or null
  const unsigned char* active;  // step: [B] or null
  void* y;
  float* h_T;               // [B, D, N] (step: in place)
  float* h_chunks;          // [B, ceil(T / 16), D, N] or null
  long long u_b, u_t, d_b, d_t, z_b, z_t;        // element strides: rows, tokens
  long long Bm_b, Bm_t, Bm_g, Cm_b, Cm_t, Cm_g;  // rows, tokens, groups
  long long y_b, y_t;
  int B, T, D, G;
  int per_group;            // D / G
  int tiles;                // channel tiles per group
  int split;                // CTAs along the tokens (one cluster)
  int softplus, out_bf16;
  // backward
  const void* dy;           // strides y_b, y_t
  const float* dh_T;        // or null
  void *du, *ddelta, *dz;   // [B, T, D] contiguous
  float* dh0;               // or null
  float* part_bc;           // [tiles][B, T, G, 2 N] partial sums of dBm, dCm
  float* part_par;          // [B split][D N + D + D] partial sums of dA, dskip, d_delta_bias
};

constexpr int kSsmTile = 16;      // tokens per tile = tokens between snapshots
constexpr int kSsmMaxSplit = 8;   // CTAs along the tokens, at most (portable cluster size)

__device__ __forceinline__ int ssm_length(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// Sums over the lanes that differ in the bits LO .. HI of the lane number, of V
// values at once: while more than one is left, each step halves the set of
// values a lane carries. Afterwards v[0 .. left) hold the sums of the values
// first .. first + left - 1, the same on lanes that differ only in bits of plain steps.
template <int V, int HI, int LO>
struct LaneSum {
  static constexpr int steps(int hi) { return hi < LO ? 0 : 1 + steps(hi / 2); }
  static constexpr int scatter(int v) { return v <= 1 ? 0 : 1 + scatter(v / 2); }
  static constexpr int kScatter = steps(HI) < scatter(V) ? steps(HI) : scatter(V);
  static constexpr int left = V >> kScatter;
  // lane bits of the steps that only add (their lanes hold copies)
  static constexpr int copies =
      kScatter == steps(HI) ? 0 : (2 * (HI >> kScatter) - 1) & ~(LO - 1);

  __device__ __forceinline__ static void run(float (&v)[V], int lane) {
    int n = V;
#pragma unroll
    for (int off = HI; off >= LO; off >>= 1) {
      if (n > 1) {
        n >>= 1;
        const bool up = lane & off;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          if (j >= n) break;
          const float send = up ? v[j] : v[j + n];
          const float keep = up ? v[j + n] : v[j];
          v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
      }
    }
  }
  __device__ __forceinline__ static int first(int lane) {
    int i = 0, n = V;
#pragma unroll
    for (int off = HI; off >= LO; off >>= 1) {
      if (n > 1) {
        n >>= 1;
        if (lane & off) i += n;
      }
    }
    return i;
  }
};

__device__ __forceinline__ float2 dup2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// One channel's four states of a lane.
struct State4 {
  float2 lo, hi;
};

__device__ __forceinline__ State4 load_state(const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void store_state(float* p, const State4& s) {
  *reinterpret_cast<float4*>(p) = make_float4(s.lo.x, s.lo.y, s.hi.x, s.hi.y);
}

// L = N / 4 lanes hold one channel, four states each; a CTA of 128 threads has
// 128 / L channels and walks tiles of 16 tokens. The step sizes are worked out once
// for each (token, channel) as a tile is staged in shared memory, the next tile's
// inputs are on their way to registers meanwhile, and the L partial sums of an
// output are added for L tokens at once (L - 1 shuffles in place of L log2 L).
template <int L>
struct SsmFwdShape {
  static constexpr int NT = 128;
  static constexpr int N = 4 * L;
  static constexpr int CH = NT / L;             // channels
  static constexpr int IT = kSsmTile / L;       // (token, channel) items per thread and tile
  static constexpr int NBC = kSsmTile * N / NT; // entries of Bm (and Cm) per thread and tile
  static constexpr int YS = CH + 32 / L;        // row of the output tile: no bank conflicts
};

// With SPLIT, a cluster of p.split CTAs shares the tokens of a (row, channel tile) when rows and
// channels alone leave SMs idle: each CTA first runs its own span from a zero state
// for its end state and decay, the cluster exchanges those through distributed
// shared memory, and each runs its span again from the state it now knows. That is
// up to twice the exponentials, over `split` times the CTAs.
template <int L, typename InT, bool SPLIT>
__global__ void __launch_bounds__(128) ssm_fwd_kernel(const SsmParams p) {
  using S = SsmFwdShape<L>;
  constexpr int N = S::N, CH = S::CH, IT = S::IT;
  __shared__ float2 s_dt[kSsmTile][CH];  // dt, dt u
  __shared__ __align__(16) float s_B[kSsmTile][N], s_C[kSsmTile][N];
  __shared__ float s_y[kSsmTile][S::YS];
  __shared__ float4 s_end[SPLIT ? S::NT : 1], s_decay[SPLIT ? S::NT : 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = SPLIT ? blockIdx.x % p.split : 0;
  const int tile = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int g = tile / p.tiles;
  const int in_group = (tile - g * p.tiles) * CH;
  const int c0 = g * p.per_group + in_group;
  const int nch = min(CH, p.per_group - in_group);

  // as part of a channel's lanes
  const int my_ch = warp * (32 / L) + lane / L;
  const int n0 = (lane % L) * 4;
  const bool on = my_ch < nch;
  const size_t par = (size_t)(c0 + (on ? my_ch : 0)) * N + n0;
  State4 A = load_state(p.A + par);
  A.lo.x *= kLog2e; A.lo.y *= kLog2e; A.hi.x *= kLog2e; A.hi.y *= kLog2e;

  // as the owner of (token, channel) items: tokens it + L i of channel ic
  const int ic = tid % CH, it = tid / CH;
  const bool i_on = ic < nch;
  const int icc = c0 + (i_on ? ic : 0);
  const float bias = p.delta_bias ? p.delta_bias[icc] : 0.f;
  const float skip = p.skip ? p.skip[icc] : 0.f;

  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int len = ssm_length(p.lengths, b, p.T);
    const int n_tiles = (len + kSsmTile - 1) / kSsmTile;
    const int per = SPLIT ? (n_tiles + p.split - 1) / p.split : n_tiles;
    const int first = min(n_tiles, rank * per), last = min(n_tiles, first + per);

    const InT* up = static_cast<const InT*>(p.u) + b * p.u_b + icc;
    const InT* dp = static_cast<const InT*>(p.delta) + b * p.d_b + icc;
    const InT* zp = static_cast<const InT*>(p.z) + b * p.z_b + icc;
    const InT* Bp = static_cast<const InT*>(p.Bm) + b * p.Bm_b + g * p.Bm_g;
    const InT* Cp = static_cast<const InT*>(p.Cm) + b * p.Cm_b + g * p.Cm_g;

    InT ru[IT], rd[IT], rz[IT], rB[S::NBC], rC[S::NBC];
    auto fetch = [&](int k, bool all) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = k * kSsmTile + it + L * i;
        const bool have = i_on && t < len;
        ru[i] = have ? up[t * p.u_t] : from_f32<InT>(0.f);
        rd[i] = have ? dp[t * p.d_t] : from_f32<InT>(0.f);
        if (all && p.z) rz[i] = have ? zp[t * p.z_t] : from_f32<InT>(0.f);
      }
#pragma unroll
      for (int j = 0; j < S::NBC; ++j) {
        const int e = tid + S::NT * j;
        const int t = k * kSsmTile + e / N;
        rB[j] = t < len ? Bp[t * p.Bm_t + e % N] : from_f32<InT>(0.f);
        if (all) rC[j] = t < len ? Cp[t * p.Cm_t + e % N] : from_f32<InT>(0.f);
      }
    };
    // dt = 0 behind the length: there the state neither decays nor takes anything
    auto stage = [&](int k, bool all) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + L * i;
        const float x = to_f32(rd[i]) + bias;
        float dt = p.softplus ? softplus(x) : x;
        if (k * kSsmTile + t >= len || !i_on) dt = 0.f;
        s_dt[t][ic] = make_float2(dt, dt * to_f32(ru[i]));
      }
#pragma unroll
      for (int j = 0; j < S::NBC; ++j) {
        const int e = tid + S::NT * j;
        (&s_B[0][0])[e] = to_f32(rB[j]);
        if (all) (&s_C[0][0])[e] = to_f32(rC[j]);
      }
    };

    State4 h = {dup2(0.f), dup2(0.f)};
    const size_t hrow = (size_t)b * p.D * N + par;

    if constexpr (SPLIT) {
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      float sum_dt = 0.f;
      if (rank + 1 < p.split) {
        if (first < last) fetch(first, false);
        for (int k = first; k < last; ++k) {
          stage(k, false);
          __syncthreads();
          if (k + 1 < last) fetch(k + 1, false);
#pragma unroll
          for (int t = 0; t < kSsmTile; ++t) {
            const float2 d = s_dt[t][my_ch];
            const State4 Bv = load_state(&s_B[t][n0]);
            const float2 dt = dup2(d.x), dtu = dup2(d.y);
            h.lo = __ffma2_rn(ex2_2(__fmul2_rn(dt, A.lo)), h.lo, __fmul2_rn(dtu, Bv.lo));
            h.hi = __ffma2_rn(ex2_2(__fmul2_rn(dt, A.hi)), h.hi, __fmul2_rn(dtu, Bv.hi));
            sum_dt += d.x;
          }
          __syncthreads();
        }
      }
      const float2 lo = ex2_2(__fmul2_rn(dup2(sum_dt), A.lo));
      const float2 hi = ex2_2(__fmul2_rn(dup2(sum_dt), A.hi));
      s_end[tid] = make_float4(h.lo.x, h.lo.y, h.hi.x, h.hi.y);
      s_decay[tid] = make_float4(lo.x, lo.y, hi.x, hi.y);
      h = p.h0 ? load_state(p.h0 + hrow) : State4{dup2(0.f), dup2(0.f)};
      cluster.sync();
      for (int r = 0; r < rank; ++r) {
        const float4 e = *cluster.map_shared_rank(&s_end[tid], r);
        const float4 a = *cluster.map_shared_rank(&s_decay[tid], r);
        h.lo = __ffma2_rn(make_float2(a.x, a.y), h.lo, make_float2(e.x, e.y));
        h.hi = __ffma2_rn(make_float2(a.z, a.w), h.hi, make_float2(e.z, e.w));
      }
      cluster.sync();  // nobody writes or leaves while its shared memory is read
    } else {
      if (p.h0) h = load_state(p.h0 + hrow);
    }

    float* chunk = p.h_chunks;
    if (chunk) chunk += ((size_t)b * ((p.T + kSsmTile - 1) / kSsmTile) + first) * p.D * N + par;
    if (first < last) fetch(first, true);
    for (int k = first; k < last; ++k) {
      stage(k, true);
      float cu[IT], cz[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        cu[i] = to_f32(ru[i]);
        cz[i] = p.z ? to_f32(rz[i]) : 0.f;
      }
      __syncthreads();
      if (k + 1 < last) fetch(k + 1, true);
      if (chunk) {
        if (on) store_state(chunk, h);
        chunk += (size_t)p.D * N;
      }
#pragma unroll
      for (int t0 = 0; t0 < kSsmTile; t0 += L) {
        float v[L];
#pragma unroll
        for (int q = 0; q < L; ++q) {
          const float2 d = s_dt[t0 + q][my_ch];
          const State4 Bv = load_state(&s_B[t0 + q][n0]), Cv = load_state(&s_C[t0 + q][n0]);
          const float2 dt = dup2(d.x), dtu = dup2(d.y);
          h.lo = __ffma2_rn(ex2_2(__fmul2_rn(dt, A.lo)), h.lo, __fmul2_rn(dtu, Bv.lo));
          h.hi = __ffma2_rn(ex2_2(__fmul2_rn(dt, A.hi)), h.hi, __fmul2_rn(dtu, Bv.hi));
          const float2 s = __ffma2_rn(Cv.lo, h.lo, __fmul2_rn(Cv.hi, h.hi));
          v[q] = s.x + s.y;
        }
        LaneSum<L, L / 2, 1>::run(v, lane);
        s_y[t0 + (lane % L)][my_ch] = v[0];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = k * kSsmTile + it + L * i;
        float r = fmaf(skip, cu[i], s_y[it + L * i][ic]);
        if (p.z) r *= cz[i] * sigmoid_fast(cz[i]);
        if (i_on && t < len) {
          const long long o = b * p.y_b + t * p.y_t + icc;
          if (p.out_bf16)
            static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(r);
          else
            static_cast<float*>(p.y)[o] = r;
        }
      }
    }
    if ((!SPLIT || rank + 1 == p.split) && on) store_state(p.h_T + hrow, h);
  }
}

// ---- one token ----
// L lanes a channel; the state is read once and written once (HBM bound: 8 N
// bytes a channel against a few of input).
template <int L, typename InT>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmParams p) {
  constexpr int N = 4 * L;
  const int c = (blockIdx.x * 256 + threadIdx.x) / L;
  const int n0 = (threadIdx.x % L) * 4;
  // whole channels leave, but their lanes stay for the shuffles
  const bool on = c < p.D;
  const int cc = on ? c : p.D - 1;
  const int g = cc / p.per_group;
  const size_t par = (size_t)cc * N + n0;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    if (p.active && !p.active[b]) continue;
    float* hp = p.h_T + (size_t)b * p.D * N + par;
    State4 h = load_state(hp), A = load_state(p.A + par);
    float Bv[4], Cv[4];
    const InT* Bp = static_cast<const InT*>(p.Bm) + b * p.Bm_b + g * p.Bm_g + n0;
    const InT* Cp = static_cast<const InT*>(p.Cm) + b * p.Cm_b + g * p.Cm_g + n0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Bv[j] = to_f32(Bp[j]);
      Cv[j] = to_f32(Cp[j]);
    }
    const float u = to_f32(static_cast<const InT*>(p.u)[b * p.u_b + cc]);
    float dt = to_f32(static_cast<const InT*>(p.delta)[b * p.d_b + cc]);
    const float z = p.z ? to_f32(static_cast<const InT*>(p.z)[b * p.z_b + cc]) : 0.f;
    if (p.delta_bias) dt += p.delta_bias[cc];
    if (p.softplus) dt = softplus(dt);
    const float x = dt * kLog2e, dtu = dt * u;
    h.lo.x = fmaf(ex2(x * A.lo.x), h.lo.x, dtu * Bv[0]);
    h.lo.y = fmaf(ex2(x * A.lo.y), h.lo.y, dtu * Bv[1]);
    h.hi.x = fmaf(ex2(x * A.hi.x), h.hi.x, dtu * Bv[2]);
    h.hi.y = fmaf(ex2(x * A.hi.y), h.hi.y, dtu * Bv[3]);
    float r = fmaf(Cv[0], h.lo.x, Cv[1] * h.lo.y) + fmaf(Cv[2], h.hi.x, Cv[3] * h.hi.y);
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
    if (!on) continue;
    store_state(hp, h);
    if (threadIdx.x % L == 0) {
      if (p.skip) r = fmaf(p.skip[cc], u, r);
      if (p.z) r *= z * sigmoid_fast(z);
      const long long o = b * p.y_b + cc;
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(r);
      else
        static_cast<float*>(p.y)[o] = r;
    }
  }
}

}  // namespace ttt
