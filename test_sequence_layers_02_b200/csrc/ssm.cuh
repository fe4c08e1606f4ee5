// Selective state space scan, forward and one-token step (include/ttt_ssm.h has the
// formulas). The backward is in ssm_bwd.cuh.
//
// Work: one exponential, one multiply and two multiply-adds for each of the N
// states of every (token, channel), against four 2- or 4-byte elements of
// traffic. With every exponential on the special-function units (16 lanes per clock and SM), as here, these bind
// first at N = 16: (N + 4) / 16 clocks per (token, channel) with the softplus and the gate counted,
// where HBM would take a quarter of that in bf16. Measured, bf16, N = 16: two prompts of 32768
// tokens by 2048 channels 1.32 ms (0.58 ms of special functions; 128 CTAs on 148 SMs), in fp32 1.39; 16 of 2048 by
// 1536 0.41 ms (0.22). The SPLIT builds, and single elements at N = 8 and 32, spill up to 420 bytes a thread at
// the 80 registers that two CTAs an SM leave. What is left is the latency of the loop, about 80 clocks a token for
// a warp of the recurrence that shares its scheduler with staging and output, 57 alone; without
// its exponentials it still takes 69.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

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
  // Element strides: batch rows, groups, tokens. The bytes of 16 tokens fit an int (checked).
  long long u_b, d_b, z_b, Bm_b, Bm_g, Cm_b, Cm_g, y_b;
  int u_t, d_t, z_t, Bm_t, Cm_t, y_t;
  int B, T, D, G;
  int per_group;            // D / G
  int tiles;                // channel tiles per group
  int vec;                  // rows can be read and written in packs of 4
  int split;                // CTAs along the tokens (one cluster)
  int softplus, out_bf16;
  int pad_zero;             // y = 0 behind a length and in rows that are not active
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

// A log2 e, kept finite: with an infinite one a step of 0 would decay by exp(0 inf), which is no number. So an
// A beyond 2.35e38 counts as that (its decay over any step above 1e-36 is 0 either way).
__device__ __forceinline__ float scaled_rate(float A) {
  constexpr float kMax = 3.402823466e38f;
  const float x = A * kLog2e;
  return x < -kMax ? -kMax : x > kMax ? kMax : x;
}
__device__ __forceinline__ float2 scaled_rate2(float2 A) {
  return make_float2(scaled_rate(A.x), scaled_rate(A.y));
}
// The same in fewer instructions, for the step, which does it for every few rows (512 x 2048 channels: 22.4 us,
// with the form above 23.5). The prompt's loop comes out slower with it: 1.37 against 1.32 ms for two of 32768 by 2048.
__device__ __forceinline__ float scaled_rate_step(float A) {
  float x = A * kLog2e;  // (and NaN stays NaN)
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(3.402823466e38f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-3.402823466e38f));
  return x;
}

// exp(dt A), the decay of one token, for A scaled by log2 e.
__device__ __forceinline__ float2 decay2(float2 dt, float2 A) {
  return ex2_2(__ffma2_rn(dt, A, dup2(kDecayBias)));
}

// d h + a, what is left of a state h behind a span with the decay d and the span's own, where d alone may leave
// fp32's range: a state that grows need not, nothing stays nothing, and a small one is multiplied in
// steps. x is the exponent of d, for ex2.
__device__ __forceinline__ float carry_span(float d, float x, float h, float a) {
  if (d != __int_as_float(0x7f800000) || h != h) return fmaf(d, h, a);
  if (h == 0.f) return a;
  const float q = ex2(0.25f * x);  // h >= 2^-149: beyond 4 * 128 it is out of range either way
  return fmaf(q * (q * (q * h)), q, a);
}

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

// P states of one channel in a lane, as pairs for the paired fp32 instructions.
template <int P>
struct States {
  float2 v[P / 2];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) v[i] = dup2(0.f);
  }
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (P == 2) {
      v[0] = *reinterpret_cast<const float2*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < P / 4; ++i) {
        const float4 x = reinterpret_cast<const float4*>(p)[i];
        v[2 * i] = make_float2(x.x, x.y);
        v[2 * i + 1] = make_float2(x.z, x.w);
      }
    }
  }
  __device__ __forceinline__ bool finite() const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) s = fmaf(0.f, v[i].x, fmaf(0.f, v[i].y, s));
    return s == 0.f;
  }
  // carry_span for all states: a span's decays and own states by index, its sum of step sizes
  template <typename Decay, typename Own>
  __device__ __forceinline__ void carry(Decay decay, Own own, float sum_dt, const States& A) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 d = decay(i), a = own(i);
      v[i] = make_float2(carry_span(d.x, sum_dt * A.v[i].x, v[i].x, a.x),
                         carry_span(d.y, sum_dt * A.v[i].y, v[i].y, a.y));
    }
  }
  __device__ __forceinline__ void store(float* p) const {
    if constexpr (P == 2) {
      *reinterpret_cast<float2*>(p) = v[0];
    } else {
#pragma unroll
      for (int i = 0; i < P / 4; ++i)
        reinterpret_cast<float4*>(p)[i] =
            make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    }
  }
};

// Copy BYTES (4, 8 or 16) to shared memory without a register; `have` false: zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool have) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES),
               "r"(have ? BYTES : 0) : "memory");
}

// A CTA has 32 CW channels. A warp of the recurrence holds P of the N states of 32 channels, a
// channel a lane, so that the tile's Bm and Cm are the same address for all its lanes; N / P
// warps share a channel and leave their parts of its output in shared memory. Two more sets
// of four warps do everything around the recurrence once for each (token, channel), VEC channels
// a thread: one stages a tile of 16 tokens in shared memory, with its step sizes and gates, one
// adds the parts and writes out. One barrier a tile: between two of them the first
// run tile k, the second stage tile k + 1 in the other half of shared memory, the third write
// out tile k - 1. The loads of the tiles behind that are on their way: RING tiles in packs of
// 4 elements, which go to a ring in shared memory by asynchronous copies (a thread
// reads back what it copied, so the ring needs no barrier), or two tiles of single
// elements in registers where rows do not allow packs. A lone CTA on an SM lives by that
// depth: a tile takes it half a microsecond, a load from HBM more than that.
template <int N, int P, typename InT, int VEC>
struct SsmFwdShape {
  static constexpr int L = N / P;               // warps that share a channel
  static constexpr int CW = L < 4 ? 4 / L : 1;  // blocks of 32 channels
  static constexpr int CH = 32 * CW;
  static constexpr int RT = CH * L;             // threads of the recurrence
  static constexpr int HT = 128;                // threads that stage, and threads that write out
  static constexpr int NT = RT + 2 * HT;
  static constexpr int QUADS = CH / VEC;        // items of a token
  static constexpr int TS = HT / QUADS;         // tokens between a helper's items
  static constexpr int IT = kSsmTile / TS;      // items per helper and tile
  static constexpr int BCQ = kSsmTile * N / VEC;             // packs of Bm (and Cm) in a tile
  static constexpr int NBC = (BCQ + HT - 1) / HT;            // ... per helper
  static constexpr int GROUP = 2;               // tokens whose exponentials are taken at once
  static constexpr int RING = VEC == 1 ? 0 : 16 / (int)sizeof(InT);
  static_assert(HT % QUADS == 0 && kSsmTile % TS == 0, "whole items");
  static_assert(BCQ % HT == 0 || BCQ < HT, "whole packs");
  struct Smem {
    alignas(16) float2 dt[2][kSsmTile][CH];     // dt, dt u
    alignas(16) float2 gate[4][kSsmTile][CH];   // SiLU(z), SiLU(z) skip u: read two tiles later
    alignas(16) float B[2][kSsmTile][N];
    alignas(16) float C[2][kSsmTile][N];
    alignas(16) float y[2][kSsmTile][L][CH];    // the warps' parts of the read-out
    struct Slot {
      Pack<InT, VEC> u[IT][HT], d[IT][HT], z[IT][HT], B[NBC][HT], C[NBC][HT];
    } ring[RING > 0 ? RING : 1];
  };
};

// With SPLIT, a cluster of p.split CTAs shares the tokens of a (row, channel tile) when rows and
// channels alone leave SMs idle: each CTA first runs its own span from a zero state
// for its end state and decay, the cluster exchanges those through distributed
// shared memory, and each runs its span again from the state it now knows. That is
// up to twice the exponentials, over `split` times the CTAs.
template <int N, int P, typename InT, int VEC, bool SPLIT>
__global__ void __launch_bounds__(SsmFwdShape<N, P, InT, VEC>::NT, N < 64 ? 2 : 1) ssm_fwd_kernel(const SsmParams p) {
  using S = SsmFwdShape<N, P, InT, VEC>;
  constexpr int L = S::L, CH = S::CH, IT = S::IT, TS = S::TS, RT = S::RT, HT = S::HT;
  constexpr int NBC = S::NBC, QUADS = S::QUADS, RING = S::RING;
  using In = Pack<InT, VEC>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(smem_raw);
  __shared__ float2 s_end[SPLIT ? P / 2 : 1][SPLIT ? RT : 1], s_decay[SPLIT ? P / 2 : 1][SPLIT ? RT : 1];
  __shared__ float s_sum[SPLIT ? RT : 1];

  enum { kRecur, kStage, kWrite };
  const int role = threadIdx.x < RT ? kRecur : threadIdx.x < RT + HT ? kStage : kWrite;
  const int tid = role == kRecur ? threadIdx.x : (threadIdx.x - RT) % HT;  // within the role
  const int rank = SPLIT ? blockIdx.x % p.split : 0;
  const int tile = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int g = tile / p.tiles;
  const int in_group = (tile - g * p.tiles) * CH;
  const int c0 = g * p.per_group + in_group;
  const int nch = min(CH, p.per_group - in_group);

  // the recurrence: states n0 .. n0 + P - 1 of channel my_ch
  const int part = (tid >> 5) % L;
  const int my_ch = (tid >> 5) / L * 32 + (tid & 31);
  const int n0 = part * P;
  const bool on = role == kRecur && my_ch < nch;
  const size_t par = (size_t)(c0 + (on ? my_ch : 0)) * N + n0;
  States<P> A;
  A.load(p.A + par);
#pragma unroll
  for (int i = 0; i < P / 2; ++i) A.v[i] = scaled_rate2(A.v[i]);

  // the others: tokens it + TS i of channels ic .. ic + VEC - 1
  const int ic = tid % QUADS * VEC, it = tid / QUADS;
  const bool i_on = ic < nch;
  const int icc = c0 + (i_on ? ic : 0);
  float bias[VEC], skip[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    bias[q] = p.delta_bias ? p.delta_bias[icc + q] : 0.f;
    skip[q] = p.skip ? p.skip[icc + q] : 0.f;
  }

  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int len = ssm_length(p.lengths, b, p.T);
    const int n_tiles = (len + kSsmTile - 1) / kSsmTile;
    const int per = SPLIT ? (n_tiles + p.split - 1) / p.split : n_tiles;
    const int first = min(n_tiles, rank * per), last = min(n_tiles, first + per);

    // ---- around the recurrence ----
    // Running pointers to a helper's items and packs of the tile to be fetched next.
    const InT *up = nullptr, *dp = nullptr, *zp = nullptr, *Bp = nullptr, *Cp = nullptr;
    const bool bc_on = S::BCQ % HT == 0 || tid < S::BCQ;
    constexpr int BROW = N / VEC;          // packs of a token
    constexpr int BS = HT / BROW;          // tokens between a helper's packs
    const int bt = tid / BROW, bn = tid % BROW * VEC;
    struct Regs {
      In u[IT], d[IT], z[IT], B[NBC], C[NBC];
    };
    auto advance = [&](bool all) {
      up += kSsmTile * p.u_t;
      dp += kSsmTile * p.d_t;
      Bp += kSsmTile * p.Bm_t;
      if (all) {
        zp += kSsmTile * p.z_t;
        Cp += kSsmTile * p.Cm_t;
      }
    };
    // The inputs of tile k, in order, to registers (0 behind the length). `all`: those of the
    // read-out too.
    auto fetch = [&](Regs& r, int k, bool all) {
      auto at = [](const InT* q) { return *reinterpret_cast<const In*>(q); };
      const int left = len - k * kSsmTile;
      const In none = {};
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        r.u[i] = r.d[i] = r.z[i] = none;
        if (it + TS * i < left) {
          r.u[i] = at(up + TS * i * p.u_t);
          r.d[i] = at(dp + TS * i * p.d_t);
          if (all && p.z) r.z[i] = at(zp + TS * i * p.z_t);
        }
      }
#pragma unroll
      for (int j = 0; j < NBC; ++j) {
        r.B[j] = r.C[j] = none;
        if (bc_on && bt + BS * j < left) {
          r.B[j] = at(Bp + BS * j * p.Bm_t);
          if (all) r.C[j] = at(Cp + BS * j * p.Cm_t);
        }
      }
      advance(all);
    };
    // The same to the ring (one group of copies a tile, also an empty one behind the last) ...
    auto send = [&](int k, bool all) {
      if (k < last) {
        typename S::Smem::Slot& r = sm.ring[k % (RING > 0 ? RING : 1)];
        const int left = len - k * kSsmTile;
        constexpr int W = sizeof(In) < 4 ? 4 : sizeof(In);  // (single bf16 have no ring)
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const bool have = it + TS * i < left;
          copy_async<W>(&r.u[i][tid], have ? up + TS * i * p.u_t : up, have);
          copy_async<W>(&r.d[i][tid], have ? dp + TS * i * p.d_t : dp, have);
          if (all && p.z) copy_async<W>(&r.z[i][tid], have ? zp + TS * i * p.z_t : zp, have);
        }
        if (bc_on) {
#pragma unroll
          for (int j = 0; j < NBC; ++j) {
            const bool have = bt + BS * j < left;
            copy_async<W>(&r.B[j][tid], have ? Bp + BS * j * p.Bm_t : Bp, have);
            if (all) copy_async<W>(&r.C[j][tid], have ? Cp + BS * j * p.Cm_t : Cp, have);
          }
        }
        advance(all);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // ... and from the ring: the oldest of the RING groups under way.
    auto receive = [&](Regs& r, int k, bool all) {
      asm volatile("cp.async.wait_group %0;" ::"n"(RING > 0 ? RING - 1 : 0) : "memory");
      const typename S::Smem::Slot& f = sm.ring[k % (RING > 0 ? RING : 1)];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        r.u[i] = f.u[i][tid];
        r.d[i] = f.d[i][tid];
        if (all && p.z) r.z[i] = f.z[i][tid];
      }
      if (bc_on) {
#pragma unroll
        for (int j = 0; j < NBC; ++j) {
          r.B[j] = f.B[j][tid];
          if (all) r.C[j] = f.C[j][tid];
        }
      }
    };
    // dt = 0 behind the length: there the state neither decays nor takes anything
    auto stage = [&](const Regs& r, int k, bool all) {
      const int h = k & 1;
      const int left = len - k * kSsmTile;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + TS * i;
        float dt[VEC], u[VEC];
        r.d[i].widen(dt);
        r.u[i].widen(u);
#pragma unroll
        for (int q = 0; q < VEC; ++q) dt[q] += bias[q];
        if (p.softplus) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) dt[q] = softplus(dt[q]);
        }
        if (t >= left) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) dt[q] = 0.f;
        }
        if constexpr (VEC == 1) {
          sm.dt[h][t][ic] = make_float2(dt[0], dt[0] * u[0]);
        } else {
          float4* o = reinterpret_cast<float4*>(&sm.dt[h][t][ic]);
#pragma unroll
          for (int q = 0; q < VEC; q += 2)
            o[q / 2] = make_float4(dt[q], dt[q] * u[q], dt[q + 1], dt[q + 1] * u[q + 1]);
        }
        if (all) {
          float f[VEC];
#pragma unroll
          for (int q = 0; q < VEC; ++q) f[q] = 1.f;
          if (p.z) {
            r.z[i].widen(f);
#pragma unroll
            for (int q = 0; q < VEC; ++q) f[q] *= sigmoid_fast(f[q]);
          }
          if constexpr (VEC == 1) {
            sm.gate[k & 3][t][ic] = make_float2(f[0], f[0] * (skip[0] * u[0]));
          } else {
            float4* o = reinterpret_cast<float4*>(&sm.gate[k & 3][t][ic]);
#pragma unroll
            for (int q = 0; q < VEC; q += 2)
              o[q / 2] = make_float4(f[q], f[q] * (skip[q] * u[q]), f[q + 1],
                                     f[q + 1] * (skip[q + 1] * u[q + 1]));
          }
        }
      }
      if (bc_on) {
#pragma unroll
        for (int j = 0; j < NBC; ++j) {
          float v[VEC];
          r.B[j].widen(v);
          store_vec<float, VEC>(&sm.B[h][bt + BS * j][bn], v);
          if (all) {
            r.C[j].widen(v);
            store_vec<float, VEC>(&sm.C[h][bt + BS * j][bn], v);
          }
        }
      }
    };
    __nv_bfloat16* y16 = nullptr;
    float* y32 = nullptr;
    // The outputs of tile k, from the warps' parts.
    auto write_out = [&](int k) {
      const int h = k & 1;
      const int left = i_on ? len - k * kSsmTile : 0;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + TS * i;
        float r[VEC];
        load_vec<float, VEC>(&sm.y[h][t][0][ic], r);
#pragma unroll
        for (int j = 1; j < L; ++j) {
          float v[VEC];
          load_vec<float, VEC>(&sm.y[h][t][j][ic], v);
#pragma unroll
          for (int q = 0; q < VEC; ++q) r[q] += v[q];
        }
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          const float2 f = sm.gate[k & 3][t][ic + q];
          r[q] = fmaf(f.x, r[q], f.y);
        }
        if (t < left) {
          if (p.out_bf16)
            store_vec<__nv_bfloat16, VEC>(y16 + TS * i * p.y_t, r);
          else
            store_vec<float, VEC>(y32 + TS * i * p.y_t, r);
        }
      }
      y16 += kSsmTile * p.y_t;
      y32 += kSsmTile * p.y_t;
    };
    // A pass over the tiles; the roles meet at one barrier a tile (and, with the read-out, one behind
    // the last): between two of them tile k is run, k + 1 staged and k - 1 written out.
    auto stage_all = [&](bool all) {
      const long long t0 = (long long)first * kSsmTile + it, e0 = (long long)first * kSsmTile + bt;
      up = static_cast<const InT*>(p.u) + b * p.u_b + t0 * p.u_t + icc;
      dp = static_cast<const InT*>(p.delta) + b * p.d_b + t0 * p.d_t + icc;
      zp = static_cast<const InT*>(p.z) + b * p.z_b + t0 * p.z_t + icc;
      Bp = static_cast<const InT*>(p.Bm) + b * p.Bm_b + g * p.Bm_g + e0 * p.Bm_t + bn;
      Cp = static_cast<const InT*>(p.Cm) + b * p.Cm_b + g * p.Cm_g + e0 * p.Cm_t + bn;
      if constexpr (RING > 0) {
        Regs r;
        for (int j = 0; j < RING; ++j) send(first + j, all);
        receive(r, first, all);
        stage(r, first, all);
        send(first + RING, all);
        for (int k = first; k < last; ++k) {
          __syncthreads();
          if (k + 1 < last) {
            receive(r, k + 1, all);
            stage(r, k + 1, all);
            send(k + 1 + RING, all);
          }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      } else {
        Regs sets[2];
        fetch(sets[0], first, all);
        if (first + 1 < last) fetch(sets[1], first + 1, all);
        stage(sets[0], first, all);
        if (first + 2 < last) fetch(sets[0], first + 2, all);
        for (int k0 = first; k0 < last; k0 += 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = k0 + j;
            if (k >= last) break;
            __syncthreads();
            if (k + 1 < last) {
              stage(sets[j ^ 1], k + 1, all);
              if (k + 3 < last) fetch(sets[j ^ 1], k + 3, all);
            }
          }
        }
      }
      if (all) __syncthreads();
    };
    auto write_all = [&]() {
      const long long t0 = (long long)first * kSsmTile + it;
      y16 = static_cast<__nv_bfloat16*>(p.y) + b * p.y_b + t0 * p.y_t + icc;
      y32 = static_cast<float*>(p.y) + b * p.y_b + t0 * p.y_t + icc;
      for (int k = first; k < last; ++k) {
        __syncthreads();
        if (k > first) write_out(k - 1);
      }
      __syncthreads();
      write_out(last - 1);
    };

    // ---- the recurrence ----
    States<P> h;
    h.zero();
    const size_t hrow = (size_t)b * p.D * N + par;
    float sum_dt = 0.f;
    // Tile k; `read`: with the read-out. The exponentials of the next GROUP tokens stand before
    // the chain of these in the program, so that the two overlap.
    auto run = [&](int k, bool read) {
      constexpr int GROUP = S::GROUP;
      const int half = k & 1;
      States<P> a[2][GROUP], x[2][GROUP], c[2][GROUP];
      auto prepare = [&](int t0, States<P>* ga, States<P>* gx, States<P>* gc) {
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          const float2 d = sm.dt[half][t0 + j][my_ch];
          States<P> Bv;
          Bv.load(&sm.B[half][t0 + j][n0]);
          if (read) gc[j].load(&sm.C[half][t0 + j][n0]);
#pragma unroll
          for (int i = 0; i < P / 2; ++i) {
            ga[j].v[i] = decay2(dup2(d.x), A.v[i]);
            gx[j].v[i] = __fmul2_rn(dup2(d.y), Bv.v[i]);
          }
          if (!read) sum_dt += d.x;
        }
      };
      prepare(0, a[0], x[0], c[0]);
#pragma unroll
      for (int t0 = 0; t0 < kSsmTile; t0 += GROUP) {
        const int cur = (t0 / GROUP) & 1;
        if (t0 + GROUP < kSsmTile) prepare(t0 + GROUP, a[cur ^ 1], x[cur ^ 1], c[cur ^ 1]);
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          float2 s;
#pragma unroll
          for (int i = 0; i < P / 2; ++i) {
            h.v[i] = __ffma2_rn(a[cur][j].v[i], h.v[i], x[cur][j].v[i]);
            if (read)
              s = i == 0 ? __fmul2_rn(c[cur][j].v[i], h.v[i])
                         : __ffma2_rn(c[cur][j].v[i], h.v[i], s);
          }
          if (read) sm.y[half][t0 + j][part][my_ch] = s.x + s.y;
        }
      }
    };

    if constexpr (SPLIT) {
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      if (rank + 1 < p.split && first < last) {
        if (role == kStage) {
          stage_all(false);
        } else {
          for (int k = first; k < last; ++k) {
            __syncthreads();
            if (role == kRecur) run(k, false);
          }
        }
      }
      if (role == kRecur) {
        s_sum[tid] = sum_dt;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          s_end[i][tid] = h.v[i];
          s_decay[i][tid] = decay2(dup2(sum_dt), A.v[i]);
        }
        h.zero();
        if (p.h0) h.load(p.h0 + hrow);
      }
      cluster.sync();
      if (role == kRecur) {
        for (int r = 0; r < rank; ++r) {
#pragma unroll
          for (int i = 0; i < P / 2; ++i)
            h.v[i] = __ffma2_rn(*cluster.map_shared_rank(&s_decay[i][tid], r), h.v[i],
                                *cluster.map_shared_rank(&s_end[i][tid], r));
        }
        if (!h.finite()) {  // once more, with care
          h.zero();
          if (p.h0) h.load(p.h0 + hrow);
          for (int r = 0; r < rank; ++r)
            h.carry([&](int i) { return *cluster.map_shared_rank(&s_decay[i][tid], r); },
                    [&](int i) { return *cluster.map_shared_rank(&s_end[i][tid], r); },
                    *cluster.map_shared_rank(&s_sum[tid], r), A);
        }
      }
      cluster.sync();  // nobody writes or leaves while its shared memory is read
    } else {
      if (role == kRecur && p.h0) h.load(p.h0 + hrow);
    }

    if (role == kStage) {
      if (first < last) stage_all(true);
    } else if (role == kWrite) {
      if (first < last) write_all();
      if (p.pad_zero && i_on) {
        const float none[VEC] = {};
        const int step = TS * (SPLIT ? p.split : 1);
        for (int t = len + it + TS * rank; t < p.T; t += step) {
          const long long o = b * p.y_b + (long long)t * p.y_t + icc;
          if (p.out_bf16)
            store_vec<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(p.y) + o, none);
          else
            store_vec<float, VEC>(static_cast<float*>(p.y) + o, none);
        }
      }
    } else {
      float* chunk = p.h_chunks;
      if (chunk) chunk += ((size_t)b * ((p.T + kSsmTile - 1) / kSsmTile) + first) * p.D * N + par;
      for (int k = first; k < last; ++k) {
        __syncthreads();
        if (chunk) {
          if (on) h.store(chunk);
          chunk += (size_t)p.D * N;
        }
        run(k, true);
      }
      if (first < last) __syncthreads();
      if ((!SPLIT || rank + 1 == p.split) && on) h.store(p.h_T + hrow);
    }
    if (b + gridDim.y < p.B) __syncthreads();  // the last tile's gates are still being read
  }
}

// ---- one token ----
// L lanes a channel, a float4 of its state each; the state is read once and written once (8 N bytes a
// channel against a few of input), and what stands in HBM's way is the issue of
// everything else. So a thread takes the same states of ROWS batch rows, with one read of the
// parameters and all loads on their way together, while a row's step size, gate and output
// are worked out by one of the channel's lanes alone: the step size goes to the others by a
// shuffle, the sums of the read-out scatter to the row's lane. (512 rows of 2048 channels, N = 16, bf16: 143 MB, 22 us
// where the 67 MB of state are still in L2, as when one call follows another on it, with the scalars of every row
// in every lane 31 us; 29 us in a run over the states of 8 layers, three quarters of the copy bandwidth, where the
// loads' latency binds.)
template <int L, typename InT, int VEC, int ROWS>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmParams p) {
  constexpr int N = 4 * L;
  using Sum = LaneSum<ROWS, L / 2, 1>;
  const int lane = threadIdx.x & 31;
  const int c = (blockIdx.x * 256 + threadIdx.x) / L;
  const int n0 = (threadIdx.x % L) * 4;
  // lanes of channels that are not there stay for the shuffles
  const bool on = c < p.D;
  const int cc = on ? c : p.D - 1;
  const int g = cc / p.per_group;
  const size_t par = (size_t)cc * N + n0;
  State4 A = load_state(p.A + par);
  A.lo = make_float2(scaled_rate_step(A.lo.x), scaled_rate_step(A.lo.y));
  A.hi = make_float2(scaled_rate_step(A.hi.x), scaled_rate_step(A.hi.y));
  const float bias = p.delta_bias ? p.delta_bias[cc] : 0.f;
  const float skip = p.skip ? p.skip[cc] : 0.f;
  const int mine = Sum::first(lane % L);  // the row of this lane's scalars
  for (int b0 = blockIdx.y * ROWS; b0 < p.B; b0 += gridDim.y * ROWS) {
    State4 h[ROWS], Bv[ROWS], Cv[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      // Also for rows that are not active: their loads would wait for the flag, and only the
      // stores matter.
      const int b = min(b0 + r, p.B - 1);
      h[r] = load_state(p.h_T + (size_t)b * p.D * N + par);
      const InT* Bp = static_cast<const InT*>(p.Bm) + b * p.Bm_b + g * p.Bm_g + n0;
      const InT* Cp = static_cast<const InT*>(p.Cm) + b * p.Cm_b + g * p.Cm_g + n0;
      float v[4], w[4];
      if constexpr (VEC == 4) {
        load_vec<InT, 4>(Bp, v);
        load_vec<InT, 4>(Cp, w);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = to_f32(Bp[j]);
          w[j] = to_f32(Cp[j]);
        }
      }
      Bv[r] = {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
      Cv[r] = {make_float2(w[0], w[1]), make_float2(w[2], w[3])};
    }
    const int bm = min(b0 + mine, p.B - 1);
    const float u = to_f32(static_cast<const InT*>(p.u)[bm * p.u_b + cc]);
    float dt = to_f32(static_cast<const InT*>(p.delta)[bm * p.d_b + cc]) + bias;
    const float z = p.z ? to_f32(static_cast<const InT*>(p.z)[bm * p.z_b + cc]) : 0.f;
    if (p.softplus) dt = softplus(dt);
    const float dtu = dt * u;
    float v[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int from = (lane & ~(L - 1)) + r * (L / ROWS);
      const float2 d = dup2(__shfl_sync(0xffffffffu, dt, from));
      const float2 x = dup2(__shfl_sync(0xffffffffu, dtu, from));
      h[r].lo = __ffma2_rn(decay2(d, A.lo), h[r].lo, __fmul2_rn(x, Bv[r].lo));
      h[r].hi = __ffma2_rn(decay2(d, A.hi), h[r].hi, __fmul2_rn(x, Bv[r].hi));
      const float2 y = __ffma2_rn(Cv[r].lo, h[r].lo, __fmul2_rn(Cv[r].hi, h[r].hi));
      v[r] = y.x + y.y;
      if (on && b0 + r < p.B && (!p.active || p.active[b0 + r]))
        store_state(p.h_T + (size_t)(b0 + r) * p.D * N + par, h[r]);
    }
    Sum::run(v, lane);
    float y = fmaf(skip, u, v[0]);
    if (p.z) y *= z * sigmoid_fast(z);
    if (on && b0 + mine < p.B && (lane % L & Sum::copies) == 0) {
      const bool live = !p.active || p.active[bm];
      if (live || p.pad_zero) {
        if (!live) y = 0.f;
        const long long o = bm * p.y_b + cc;
        if (p.out_bf16)
          static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(y);
        else
          static_cast<float*>(p.y)[o] = y;
      }
    }
  }
}

}  // namespace ttt
