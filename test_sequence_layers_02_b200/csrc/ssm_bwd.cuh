// Selective state space scan, backward (include/ttt_ssm.h).
//
// With g the gradient that reaches h_t, r the read-out before the gate and
// q_t = a_t h_{t-1} (a_t = exp(dt_t A)), token by token from the last:
//
//     g  += Cm_t dr_t                        dr = dy SiLU(z)
//     h_t = q_t + dt_t u_t Bm_t
//     dCm_t += dr_t h_t,  dBm_t += g dt_t u_t        (summed over the channels)
//     s1 = sum_n g Bm,  s2 = sum_n g q A,  s3 = sum_n Cm h
//     du = dt s1 + skip dr,  d(dt) = s2 + u s1,  dz = dy (s3 + skip u) SiLU'(z)
//     dA += g q dt                           (summed over rows and tokens)
//     g  <- a_t g
//
// The states come from the forward's snapshots, 16 tokens apart: a tile is walked
// in two halves of 8 tokens, whose decays and q stay in registers between the
// way forward and the way back (the later half first, after a run over the earlier
// half for its end state: half a tile's exponentials more, where snapshots every 8
// tokens would be as much traffic as u, delta, z and dy together).
//
// Work: about 20 fp32 operations, 1.5 exponentials and two lane sums per state of
// every (token, channel); the fp32 and shuffle issue binds, not HBM.
//
// The sums over the channels of dBm and dCm: 8 values a lane are added over a warp's
// channels by scatter steps (7 shuffles for 8 values), over the CTA's warps
// in shared memory, and over the channel tiles from partial sums in global memory
// in tile order. No atomics: the same bits on every call.
#pragma once

#include "ssm.cuh"

namespace ttt {

template <int L>
struct SsmBwdShape {
  static constexpr int NT = 256;
  static constexpr int N = 4 * L;
  static constexpr int CH = NT / L;
  static constexpr int IT = kSsmTile / L;
  static constexpr int NBC = (kSsmTile * N + NT - 1) / NT;
  static constexpr int ROW = CH + 32 / L;       // row of the s1, s2, s3 tiles
  static constexpr int V = L < 4 ? L : 4;       // tokens whose s-sums are added at once
  static constexpr int kHalf = 8;
  struct Smem {
    float2 dt[kSsmTile][CH];                    // dt, dt u
    float dr[kSsmTile][CH];
    alignas(16) float B[kSsmTile][N];
    alignas(16) float C[kSsmTile][N];
    float s1[kSsmTile][ROW], s2[kSsmTile][ROW], s3[kSsmTile][ROW];
    alignas(16) float part[NT / 32][kSsmTile][2 * N];
    float4 start[NT], decay[NT];                // exchange of a cluster
  };
};

template <int L, typename InT, bool SPLIT>
__global__ void __launch_bounds__(256) ssm_bwd_kernel(const SsmParams p) {
  using S = SsmBwdShape<L>;
  constexpr int N = S::N, CH = S::CH, IT = S::IT, NT = S::NT, V = S::V, kHalf = S::kHalf;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(smem_raw);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = SPLIT ? blockIdx.x % p.split : 0;
  const int tile = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int g = tile / p.tiles;
  const int tile_in_group = tile - g * p.tiles;
  const int in_group = tile_in_group * CH;
  const int c0 = g * p.per_group + in_group;
  const int nch = min(CH, p.per_group - in_group);

  const int my_ch = warp * (32 / L) + lane / L;
  const int n0 = (lane % L) * 4;
  const bool on = my_ch < nch;
  const size_t par = (size_t)(c0 + (on ? my_ch : 0)) * N + n0;
  State4 A = load_state(p.A + par);
  A.lo.x *= kLog2e; A.lo.y *= kLog2e; A.hi.x *= kLog2e; A.hi.y *= kLog2e;

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
    const long long yb = b * p.y_b + icc;
    const size_t ob = (size_t)b * p.T * p.D + icc;  // du, ddelta, dz

    InT ru[IT], rd[IT], rz[IT], rB[S::NBC], rC[S::NBC];
    float rg[IT];
    auto fetch = [&](int k, bool all) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = k * kSsmTile + it + L * i;
        const bool have = i_on && t < len;
        if (all) ru[i] = have ? up[(long long)t * p.u_t] : from_f32<InT>(0.f);
        rd[i] = have ? dp[(long long)t * p.d_t] : from_f32<InT>(0.f);
        if (p.z) rz[i] = have ? zp[(long long)t * p.z_t] : from_f32<InT>(0.f);
        rg[i] = 0.f;
        if (have)
          rg[i] = p.out_bf16
                      ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.dy)[yb + (long long)t * p.y_t])
                      : static_cast<const float*>(p.dy)[yb + (long long)t * p.y_t];
      }
#pragma unroll
      for (int j = 0; j < S::NBC; ++j) {
        const int e = tid + NT * j;
        const int t = k * kSsmTile + e / N;
        const bool have = e < kSsmTile * N && t < len;
        if (all) rB[j] = have ? Bp[(long long)t * p.Bm_t + e % N] : from_f32<InT>(0.f);
        rC[j] = have ? Cp[(long long)t * p.Cm_t + e % N] : from_f32<InT>(0.f);
      }
    };
    // behind the length dt = dr = 0: the gradient passes, nothing is added
    auto stage = [&](int k, bool all) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + L * i;
        const float x = to_f32(rd[i]) + bias;
        float dt = p.softplus ? softplus(x) : x;
        if (k * kSsmTile + t >= len || !i_on) dt = 0.f;
        float dr = rg[i];
        if (p.z) {
          const float z = to_f32(rz[i]);
          dr *= z * sigmoid_fast(z);
        }
        sm.dt[t][ic] = make_float2(dt, all ? dt * to_f32(ru[i]) : 0.f);
        sm.dr[t][ic] = dr;
      }
#pragma unroll
      for (int j = 0; j < S::NBC; ++j) {
        const int e = tid + NT * j;
        if (e < kSsmTile * N) {
          if (all) (&sm.B[0][0])[e] = to_f32(rB[j]);
          (&sm.C[0][0])[e] = to_f32(rC[j]);
        }
      }
    };

    const size_t hrow = (size_t)b * p.D * N + par;
    State4 gr = {dup2(0.f), dup2(0.f)};  // gradient of the state after the tokens still to come

    if constexpr (SPLIT) {
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      float sum_dt = 0.f;
      if (rank > 0) {
        if (first < last) fetch(last - 1, false);
        for (int k = last - 1; k >= first; --k) {
          stage(k, false);
          __syncthreads();
          if (k > first) fetch(k - 1, false);
#pragma unroll
          for (int t = kSsmTile - 1; t >= 0; --t) {
            const float2 dt = dup2(sm.dt[t][my_ch].x), dr = dup2(sm.dr[t][my_ch]);
            const State4 Cv = load_state(&sm.C[t][n0]);
            gr.lo = __fmul2_rn(ex2_2(__fmul2_rn(dt, A.lo)), __ffma2_rn(Cv.lo, dr, gr.lo));
            gr.hi = __fmul2_rn(ex2_2(__fmul2_rn(dt, A.hi)), __ffma2_rn(Cv.hi, dr, gr.hi));
            sum_dt += dt.x;
          }
          __syncthreads();
        }
      }
      const float2 lo = ex2_2(__fmul2_rn(dup2(sum_dt), A.lo));
      const float2 hi = ex2_2(__fmul2_rn(dup2(sum_dt), A.hi));
      sm.start[tid] = make_float4(gr.lo.x, gr.lo.y, gr.hi.x, gr.hi.y);
      sm.decay[tid] = make_float4(lo.x, lo.y, hi.x, hi.y);
      gr = p.dh_T ? load_state(p.dh_T + hrow) : State4{dup2(0.f), dup2(0.f)};
      cluster.sync();
      for (int r = p.split - 1; r > rank; --r) {
        const float4 e = *cluster.map_shared_rank(&sm.start[tid], r);
        const float4 a = *cluster.map_shared_rank(&sm.decay[tid], r);
        gr.lo = __ffma2_rn(make_float2(a.x, a.y), gr.lo, make_float2(e.x, e.y));
        gr.hi = __ffma2_rn(make_float2(a.z, a.w), gr.hi, make_float2(e.z, e.w));
      }
      cluster.sync();  // nobody writes or leaves while its shared memory is read
    } else {
      if (p.dh_T) gr = load_state(p.dh_T + hrow);
    }

    State4 dA = {dup2(0.f), dup2(0.f)};
    float dskip = 0.f, dbias = 0.f;
    const float* chunks =
        p.h_chunks + (size_t)b * ((p.T + kSsmTile - 1) / kSsmTile) * p.D * N + par;
    State4 snap_next = {dup2(0.f), dup2(0.f)};
    if (first < last) {
      fetch(last - 1, true);
      snap_next = load_state(chunks + (size_t)(last - 1) * p.D * N);
    }
    for (int k = last - 1; k >= first; --k) {
      stage(k, true);
      float cu[IT], cx[IT], cz[IT], cg_[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        cu[i] = to_f32(ru[i]);
        cx[i] = to_f32(rd[i]) + bias;
        cz[i] = p.z ? to_f32(rz[i]) : 0.f;
        cg_[i] = rg[i];
      }
      const State4 snap = snap_next;
      __syncthreads();
      if (k > first) {
        fetch(k - 1, true);
        snap_next = load_state(chunks + (size_t)(k - 1) * p.D * N);
      }

      State4 a[kHalf], q[kHalf];
      // one token on the way forward
      auto ahead = [&](int t, State4& h, State4& at, State4& qt) {
        const float2 d = sm.dt[t][my_ch];
        const State4 Bv = load_state(&sm.B[t][n0]);
        const float2 dt = dup2(d.x), dtu = dup2(d.y);
        at.lo = ex2_2(__fmul2_rn(dt, A.lo));
        at.hi = ex2_2(__fmul2_rn(dt, A.hi));
        qt.lo = __fmul2_rn(at.lo, h.lo);
        qt.hi = __fmul2_rn(at.hi, h.hi);
        h.lo = __ffma2_rn(dtu, Bv.lo, qt.lo);
        h.hi = __ffma2_rn(dtu, Bv.hi, qt.hi);
      };
#pragma unroll 1
      for (int half = 1; half >= 0; --half) {
        State4 h = snap;
        if (half) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            State4 x, y;
            ahead(j, h, x, y);
          }
        }
        const int base = half * kHalf;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) ahead(base + j, h, a[j], q[j]);
        float v1[V], v2[V], v3[V];
#pragma unroll
        for (int j = kHalf - 1; j >= 0; --j) {
          const int t = base + j;
          const float2 d = sm.dt[t][my_ch];
          const float2 dt = dup2(d.x), dtu = dup2(d.y), dr = dup2(sm.dr[t][my_ch]);
          const State4 Bv = load_state(&sm.B[t][n0]), Cv = load_state(&sm.C[t][n0]);
          gr.lo = __ffma2_rn(Cv.lo, dr, gr.lo);
          gr.hi = __ffma2_rn(Cv.hi, dr, gr.hi);
          const float2 hlo = __ffma2_rn(dtu, Bv.lo, q[j].lo), hhi = __ffma2_rn(dtu, Bv.hi, q[j].hi);
          const float2 clo = __fmul2_rn(dr, hlo), chi = __fmul2_rn(dr, hhi);
          const float2 blo = __fmul2_rn(gr.lo, dtu), bhi = __fmul2_rn(gr.hi, dtu);
          const float2 x1 = __ffma2_rn(gr.lo, Bv.lo, __fmul2_rn(gr.hi, Bv.hi));
          const float2 x3 = __ffma2_rn(Cv.lo, hlo, __fmul2_rn(Cv.hi, hhi));
          const float2 qlo = __fmul2_rn(gr.lo, q[j].lo), qhi = __fmul2_rn(gr.hi, q[j].hi);
          const float2 x2 = __ffma2_rn(qlo, A.lo, __fmul2_rn(qhi, A.hi));
          dA.lo = __ffma2_rn(qlo, dt, dA.lo);
          dA.hi = __ffma2_rn(qhi, dt, dA.hi);
          gr.lo = __fmul2_rn(a[j].lo, gr.lo);
          gr.hi = __fmul2_rn(a[j].hi, gr.hi);
          v1[j % V] = x1.x + x1.y;
          v2[j % V] = x2.x + x2.y;
          v3[j % V] = x3.x + x3.y;
          // dBm, dCm of this token, over the warp's channels
          using Over = LaneSum<8, 16, L>;
          float w[8] = {blo.x, blo.y, bhi.x, bhi.y, clo.x, clo.y, chi.x, chi.y};
          Over::run(w, lane);
          if ((lane & Over::copies) == 0) {
            const int f = Over::first(lane);
            float* dst = &sm.part[warp][t][(f < 4 ? n0 : N + n0 - 4) + f];
#pragma unroll
            for (int m = 0; m < Over::left; ++m) dst[m] = w[m];
          }
          if (j % V == 0) {
            // s1, s2, s3 of V tokens, over a channel's lanes
            using Sum = LaneSum<V, L / 2, 1>;
            Sum::run(v1, lane);
            Sum::run(v2, lane);
            Sum::run(v3, lane);
            if ((lane & Sum::copies) == 0) {
              const int tt = t + Sum::first(lane);
              sm.s1[tt][my_ch] = v1[0];
              sm.s2[tt][my_ch] = v2[0];
              sm.s3[tt][my_ch] = v3[0];
            }
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int tt = it + L * i, t = k * kSsmTile + tt;
        if (!i_on || t >= p.T) continue;
        float du = 0.f, dd = 0.f, dz = 0.f;
        if (t < len) {
          const float dt = sm.dt[tt][ic].x, dr = sm.dr[tt][ic], s1 = sm.s1[tt][ic];
          du = fmaf(dt, s1, skip * dr);
          dd = fmaf(cu[i], s1, sm.s2[tt][ic] * (1.0f / kLog2e));  // A was scaled by log2 e
          if (p.softplus) dd *= sigmoid_fast(cx[i]);
          if (p.z) {
            const float sg = sigmoid_fast(cz[i]);
            dz = cg_[i] * fmaf(skip, cu[i], sm.s3[tt][ic]) * sg * fmaf(cz[i], 1.f - sg, 1.f);
          }
          dskip = fmaf(dr, cu[i], dskip);
          dbias += dd;
        }
        const size_t o = ob + (size_t)t * p.D;
        static_cast<InT*>(p.du)[o] = from_f32<InT>(du);
        static_cast<InT*>(p.ddelta)[o] = from_f32<InT>(dd);
        if (p.z) static_cast<InT*>(p.dz)[o] = from_f32<InT>(dz);
      }
#pragma unroll
      for (int o = tid; o < kSsmTile * 2 * N; o += NT) {
        const int tt = o / (2 * N), i = o % (2 * N), t = k * kSsmTile + tt;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) s += sm.part[w][tt][i];
        if (t < len)
          p.part_bc[((((size_t)tile_in_group * p.B + b) * p.T + t) * p.G + g) * (2 * N) + i] = s;
      }
    }

    // tokens behind the last tile
    if (rank == 0 && i_on) {
      for (int t = n_tiles * kSsmTile + it; t < p.T; t += L) {
        const size_t o = ob + (size_t)t * p.D;
        static_cast<InT*>(p.du)[o] = from_f32<InT>(0.f);
        static_cast<InT*>(p.ddelta)[o] = from_f32<InT>(0.f);
        if (p.z) static_cast<InT*>(p.dz)[o] = from_f32<InT>(0.f);
      }
    }
    if (rank == 0 && on && p.dh0) store_state(p.dh0 + hrow, gr);

    float* pp = p.part_par + ((size_t)b * p.split + rank) * ((size_t)p.D * (N + 2));
    if (on) {
      pp[par] = dA.lo.x; pp[par + 1] = dA.lo.y; pp[par + 2] = dA.hi.x; pp[par + 3] = dA.hi.y;
    }
    // dskip, d_delta_bias: over the L threads of a channel's items
    __syncthreads();
    float* red = &sm.part[0][0][0];
    red[tid] = dskip;
    red[NT + tid] = dbias;
    __syncthreads();
    if (tid < 2 * CH) {
      const int ch = tid % CH, which = tid / CH;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < L; ++j) s += red[which * NT + j * CH + ch];
      if (ch < nch) pp[(size_t)p.D * (N + which) + c0 + ch] = s;
    }
    __syncthreads();
  }
}

// dBm and dCm: the partial sums of a group's channel tiles, added in tile order;
// 0 behind a row's length. Four numbers a thread.
template <typename InT>
__global__ void __launch_bounds__(256) ssm_sum_bc_kernel(const float* part, int tiles, int B, int T,
                                                         int G, int N, const int* lengths, InT* dB,
                                                         InT* dC) {
  const size_t n = (size_t)B * T * G * 2 * N;
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const size_t row = i / (2 * N);
  const int e = (int)(i - row * (2 * N));
  const size_t token = row / G;
  const int b = (int)(token / T), t = (int)(token - (size_t)b * T);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (t < ssm_length(lengths, b, T)) {
    for (int k = 0; k < tiles; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(part + k * n + i);
      s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
    }
  }
  InT* o = e < N ? dB + row * N + e : dC + row * N + (e - N);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = from_f32<InT>(s[j]);
}

}  // namespace ttt
