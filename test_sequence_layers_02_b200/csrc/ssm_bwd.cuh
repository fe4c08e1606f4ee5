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
// The states come from the forward's snapshots, 16 tokens apart. A tile is walked in four
// quarters of 4 tokens, the last first: a run over its first 12 tokens leaves the states before
// the quarters, and each quarter's decays and q stay in registers between its way forward
// and its way back. That is 1.75 exponentials a token; with halves of 8 tokens it would be 1.5,
// but the registers of a half leave an SM one CTA in place of two.
//
// Work: about 25 packed fp32 operations and 1.75 exponentials for 4 states of a (token,
// channel), and two sums over the channels for each (token, state): at N = 16, 32 values a lane
// (four tokens) over a warp's 32 channels in five scatter steps, 31 shuffles where adding
// value by value would be 160 (and where four times the steps for one token each took a fifth
// longer: the steps wait for one another). The issue of all that binds, not HBM and not the special-function units.
// The sums over channel tiles go through partial sums in global memory, added in tile
// order. No atomics: the same bits on every call.
//
// Measured, bf16, N = 16, with the reductions: 8 x 4096 tokens by 768 channels 0.90 ms (fp32 0.91), 16 x 2048 by 1536
// 1.34 ms, 4 x 2048 by 256 0.09 ms; about half an instruction a clock and scheduler. At 128 registers the SPLIT
// builds spill up to 80 bytes a thread and single elements at N = 8 up to 368; N = 64, at 168, up to 628.
#pragma once

#include "ssm.cuh"

namespace ttt {

// Roles as in the forward, with one set of four warps around the recurrence: between two
// barriers the recurrence takes tile k (from the last down), the others finish tile k + 1
// and stage tile k - 1. A tile's sums (s1 .. s3, dBm, dCm) have one buffer: the others
// read it at once, and the recurrence waits for that at a second barrier, behind its
// run over the first 12 tokens.
template <int N, int P, typename InT, typename OutT, int VEC>
struct SsmBwdShape {
  static constexpr int L = N / P;               // warps that share a channel
  static constexpr int CW = L < 4 ? 4 / L : 1;  // blocks of 32 channels
  static constexpr int CH = 32 * CW;
  static constexpr int RT = CH * L;             // threads of the recurrence
  static constexpr int HT = 128;                // threads around it
  static constexpr int NT = RT + HT;
  static constexpr int QUADS = CH / VEC;
  static constexpr int TS = HT / QUADS;         // tokens between a thread's items
  static constexpr int IT = kSsmTile / TS;      // items per thread and tile
  static constexpr int BCQ = kSsmTile * N / VEC;
  static constexpr int NBC = (BCQ + HT - 1) / HT;
  // Slots of raw inputs: from the copy to the end of the tile's epilogue, two tiles after
  // its use in staging.
  static constexpr int RING = VEC > 1 && sizeof(InT) == 2 ? 6 : 5;
  static constexpr int AHEAD = RING - 3;        // tiles on their way
  static constexpr int SUMS = CW * kSsmTile * 2 * N;
  struct Single {                               // a tile's single elements on their way
    Pack<InT, VEC> u[IT], d[IT], z[IT], B[NBC], C[NBC];
    Pack<OutT, VEC> g[IT];
  };
  struct Smem {
    alignas(16) float2 dt[2][kSsmTile][CH];     // dt, dt u
    alignas(16) float dr[2][kSsmTile][CH];
    alignas(16) float B[2][kSsmTile][N];
    alignas(16) float C[2][kSsmTile][N];
    alignas(16) float s[3][kSsmTile][L][CH];    // s1, s2, s3: a part for each of a channel's warps
    alignas(16) float bc[CW][kSsmTile][2 * N];  // dBm, dCm of 32 channels
    struct Slot {
      Pack<InT, VEC> u[IT][HT], d[IT][HT], z[IT][HT], B[NBC][HT], C[NBC][HT];
      Pack<OutT, VEC> g[IT][HT];
    } ring[RING];
  };
};

template <int N, int P, typename InT, typename OutT, int VEC, bool SPLIT>
__global__ void __launch_bounds__(SsmBwdShape<N, P, InT, OutT, VEC>::NT, N <= 16 ? 2 : 1)
    ssm_bwd_kernel(const SsmParams p) {
  using S = SsmBwdShape<N, P, InT, OutT, VEC>;
  constexpr int L = S::L, CW = S::CW, CH = S::CH, IT = S::IT, TS = S::TS, RT = S::RT, HT = S::HT;
  constexpr int NBC = S::NBC, QUADS = S::QUADS, RING = S::RING, AHEAD = S::AHEAD;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(smem_raw);
  __shared__ float2 s_start[SPLIT ? P / 2 : 1][SPLIT ? RT : 1], s_decay[SPLIT ? P / 2 : 1][SPLIT ? RT : 1];
  __shared__ float s_sum[SPLIT ? RT : 1];

  const bool recur = threadIdx.x < RT;
  const int tid = recur ? threadIdx.x : threadIdx.x - RT;  // within the role
  const int lane = threadIdx.x & 31;
  const int rank = SPLIT ? blockIdx.x % p.split : 0;
  const int tile = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int cta_tiles = (p.per_group + CH - 1) / CH;
  const int g = tile / cta_tiles;
  const int tile_in_group = tile - g * cta_tiles;
  const int in_group = tile_in_group * CH;
  const int c0 = g * p.per_group + in_group;
  const int nch = min(CH, p.per_group - in_group);

  // the recurrence: states n0 .. n0 + P - 1 of channel my_ch
  const int part = (tid >> 5) % L;
  const int block = (tid >> 5) / L;
  const int my_ch = (block * 32 + lane) % CH;
  const int n0 = part * P;
  const bool on = recur && my_ch < nch;
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
    const InT *up = nullptr, *dp = nullptr, *zp = nullptr, *Bp = nullptr, *Cp = nullptr;
    const OutT* gp = nullptr;
    const bool bc_on = S::BCQ % HT == 0 || tid < S::BCQ;
    constexpr int BROW = N / VEC, BS = HT / BROW;
    const int bt = tid / BROW, bn = tid % BROW * VEC;
    // Pointers to a thread's items and packs of tile k, which move down a tile at a time.
    auto seek = [&](int k) {
      const long long t0 = (long long)k * kSsmTile + it, e0 = (long long)k * kSsmTile + bt;
      up = static_cast<const InT*>(p.u) + b * p.u_b + t0 * p.u_t + icc;
      dp = static_cast<const InT*>(p.delta) + b * p.d_b + t0 * p.d_t + icc;
      zp = static_cast<const InT*>(p.z) + b * p.z_b + t0 * p.z_t + icc;
      gp = static_cast<const OutT*>(p.dy) + b * p.y_b + t0 * p.y_t + icc;
      Bp = static_cast<const InT*>(p.Bm) + b * p.Bm_b + g * p.Bm_g + e0 * p.Bm_t + bn;
      Cp = static_cast<const InT*>(p.Cm) + b * p.Cm_b + g * p.Cm_g + e0 * p.Cm_t + bn;
    };
    auto slot = [&](int k) -> typename S::Smem::Slot& { return sm.ring[k % RING]; };
    // The inputs of tile k on their way to its slot (0 behind the length). Packs are copied
    // asynchronously, one group of copies a tile, also an empty one below the first; single
    // elements wait in registers until the next call stores them, a tile later.
    typename S::Single hold;
    int held = -1;
    auto send = [&](int k) {
      if constexpr (VEC == 1) {
        if (held >= 0) {
          typename S::Smem::Slot& r = slot(held);
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            r.u[i][tid] = hold.u[i];
            r.d[i][tid] = hold.d[i];
            r.z[i][tid] = hold.z[i];
            r.g[i][tid] = hold.g[i];
          }
          if (bc_on) {
#pragma unroll
            for (int j = 0; j < NBC; ++j) {
              r.B[j][tid] = hold.B[j];
              r.C[j][tid] = hold.C[j];
            }
          }
        }
        held = k >= first ? k : -1;
      }
      if (k >= first) {
        typename S::Smem::Slot& r = slot(k);
        const int left = len - k * kSsmTile;
        auto move = [&](auto& dst, auto& reg, const auto* src, bool have) {
          using T = std::remove_reference_t<decltype(dst)>;
          if constexpr (VEC > 1) {
            copy_async<sizeof(T)>(&dst, src, have);
          } else {
            reg = {};
            if (have) reg = *reinterpret_cast<const T*>(src);
          }
        };
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const bool have = it + TS * i < left;
          move(r.u[i][tid], hold.u[i], have ? up + TS * i * p.u_t : up, have);
          move(r.d[i][tid], hold.d[i], have ? dp + TS * i * p.d_t : dp, have);
          if (p.z) move(r.z[i][tid], hold.z[i], have ? zp + TS * i * p.z_t : zp, have);
          move(r.g[i][tid], hold.g[i], have ? gp + TS * i * p.y_t : gp, have);
        }
        if (bc_on) {
#pragma unroll
          for (int j = 0; j < NBC; ++j) {
            const bool have = bt + BS * j < left;
            move(r.B[j][tid], hold.B[j], have ? Bp + BS * j * p.Bm_t : Bp, have);
            move(r.C[j][tid], hold.C[j], have ? Cp + BS * j * p.Cm_t : Cp, have);
          }
        }
        up -= kSsmTile * p.u_t;
        dp -= kSsmTile * p.d_t;
        zp -= kSsmTile * p.z_t;
        gp -= kSsmTile * p.y_t;
        Bp -= kSsmTile * p.Bm_t;
        Cp -= kSsmTile * p.Cm_t;
      }
      if constexpr (VEC > 1) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Tile k from its slot to the recurrence's half of shared memory. Behind the length, and
    // in channels that are not there, dt = dr = 0: the gradient passes, nothing is added.
    auto stage = [&](int k) {
      if constexpr (VEC > 1) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
      const typename S::Smem::Slot& f = slot(k);
      const int h = k & 1, left = i_on ? len - k * kSsmTile : 0;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + TS * i;
        float dt[VEC], u[VEC], dr[VEC];
        f.d[i][tid].widen(dt);
        f.u[i][tid].widen(u);
        f.g[i][tid].widen(dr);
#pragma unroll
        for (int q = 0; q < VEC; ++q) dt[q] += bias[q];
        if (p.softplus) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) dt[q] = softplus(dt[q]);
        }
        if (p.z) {
          float z[VEC];
          f.z[i][tid].widen(z);
#pragma unroll
          for (int q = 0; q < VEC; ++q) dr[q] *= z[q] * sigmoid_fast(z[q]);
        }
        if (t >= left) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) dt[q] = dr[q] = 0.f;
        }
        if constexpr (VEC == 1) {
          sm.dt[h][t][ic] = make_float2(dt[0], dt[0] * u[0]);
        } else {
          float4* o = reinterpret_cast<float4*>(&sm.dt[h][t][ic]);
#pragma unroll
          for (int q = 0; q < VEC; q += 2)
            o[q / 2] = make_float4(dt[q], dt[q] * u[q], dt[q + 1], dt[q + 1] * u[q + 1]);
        }
        store_vec<float, VEC>(&sm.dr[h][t][ic], dr);
      }
      if (bc_on) {
#pragma unroll
        for (int j = 0; j < NBC; ++j) {
          float v[VEC];
          f.B[j][tid].widen(v);
          store_vec<float, VEC>(&sm.B[h][bt + BS * j][bn], v);
          f.C[j][tid].widen(v);
          store_vec<float, VEC>(&sm.C[h][bt + BS * j][bn], v);
        }
      }
    };

    float dskip[VEC], dbias[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) dskip[q] = dbias[q] = 0.f;
    const size_t ob = (size_t)b * p.T * p.D + icc;  // du, ddelta, dz
    // Tile k behind the recurrence: first the sums out of their buffers (then `free`), then the
    // gradients of u, delta and z and the partial sums of dBm and dCm.
    auto finish = [&](int k, auto free) {
      const int h = k & 1;
      const typename S::Smem::Slot& f = slot(k);
      float s1[IT][VEC], s2[IT][VEC], s3[IT][VEC];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int t = it + TS * i;
        load_vec<float, VEC>(&sm.s[0][t][0][ic], s1[i]);
        load_vec<float, VEC>(&sm.s[1][t][0][ic], s2[i]);
        load_vec<float, VEC>(&sm.s[2][t][0][ic], s3[i]);
#pragma unroll
        for (int j = 1; j < L; ++j) {
          float v[3][VEC];
          load_vec<float, VEC>(&sm.s[0][t][j][ic], v[0]);
          load_vec<float, VEC>(&sm.s[1][t][j][ic], v[1]);
          load_vec<float, VEC>(&sm.s[2][t][j][ic], v[2]);
#pragma unroll
          for (int q = 0; q < VEC; ++q) {
            s1[i][q] += v[0][q];
            s2[i][q] += v[1][q];
            s3[i][q] += v[2][q];
          }
        }
      }
      const int left_all = len - k * kSsmTile;
#pragma unroll
      for (int e = tid * 4; e < S::SUMS; e += HT * 4) {
        const int cw = e / (kSsmTile * 2 * N), t = e / (2 * N) % kSsmTile, n = e % (2 * N);
        if (t < left_all && cw * 32 < nch) {
          const size_t row =
              (((size_t)(tile_in_group * CW + cw) * p.B + b) * p.T + (size_t)k * kSsmTile + t) * p.G + g;
          *reinterpret_cast<float4*>(p.part_bc + row * (2 * N) + n) =
              *reinterpret_cast<const float4*>(&sm.bc[0][0][0] + e);
        }
      }
      free();
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int tt = it + TS * i, t = k * kSsmTile + tt;
        if (!i_on || t >= p.T) continue;
        float du[VEC], dd[VEC], dz[VEC], u[VEC], x[VEC], dr[VEC];
        f.u[i][tid].widen(u);
        f.d[i][tid].widen(x);
        load_vec<float, VEC>(&sm.dr[h][tt][ic], dr);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          du[q] = fmaf(sm.dt[h][tt][ic + q].x, s1[i][q], skip[q] * dr[q]);
          dd[q] = fmaf(u[q], s1[i][q], s2[i][q] * (1.0f / kLog2e));  // A was scaled by log2 e
          if (p.softplus) dd[q] *= sigmoid_fast(x[q] + bias[q]);
        }
        if (p.z) {
          float z[VEC], dy[VEC];
          f.z[i][tid].widen(z);
          f.g[i][tid].widen(dy);
#pragma unroll
          for (int q = 0; q < VEC; ++q) {
            const float sg = sigmoid_fast(z[q]);
            dz[q] = dy[q] * fmaf(skip[q], u[q], s3[i][q]) * sg * fmaf(z[q], 1.f - sg, 1.f);
          }
        }
        if (t >= len) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) du[q] = dd[q] = dz[q] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          dskip[q] = fmaf(dr[q], u[q], dskip[q]);
          dbias[q] += dd[q];
        }
        const size_t o = ob + (size_t)t * p.D;
        store_vec<InT, VEC>(static_cast<InT*>(p.du) + o, du);
        store_vec<InT, VEC>(static_cast<InT*>(p.ddelta) + o, dd);
        if (p.z) store_vec<InT, VEC>(static_cast<InT*>(p.dz) + o, dz);
      }
    };

    // ---- the recurrence ----
    const size_t hrow = (size_t)b * p.D * N + par;
    States<P> gr;  // gradient of the state after the tokens still to come
    gr.zero();
    // one token on the way forward
    auto ahead = [&](int half, int t, States<P>& h, States<P>& at, States<P>& qt) {
      const float2 d = sm.dt[half][t][my_ch];
      States<P> Bv;
      Bv.load(&sm.B[half][t][n0]);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        at.v[i] = decay2(dup2(d.x), A.v[i]);
        qt.v[i] = __fmul2_rn(at.v[i], h.v[i]);
        h.v[i] = __ffma2_rn(dup2(d.y), Bv.v[i], qt.v[i]);
      }
    };

    if constexpr (SPLIT) {
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      float sum_dt = 0.f;
      if (rank > 0 && first < last) {
        if (!recur) {
          seek(last - 1);
          for (int j = 0; j < AHEAD; ++j) send(last - 1 - j);
          stage(last - 1);
          send(last - 1 - AHEAD);
        }
        for (int k = last - 1; k >= first; --k) {
          __syncthreads();
          if (recur) {
#pragma unroll
            for (int t = kSsmTile - 1; t >= 0; --t) {
              const float2 dt = dup2(sm.dt[k & 1][t][my_ch].x), dr = dup2(sm.dr[k & 1][t][my_ch]);
              States<P> Cv;
              Cv.load(&sm.C[k & 1][t][n0]);
#pragma unroll
              for (int i = 0; i < P / 2; ++i)
                gr.v[i] = __fmul2_rn(decay2(dt, A.v[i]), __ffma2_rn(Cv.v[i], dr, gr.v[i]));
              sum_dt += dt.x;
            }
          } else if (k > first) {
            stage(k - 1);
            send(k - 1 - AHEAD);
          }
        }
        if constexpr (VEC > 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      if (recur) {
        s_sum[tid] = sum_dt;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          s_start[i][tid] = gr.v[i];
          s_decay[i][tid] = decay2(dup2(sum_dt), A.v[i]);
        }
        gr.zero();
        if (p.dh_T) gr.load(p.dh_T + hrow);
      }
      cluster.sync();
      if (recur) {
        for (int r = p.split - 1; r > rank; --r) {
#pragma unroll
          for (int i = 0; i < P / 2; ++i)
            gr.v[i] = __ffma2_rn(*cluster.map_shared_rank(&s_decay[i][tid], r), gr.v[i],
                                 *cluster.map_shared_rank(&s_start[i][tid], r));
        }
        if (!gr.finite()) {  // once more, with care
          gr.zero();
          if (p.dh_T) gr.load(p.dh_T + hrow);
          for (int r = p.split - 1; r > rank; --r)
            gr.carry([&](int i) { return *cluster.map_shared_rank(&s_decay[i][tid], r); },
                     [&](int i) { return *cluster.map_shared_rank(&s_start[i][tid], r); },
                     *cluster.map_shared_rank(&s_sum[tid], r), A);
        }
      }
      cluster.sync();  // nobody writes or leaves while its shared memory is read
    } else {
      if (recur && p.dh_T) gr.load(p.dh_T + hrow);
    }

    // The second barrier of a tile: its sums of the tile before have been read.
    auto sums_read = [] { asm volatile("bar.arrive 1, %0;" ::"n"(S::NT) : "memory"); };
    if (recur) {
      States<P> dA;
      dA.zero();
      const float* chunks =
          p.h_chunks + (size_t)b * ((p.T + kSsmTile - 1) / kSsmTile) * p.D * N + par;
      States<P> next;
      next.zero();
      if (first < last) next.load(chunks + (size_t)(last - 1) * p.D * N);
      for (int k = last - 1; k >= first; --k) {
        const int half = k & 1;
        __syncthreads();
        States<P> before[4];  // the state before each quarter
        before[0] = next;
        if (k > first) next.load(chunks + (size_t)(k - 1) * p.D * N);
        {
          States<P> h = before[0], x, y;
#pragma unroll
          for (int t = 0; t < 12; ++t) {
            ahead(half, t, h, x, y);
            if (t % 4 == 3) before[t / 4 + 1] = h;
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(S::NT) : "memory");
#pragma unroll 1
        for (int quarter = 3; quarter >= 0; --quarter) {
          States<P> a[4], q[4], h = before[3];
          before[3] = before[2];
          before[2] = before[1];
          before[1] = before[0];
#pragma unroll
          for (int j = 0; j < 4; ++j) ahead(half, quarter * 4 + j, h, a[j], q[j]);
          constexpr int SET = P == 4 ? 4 : 2;  // tokens whose sums are taken at once
          float w[SET * 2 * P];
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            float* wj = w + j % SET * 2 * P;
            const int t = quarter * 4 + j;
            const float2 d = sm.dt[half][t][my_ch];
            const float2 dt = dup2(d.x), dtu = dup2(d.y), dr = dup2(sm.dr[half][t][my_ch]);
            States<P> Bv, Cv;
            Bv.load(&sm.B[half][t][n0]);
            Cv.load(&sm.C[half][t][n0]);
            float2 x1, x2, x3;
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
              gr.v[i] = __ffma2_rn(Cv.v[i], dr, gr.v[i]);
              const float2 hh = __ffma2_rn(dtu, Bv.v[i], q[j].v[i]);
              const float2 cc = __fmul2_rn(dr, hh), bb = __fmul2_rn(gr.v[i], dtu);
              wj[2 * i] = bb.x;
              wj[2 * i + 1] = bb.y;
              wj[P + 2 * i] = cc.x;
              wj[P + 2 * i + 1] = cc.y;
              const float2 gq = __fmul2_rn(gr.v[i], q[j].v[i]);
              x1 = i ? __ffma2_rn(gr.v[i], Bv.v[i], x1) : __fmul2_rn(gr.v[i], Bv.v[i]);
              x2 = i ? __ffma2_rn(gq, A.v[i], x2) : __fmul2_rn(gq, A.v[i]);
              x3 = i ? __ffma2_rn(Cv.v[i], hh, x3) : __fmul2_rn(Cv.v[i], hh);
              dA.v[i] = __ffma2_rn(gq, dt, dA.v[i]);
              gr.v[i] = __fmul2_rn(a[j].v[i], gr.v[i]);
            }
            sm.s[0][t][part][my_ch] = x1.x + x1.y;
            sm.s[1][t][part][my_ch] = x2.x + x2.y;
            sm.s[2][t][part][my_ch] = x3.x + x3.y;
            if (j % SET) continue;
            // dBm, dCm of this token and the next, over the warp's channels
            using Over = LaneSum<SET * 2 * P, 16, 1>;
            Over::run(w, lane);
            if ((lane & Over::copies) == 0) {
              const int f = Over::first(lane) % (2 * P);
              float* dst = &sm.bc[block][t + Over::first(lane) / (2 * P)][f < P ? n0 + f : N + n0 + f - P];
#pragma unroll
              for (int m = 0; m < Over::left; ++m) dst[m] = w[m];
            }
          }
        }
      }
      if (first < last) {
        __syncthreads();
        asm volatile("bar.sync 1, %0;" ::"n"(S::NT) : "memory");
      }
      if (rank == 0 && on && p.dh0) gr.store(p.dh0 + hrow);
      if (on) {
        float* pp = p.part_par + ((size_t)b * p.split + rank) * ((size_t)p.D * (N + 2)) + par;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          pp[2 * i] = dA.v[i].x;
          pp[2 * i + 1] = dA.v[i].y;
        }
      }
    } else if (first < last) {
      seek(last - 1);
      for (int j = 0; j < AHEAD; ++j) send(last - 1 - j);
      stage(last - 1);
      send(last - 1 - AHEAD);
      for (int k = last - 1; k >= first; --k) {
        __syncthreads();
        if (k + 1 < last)
          finish(k + 1, sums_read);
        else
          sums_read();
        if (k > first) {
          stage(k - 1);
          send(k - 1 - AHEAD);
        }
      }
      __syncthreads();
      finish(first, sums_read);
      if constexpr (VEC > 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    }

    if (!recur) {
      // tokens behind the last tile
      if (rank == 0 && i_on) {
        const float none[VEC] = {};
        for (int t = n_tiles * kSsmTile + it; t < p.T; t += TS) {
          const size_t o = ob + (size_t)t * p.D;
          store_vec<InT, VEC>(static_cast<InT*>(p.du) + o, none);
          store_vec<InT, VEC>(static_cast<InT*>(p.ddelta) + o, none);
          if (p.z) store_vec<InT, VEC>(static_cast<InT*>(p.dz) + o, none);
        }
      }
    }
    // dskip, d_delta_bias: over the TS threads of a channel's items
    __syncthreads();
    float* red = &sm.s[0][0][0][0];  // [2][TS][CH]
    if (!recur) {
      store_vec<float, VEC>(red + it * CH + ic, dskip);
      store_vec<float, VEC>(red + (TS + it) * CH + ic, dbias);
    }
    __syncthreads();
    if (!recur) {
      for (int e = tid; e < 2 * CH; e += HT) {
        const int ch = e % CH, which = e / CH;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < TS; ++j) s += red[(which * TS + j) * CH + ch];
        if (ch < nch)
          p.part_par[((size_t)b * p.split + rank) * ((size_t)p.D * (N + 2)) +
                     (size_t)p.D * (N + which) + c0 + ch] = s;
      }
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
