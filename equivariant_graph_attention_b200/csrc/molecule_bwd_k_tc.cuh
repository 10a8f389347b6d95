// Attention within each molecule on tensor cores: the key side of the backward
// pass.
#pragma once

#include "molecule_tc.cuh"

namespace egat {
namespace {

// Bound by latency at two blocks an SM: the accumulators and the key rows' fragments
// fill the registers (4,096 atoms capped: 0.73 ms, 39 % of the tensor pipe, a third of
// the issue slots).
//
// dL/dk, dL/dh' and, with POS, the key side of dL/dr: a warp owns 16 key rows
// and meets the molecule's query rows.  The products are transposed (S^T = K Q^T,
// dP^T = H' G^T), so that the weights and dS land as the A operands of
// dh' = a^T G and dk = dS^T Q.  A query row past the molecule has lse2 = +inf: no weight.
template <int NT, int KC, int HP, int PL, bool CAP, bool BIAS, bool POS>
__global__ void __launch_bounds__(kTcThreads, 2) mol_bwd_k_tc_kernel(MolParams p) {
  using L = TcLay<NT, KC, HP, PL>;
  using T = typename L::T;
  // planes of dS: its terms cancel in the sum, and two planes of bf16 storage take the
  // rounding of one out of it (1.6 times the error of the result's own rounding)
  constexpr int DP = PL == 1 ? 2 : 3;
  // planes of the weights: as many, or dh' would hold each one's rounding beside its own
  // (4,096 atoms capped: 0.63 ms with one)
  constexpr int WP = DP;
  // the key rows' values as A fragments: in registers, or read again for every
  // step where they would not fit beside the accumulators
  constexpr bool VREG = NT * PL <= 27;
  extern __shared__ __align__(128) unsigned char tsm[];
  const int head0 = blockIdx.y * HP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const MolTile t = mol_tile(4 + p.rwlog, p.a.kptr, p.a.qptr, p.nmol, p.nk, p.nq, blockIdx.x);
  if (t.rows <= 0) return;
  const int rw = warp & ((1 << p.rwlog) - 1), kw = warp >> p.rwlog, kws = 4 >> p.rwlog;
  const int rA = rw * 16 + g, rB = rA + 8;
  const bool warp_live = rw * 16 < t.rows, lA = rA < t.rows, lB = rB < t.rows;
  const size_t rowA = size_t(t.row0) + rA, rowB = rowA + 8;
  const uint32_t sbase = tc_smem(tsm);
  TcLoader<NT, KC, HP, PL> ld;
  // a stage, with minus lse2 and delta of the query rows; no weight past the molecule
  auto load = [&](int r0, int b) {
    const uint32_t st = sbase + b * L::STAGE;
    ld.load(st, t.o1 - r0);
    for (int i = threadIdx.x; i < kTcStage * HP; i += kTcThreads) {
      const int r = i / HP, h = i % HP, o = (PL == 1 ? L::ROW : L::RAWP + kTcStage * 12) + (h * 2 * kTcStage + r) * 4;
      const size_t at = size_t(r0 + r) * p.H + head0 + h;
      if (r0 + r < t.o1) {
        tc_cp4(st + o, p.nlse2 + at, true);
        tc_cp4(st + o + kTcStage * 4, p.delta + at, true);
      } else {
        *reinterpret_cast<float*>(tsm + b * L::STAGE + o) = -INFINITY;
        *reinterpret_cast<float*>(tsm + b * L::STAGE + o + kTcStage * 4) = 0.f;
      }
    }
  };
  auto split = [&](int left) {
    ld.split(sbase, left);
    for (int r = threadIdx.x; r < kTcStage; r += kTcThreads)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        tc_move4(sbase + L::ROW + (e * kTcStage + r) * 4, sbase + L::RAWP + kTcStage * 12 + (e * kTcStage + r) * 4);
  };
  // its own rows of k and h' pass through the stage that the queries take last
  const uint32_t own = sbase + (L::BUFS - 1) * L::STAGE, own_rows = rw * 16;
  {
    TcLoader<NT, KC, HP, PL> rows;
    rows.init(p, p.a.k, p.a.hp, nullptr, head0, t.row0);
    rows.pos = nullptr;
    rows.load(own, t.rows);
    tc_commit();
    if constexpr (L::BUFS == 1) {
      tc_wait<0>();
      rows.split(own, t.rows);
    }
  }
  if (t.o0 < t.o1) {
    ld.init(p, p.a.q, p.g.g, p.a.posq, head0, t.o0);
    load(t.o0, 0);
  }
  tc_commit();

  uint32_t kf[HP][PL][KC][2], vf[HP][PL][VREG ? NT : 1][2];
  f32x2 slope[HP] = {}, px[2] = {}, py[2] = {}, pz[2] = {};
  tc_wait<1>();
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    tc_frag_rows<KC, PL>(own + L::QK + own_rows * L::RK + h * KC * 16 + tc_lane_t(L::RK, 16), 16, L::PK, kf[h]);
    if constexpr (VREG)
      tc_frag_rows<NT, PL>(own + L::VAL + own_rows * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16, L::PV, vf[h]);
    if constexpr (BIAS) slope[h] = f2_set(-p.a.slope[head0 + h] * kLog2e);
  }
  if constexpr (BIAS)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (r ? lB : lA) {
        const float* x = p.a.posk + (r ? rowB : rowA) * 3;
        px[r] = f2_set(-x[0]);
        py[r] = f2_set(-x[1]);
        pz[r] = f2_set(-x[2]);
      }
  const f32x2 c_in = f2_set(CAP ? p.scale * p.inv_cap : p.scale * kLog2e), c_cap = f2_set(p.cap * kLog2e);

  float dk[HP][KC][4] = {}, dv[HP][NT][4] = {};
  f32x2 gs[2][3] = {};
  __syncthreads();   // the loop fills that stage
  int buf = 0;
  for (int q0 = t.o0; q0 < t.o1; q0 += kTcStage, buf ^= L::BUFS - 1) {
    if constexpr (L::BUFS == 2) {
      if (q0 + kTcStage < t.o1) load(q0 + kTcStage, buf ^ 1);
      tc_commit();
      tc_wait<1>();
    } else {
      tc_wait<0>();
      split(t.o1 - q0);
      if (q0 + kTcStage < t.o1) load(q0 + kTcStage, 0);
      tc_commit();
    }
    __syncthreads();
    const uint32_t st = sbase + buf * L::STAGE;
    const float* sp = reinterpret_cast<const float*>(tsm + buf * L::STAGE + L::POS);
    const float* sl = reinterpret_cast<const float*>(tsm + buf * L::STAGE + L::ROW);
    const int n = min(kTcStage, t.o1 - q0);
    if (warp_live)
#pragma unroll 1
      for (int j = kw * 16; j < n; j += kws * 16) {
        f32x2 d[2][2] = {}, ri[2][2] = {};
        if constexpr (BIAS) tc_dists<POS>(sp + j + t2, px, py, pz, d, ri);
        f32x2 u[2][2] = {};   // POS: sum over the heads of slope dS
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          float s[2][4] = {}, dp[2][4] = {};
          tc_dot<KC, PL>(s, kf[h], st + L::QK + j * L::RK + h * KC * 16 + tc_lane_n(L::RK, 16), 0, 16, L::PK);
          const uint32_t gb = st + L::VAL + j * L::RV + h * 16;
          if constexpr (VREG) {
            tc_dot<NT, PL>(dp, vf[h], gb + tc_lane_n(L::RV, HP * 16), gb + tc_lane_n2(L::RV), HP * 16, L::PV);
          } else {
#pragma unroll 4
            for (int c = 0; c < NT; c += 2) {
              uint32_t a[PL][2][2];
              tc_frag_val<2, PL>(p, p.a.hp, rowA, rowB, lA, lB, head0 + h, a, c);
              tc_dot<2, PL, true>(dp, a, gb + c * HP * 16 + tc_lane_n(L::RV, HP * 16), 0, HP * 16, L::PV);
            }
          }
          f32x2 x[4], fx[CAP ? 4 : 1];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            x[2 * c] = f2_pack(s[c][0], s[c][1]);
            x[2 * c + 1] = f2_pack(s[c][2], s[c][3]);
          }
          if constexpr (CAP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], c_in);
            tc_cap<4, true>(x, fx);
          }
          uint32_t fd[DP][2][2], fa[WP][2][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = i >> 1, r = i & 1;
            const f32x2* row = reinterpret_cast<const f32x2*>(sl + h * 2 * kTcStage + j + 8 * c + t2);
            x[i] = f2_fma(x[i], CAP ? c_cap : c_in, row[0]);
            if constexpr (BIAS) x[i] = f2_fma(d[c][r], slope[h], x[i]);
            float a, b;
            f2_unpack(x[i], a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            tc_put<WP>(fa, c, r, a, b);
            f32x2 ds = f2_mul(f2_pack(a, b), f2_add(f2_pack(dp[c][2 * r], dp[c][2 * r + 1]), row[kTcStage / 2]));
            if (POS) u[c][r] = f2_fma(ds, slope[h], u[c][r]);
            if constexpr (CAP) ds = f2_mul(ds, fx[i]);
            f2_unpack(ds, a, b);
            tc_put<DP>(fd, c, r, a, b);
          }
          tc_apply<NT, WP>(dv[h], fa, st + L::VAL + j * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16, L::PV);
          tc_apply<KC, DP>(dk[h], fd, st + L::QK + j * L::RK + h * KC * 16 + tc_lane_t(L::RK, 16), 16, L::PK);
        }
        if (POS) {
          const bool far = tc_far(d);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
              tc_pull(far, reinterpret_cast<const f32x2*>(sp + j + 8 * c + t2), px[r], py[r], pz[r],
                      f2_mul(u[c][r], ri[c][r]), gs[r]);
          }
        }
      }
    __syncthreads();
  }

  tc_wait<0>();
  __syncthreads();
  float gs2[2][3];
  if (POS)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        float lo, hi;
        f2_unpack(gs[r][e], lo, hi);
        gs2[r][e] = quad_sum(lo + hi);
      }
  if (kws > 1)
    tc_join<HP * (NT + KC) * 4 + (POS ? 6 : 0)>(reinterpret_cast<float*>(tsm), rw, 1 << p.rwlog, kw, kws, [&](auto&& f) {
#pragma unroll
      for (int h = 0; h < HP; ++h) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) f(dv[h][x][e]);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) f(dk[h][c][e]);
      }
      if constexpr (POS)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 3; ++e) f(gs2[r][e]);
    });
  if (kw != 0 || !warp_live) return;
  constexpr int OUT = HP * KC * 8 + 8;
  T* rows = reinterpret_cast<T*>(tsm) + rw * 16 * (L::OUTROW + OUT);   // [16][OUTROW] values, [16][OUT] keys
  T* krows = rows + 16 * L::OUTROW;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int h = 0; h < HP; ++h) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
        tc_store2(rows + (g + 8 * r) * L::OUTROW + (x * HP + h) * 8 + t2, dv[h][x][2 * r], dv[h][x][2 * r + 1]);
#pragma unroll
      for (int c = 0; c < KC; ++c)
        tc_store2(krows + (g + 8 * r) * OUT + (h * KC + c) * 8 + t2, p.scale * dk[h][c][2 * r], p.scale * dk[h][c][2 * r + 1]);
    }
    if (POS && t2 == 0 && (r ? lB : lA)) {
      float* at = p.part_dk + (size_t(blockIdx.y) * p.nk + (r ? rowB : rowA)) * 3;
#pragma unroll
      for (int e = 0; e < 3; ++e) at[e] = -kLn2 * gs2[r][e];
    }
  }
  __syncwarp();
  const int live = min(16, t.rows - rw * 16);
  tc_write_vals<NT, HP, L::OUTROW>(p, rows, p.g.dhp, head0, size_t(t.row0) + rw * 16, live);
  tc_write_qk<KC, HP, OUT>(p, krows, p.g.dk, head0, size_t(t.row0) + rw * 16, live);
}

template <int PL>
int tc_backward_k(const MolParams& p, cudaStream_t st) {
  return tc_dispatch<PL, 2>(p.dv / 8, p.dk, [&](auto nt, auto kc, auto hp) {
    constexpr int NT = decltype(nt)::value, KC = decltype(kc)::value, HP = decltype(hp)::value;
    using L = TcLay<NT, KC, HP, PL>;
    const int shm = std::max({L::BYTES, tc_join_bytes(HP * (NT + KC) * 4 + 6),
                              int(64 * (L::OUTROW + HP * KC * 8 + 8) * sizeof(typename L::T))});
    const dim3 grid(mol_slots(p.nk, p.nmol, 16 << p.rwlog), p.H / HP);
    // positions come with a bias
    if (p.want_pos)
      return mol_flags(p.cap > 0.f, true, [&](auto cap, auto) {
        return tc_launch(mol_bwd_k_tc_kernel<NT, KC, HP, PL, decltype(cap)::value, true, true>, grid, shm, p, st);
      });
    return mol_flags(p.cap > 0.f, p.a.slope != nullptr, [&](auto cap, auto bias) {
      return tc_launch(mol_bwd_k_tc_kernel<NT, KC, HP, PL, decltype(cap)::value, decltype(bias)::value, false>, grid, shm,
                       p, st);
    });
  });
}

}  // namespace
}  // namespace egat
