// Attention within each molecule on tensor cores: the query side of the backward
// pass.
#pragma once

#include "molecule_tc.cuh"

namespace egat {
namespace {

// sums of a thread that the warps of a row join
constexpr int q_sums(int kc, int hp, bool fix, bool pos) {
  return hp * (kc * 4 * (fix ? 2 : 1) + 2 * ((fix ? 1 : 0) + (pos ? (fix ? 5 : 1) : 0))) + (pos ? 6 : 0);
}

// dL/dq, the row sums delta_i = sum_j a_ij dP_ij and, with POS, the query side
// of dL/dr and dL/dslope, in one sweep over the keys.  The sweep takes
// dS' = a (dP - delta') with delta' = G . m from the stored, rounded m, and sums
// delta itself in float32 beside it.  Every output is linear in delta:
//   dq = sum dS' f' k + (delta' - delta) sum a f' k,
// so the second sum, of weights alone, takes the rounding of m out at the end;
// the correction is small, so nothing cancels.  A float32 m needs none of that.
template <int NT, int KC, int HP, int PL, bool CAP, bool BIAS, bool POS>
__global__ void __launch_bounds__(kTcThreads, PL == 1 && NT * HP <= 9 ? (POS ? 3 : 4) : 2) mol_bwd_q_tc_kernel(MolParams p) {
  using L = TcLay<NT, KC, HP, PL>;
  using T = typename L::T;
  // planes of dS: its terms cancel in the sum, and two planes of bf16 storage take the
  // rounding of one out of it (1.6 times the error of the result's own rounding)
  constexpr int DP = PL == 1 ? 2 : 3;
  constexpr bool FIX = PL == 1;   // m is rounded
  constexpr int SUMS = q_sums(KC, HP, FIX, POS), OUT = HP * KC * 8 + 8;
  extern __shared__ __align__(128) unsigned char tsm[];
  const int head0 = blockIdx.y * HP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const MolTile t = mol_tile(4 + p.rwlog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) {
    if (POS && threadIdx.x < HP) p.part_ds[size_t(head0 + threadIdx.x) * p.slots + blockIdx.x] = 0.f;
    return;
  }
  const int rw = warp & ((1 << p.rwlog) - 1), kw = warp >> p.rwlog, kws = 4 >> p.rwlog;
  const int rA = rw * 16 + g, rB = rA + 8;
  const bool warp_live = rw * 16 < t.rows, lA = rA < t.rows, lB = rB < t.rows;
  const size_t rowA = size_t(t.row0) + rA, rowB = rowA + 8;
  const uint32_t sbase = tc_smem(tsm);
  // its own rows of q and G, then of m, pass through the stage that the keys take last
  const uint32_t own = sbase + (L::BUFS - 1) * L::STAGE, own_rows = rw * 16;
  {
    TcLoader<NT, KC, HP, PL> rows;
    rows.init(p, p.a.q, p.g.g, nullptr, head0, t.row0);
    rows.pos = nullptr;
    rows.load(own, t.rows);
    tc_commit();
    if constexpr (L::BUFS == 1) {
      tc_wait<0>();
      rows.split(own, t.rows);
    }
  }
  TcLoader<NT, KC, HP, PL> ld;
  if (t.o0 < t.o1) {
    ld.init(p, p.a.k, p.a.hp, p.a.posk, head0, t.o0);
    if (L::BUFS == 2) ld.load(sbase, t.o1 - t.o0);
  }
  tc_commit();

  uint32_t qf[HP][PL][KC][2], gf[HP][PL][NT][2];
  float lse2[HP][2], dlt[HP][2];   // rows that are not there: lse2 = +inf, no weight
  f32x2 slope[HP] = {}, px[2] = {}, py[2] = {}, pz[2] = {};
  tc_wait<1>();
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    tc_frag_rows<KC, PL>(own + L::QK + own_rows * L::RK + h * KC * 16 + tc_lane_t(L::RK, 16), 16, L::PK, qf[h]);
    tc_frag_rows<NT, PL>(own + L::VAL + own_rows * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16, L::PV, gf[h]);
  }
  __syncthreads();
  {
    TcPart<HP * NT, PL> rows;
    const int c = lane % (HP * NT);
    rows.init(static_cast<const T*>(p.g.m), p.D * p.C, tc_val_off(p, head0 + c % HP, c / HP), t.row0, L::VAL, L::RV);
    rows.template load<L::RV>(L::BUFS == 2 ? own : own + L::RAWV, t.rows, true);
    tc_commit();
    tc_wait<0>();
    if constexpr (L::BUFS == 1) rows.template split<L::RV>(own, own + L::RAWV, t.rows);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    float d0 = 0.f, d1 = 0.f;
    uint32_t mf[PL][NT][2];
    tc_frag_rows<NT, PL>(own + L::VAL + own_rows * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16, L::PV, mf);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t mw[PL], gw[PL];
#pragma unroll
        for (int k = 0; k < PL; ++k) mw[k] = mf[k][c][r], gw[k] = gf[h][k][c][r];
        const float2 m = tc_value<PL>(mw), x = tc_value<PL>(gw);
        (r ? d1 : d0) += fmaf(m.x, x.x, m.y * x.y);
      }
    dlt[h][0] = quad_sum(d0);
    dlt[h][1] = quad_sum(d1);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = r ? lB : lA;
      const float x = ok ? p.g.lse[(r ? rowB : rowA) * p.H + head0 + h] * kLog2e : INFINITY;
      lse2[h][r] = x == -INFINITY ? INFINITY : x;
    }
    if constexpr (BIAS) slope[h] = f2_set(-p.a.slope[head0 + h] * kLog2e);
  }
  if constexpr (BIAS)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (r ? lB : lA) {
        const float* x = p.a.posq + (r ? rowB : rowA) * 3;
        px[r] = f2_set(-x[0]);
        py[r] = f2_set(-x[1]);
        pz[r] = f2_set(-x[2]);
      }
  const f32x2 c_in = f2_set(CAP ? p.scale * p.inv_cap : p.scale * kLog2e), c_cap = f2_set(p.cap * kLog2e);
  f32x2 nlse[HP][2], ndel[HP][2];   // minus lse2 and delta'
#pragma unroll
  for (int h = 0; h < HP; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      nlse[h][r] = f2_set(-lse2[h][r]);
      ndel[h][r] = f2_set(-dlt[h][r]);
    }

  float dq[HP][KC][4] = {}, bk[FIX ? HP : 1][KC][4] = {};
  f32x2 del[HP][2] = {};
  // POS: sums over j of (slope dS', slope a) (r_j - r_i) / d and of (dS', a) d
  f32x2 gs[2][3] = {}, ga[HP][2][3] = {};
  f32x2 sd[HP][2] = {}, sa[HP][2] = {};

  if (L::BUFS == 1 && t.o0 < t.o1) ld.load(sbase, t.o1 - t.o0);
  tc_commit();
  __syncthreads();   // the loop fills that stage
  int buf = 0;
  for (int k0 = t.o0; k0 < t.o1; k0 += kTcStage, buf ^= L::BUFS - 1) {
    if constexpr (L::BUFS == 2) {
      if (k0 + kTcStage < t.o1) ld.load(sbase + (buf ^ 1) * L::STAGE, t.o1 - k0 - kTcStage);
      tc_commit();
      tc_wait<1>();
    } else {
      tc_wait<0>();
      ld.split(sbase, t.o1 - k0);
      if (k0 + kTcStage < t.o1) ld.load(sbase, t.o1 - k0 - kTcStage);
      tc_commit();
    }
    __syncthreads();
    const uint32_t st = sbase + buf * L::STAGE;
    const float* sp = reinterpret_cast<const float*>(tsm + buf * L::STAGE + L::POS);
    const int n = min(kTcStage, t.o1 - k0);
    if (warp_live)
#pragma unroll 1
      for (int j = kw * 16; j < n; j += kws * 16) {
        f32x2 d[2][2] = {}, ri[2][2] = {};   // distances (and their reciprocals): [8-key tile][row]
        if constexpr (BIAS) tc_dists<POS>(sp + j + t2, px, py, pz, d, ri);
        f32x2 u[2][2] = {}, dc[2][2] = {};   // POS: sum over the heads of slope dS; finite distances
        bool far = false;
        if constexpr (POS) {
          far = tc_far(d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;   // a distance may be inf where the weight is zero
            f2_unpack(d[i >> 1][i & 1], a, b);
            dc[i >> 1][i & 1] = f2_pack(fminf(a, 3e38f), fminf(b, 3e38f));
          }
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          float s[2][4], dp[2][4];
          tc_dot<KC, PL>(s, qf[h], st + L::QK + j * L::RK + h * KC * 16 + tc_lane_n(L::RK, 16), 0, 16, L::PK);
          const uint32_t vb = st + L::VAL + j * L::RV + h * 16;
          tc_dot<NT, PL>(dp, gf[h], vb + tc_lane_n(L::RV, HP * 16), vb + tc_lane_n2(L::RV), HP * 16, L::PV);
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
          uint32_t fd[DP][2][2], fa[PL][2][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = i >> 1, r = i & 1;
            x[i] = f2_fma(x[i], CAP ? c_cap : c_in, nlse[h][r]);
            if constexpr (BIAS) x[i] = f2_fma(d[c][r], slope[h], x[i]);
            float a, b;
            f2_unpack(x[i], a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            if (j + 16 > n) {   // keys past the molecule
              if (j + 8 * c + t2 >= n) a = 0.f;
              if (j + 8 * c + t2 + 1 >= n) b = 0.f;
            }
            f32x2 w = f2_pack(a, b);
            const f32x2 dP = f2_pack(dp[c][2 * r], dp[c][2 * r + 1]);
            if (FIX) del[h][r] = f2_fma(w, dP, del[h][r]);
            f32x2 ds = f2_mul(w, f2_add(dP, ndel[h][r]));
            float lo, hi;
            if (POS) {
              u[c][r] = f2_fma(ds, slope[h], u[c][r]);
              sd[h][r] = f2_fma(ds, dc[c][r], sd[h][r]);
              if (FIX) {
                tc_pull(far, reinterpret_cast<const f32x2*>(sp + j + 8 * c + t2), px[r], py[r], pz[r], f2_mul(w, ri[c][r]),
                        ga[h][r]);
                sa[h][r] = f2_fma(w, dc[c][r], sa[h][r]);
              }
            }
            if constexpr (CAP) {
              ds = f2_mul(ds, fx[i]);
              w = f2_mul(w, fx[i]);
              f2_unpack(w, a, b);
            }
            f2_unpack(ds, lo, hi);
            tc_put<DP>(fd, c, r, lo, hi);
            if (FIX) tc_put<PL>(fa, c, r, a, b);
          }
          const uint32_t kb = st + L::QK + j * L::RK + h * KC * 16 + tc_lane_t(L::RK, 16);
          tc_apply<KC, DP>(dq[h], fd, kb, 16, L::PK);
          if constexpr (FIX) tc_apply<KC, PL>(bk[h], fa, kb, 16, L::PK);
        }
        if constexpr (POS) {
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
  // sums of a row: its four lanes', then those of the warps that shared it
  float del2[HP][2], sd2[HP][2], sa2[HP][2], ga2[HP][2][3], gs2[2][3];
  auto both = [](f32x2 v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return quad_sum(lo + hi);
  };
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      if (FIX) del2[h][r] = both(del[h][r]);
      if (POS) {
        sd2[h][r] = both(sd[h][r]);
        if (FIX) {
          sa2[h][r] = both(sa[h][r]);
#pragma unroll
          for (int e = 0; e < 3; ++e) ga2[h][r][e] = both(ga[h][r][e]);
        }
      }
    }
    if (POS)
#pragma unroll
      for (int e = 0; e < 3; ++e) gs2[r][e] = both(gs[r][e]);
  }
  const int rws = 1 << p.rwlog;
  if (kws > 1)
    tc_join<SUMS>(reinterpret_cast<float*>(tsm), rw, rws, kw, kws, [&](auto&& f) {
#pragma unroll
      for (int h = 0; h < HP; ++h) {
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f(dq[h][c][e]);
            if constexpr (FIX) f(bk[h][c][e]);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (FIX) f(del2[h][r]);
          if constexpr (POS) {
            f(sd2[h][r]);
            if constexpr (FIX) {
              f(sa2[h][r]);
#pragma unroll
              for (int e = 0; e < 3; ++e) f(ga2[h][r][e]);
            }
          }
        }
      }
      if constexpr (POS)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 3; ++e) f(gs2[r][e]);
    });
  __shared__ float warp_ds[4][HP];
  if (kw == 0 && warp_live) {
    T* rows = reinterpret_cast<T*>(tsm) + rw * 16 * OUT;
    float ds_sum[HP] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = r ? lB : lA;
      const size_t row = r ? rowB : rowA;
      float pos[3];
      if (POS)
#pragma unroll
        for (int e = 0; e < 3; ++e) pos[e] = -kLn2 * gs2[r][e];   // slope was -slope log2 e there
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        const float eps = FIX ? dlt[h][r] - del2[h][r] : 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          float x = dq[h][c][2 * r], y = dq[h][c][2 * r + 1];
          if constexpr (FIX) {
            x = fmaf(eps, bk[h][c][2 * r], x);
            y = fmaf(eps, bk[h][c][2 * r + 1], y);
          }
          tc_store2(rows + (g + 8 * r) * OUT + (h * KC + c) * 8 + t2, p.scale * x, p.scale * y);
        }
        if (t2 == 0 && ok) {
          p.delta[row * p.H + head0 + h] = eps - dlt[h][r];
          p.nlse2[row * p.H + head0 + h] = lse2[h][r] == INFINITY ? -INFINITY : -lse2[h][r];
        }
        if (POS) {
          // directions point from i to j: dL/dr_i = sum slope dS (r_j - r_i) / d
          if (FIX)
#pragma unroll
            for (int e = 0; e < 3; ++e) pos[e] = fmaf(p.a.slope[head0 + h] * eps, ga2[h][r][e], pos[e]);
          if (t2 == 0 && ok) ds_sum[h] -= FIX ? fmaf(eps, sa2[h][r], sd2[h][r]) : sd2[h][r];
        }
      }
      if (POS && t2 == 0 && ok) {
        float* at = p.part_dq + (size_t(blockIdx.y) * p.nq + row) * 3;
        at[0] = pos[0], at[1] = pos[1], at[2] = pos[2];
      }
    }
    __syncwarp();
    tc_write_qk<KC, HP, OUT>(p, rows, p.g.dq, head0, size_t(t.row0) + rw * 16, min(16, t.rows - rw * 16));
    if (POS) {
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        float x = ds_sum[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        if (lane == 0) warp_ds[rw][h] = x;
      }
    }
  }
  if constexpr (POS) {
    __syncthreads();
    if (threadIdx.x < HP) {
      float x = 0.f;
      for (int w = 0; w < rws && w * 16 < t.rows; ++w) x += warp_ds[w][threadIdx.x];
      p.part_ds[size_t(head0 + threadIdx.x) * p.slots + blockIdx.x] = x;
    }
  }
}

// One head a warp at 72 columns: three or four blocks an SM instead of two (4,096
// atoms capped: 0.61 -> 0.52 ms; the key side and the forward pass lose by it).  Two heads
// of up to 32 columns fall under the same bound, unmeasured, and spill (340 bytes a thread,
// 980 with position gradients).  Bound
// by instruction issue and latency: half of the issue slots are busy, a quarter of
// the tensor pipe.
template <int PL>
int tc_backward_q(const MolParams& p, cudaStream_t st) {
  return tc_dispatch<PL, 1>(p.dv / 8, p.dk, [&](auto nt, auto kc, auto hp) {
    constexpr int NT = decltype(nt)::value, KC = decltype(kc)::value, HP = decltype(hp)::value;
    using L = TcLay<NT, KC, HP, PL>;
    const int shm = std::max({L::BYTES, tc_join_bytes(q_sums(KC, HP, PL == 1, true)),
                              int(64 * (HP * KC * 8 + 8) * sizeof(typename L::T))});
    const dim3 grid(p.slots, p.H / HP);
    // positions come with a bias
    if (p.want_pos)
      return mol_flags(p.cap > 0.f, true, [&](auto cap, auto) {
        return tc_launch(mol_bwd_q_tc_kernel<NT, KC, HP, PL, decltype(cap)::value, true, true>, grid, shm, p, st);
      });
    return mol_flags(p.cap > 0.f, p.a.slope != nullptr, [&](auto cap, auto bias) {
      return tc_launch(mol_bwd_q_tc_kernel<NT, KC, HP, PL, decltype(cap)::value, decltype(bias)::value, false>, grid, shm,
                       p, st);
    });
  });
}

}  // namespace
}  // namespace egat
