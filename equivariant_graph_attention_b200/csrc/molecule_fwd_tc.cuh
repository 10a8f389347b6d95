// Attention within each molecule on tensor cores: the forward pass.
#pragma once

#include "molecule_tc.cuh"

namespace egat {
namespace {

// Short molecules, few rows and float32.  Bound by latency: three blocks of four warps
// an SM keep 45 % of the issue slots busy (512 molecules of 5 to 120 atoms: 137 us, of
// which the memory traffic is 27).  With one plane of the weights, at 124 us: four blocks an
// SM spill or take one head a warp, two hide less (142 to 162 us); blocks that take several
// head groups in turn are fewer and end less evenly (138 us).
//
// Per 16 x 16 pairs and head: S = Q K^T (one k-step of 16, two at dk 32), base-2
// scores in packed float32 pairs, the online softmax, and m += P H' with P as the
// sum of two bf16 numbers (bf16 storage; the normaliser adds the unrounded weights): with
// one, m was off by up to 1.4 times its own rounding (0.0023 of it in place of 0.0017), for
// 124 us in place of 137 at 512 molecules, 39 in place of 41 for one row against 32,768.  A row's
// reference moves only when a score passes it by 2^8, so most steps need no
// exchange between lanes and no rescaling; the rare step that moves it works its
// scores out again, which keeps them out of the registers in between.
template <int NT, int KC, int HP, int PL, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kTcThreads, NT <= 18 ? 3 : 2) mol_fwd_tc_kernel(MolParams p) {
  using L = TcLay<NT, KC, HP, PL>;
  using T = typename L::T;
  constexpr int WP = PL == 1 ? 2 : 3;   // planes of the weights
  extern __shared__ __align__(128) unsigned char tsm[];
  const int head0 = blockIdx.y * HP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const MolTile t = mol_tile(4 + p.rwlog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) return;
  const int rw = warp & ((1 << p.rwlog) - 1), kw = warp >> p.rwlog, kws = 4 >> p.rwlog;
  const int rA = rw * 16 + g, rB = rA + 8;
  const bool warp_live = rw * 16 < t.rows, lA = rA < t.rows, lB = rB < t.rows;
  const size_t rowA = size_t(t.row0) + rA, rowB = rowA + 8;

  // this split's share of the molecule's stages
  const int stages = (t.o1 - t.o0 + kTcStage - 1) / kTcStage, per = (stages + p.splits - 1) / p.splits;
  const int k_begin = t.o0 + int(blockIdx.z) * per * kTcStage;
  const int k_end = min(t.o1, k_begin + per * kTcStage);
  const uint32_t sbase = tc_smem(tsm);
  // its own query rows pass through the stage that the keys take last
  const uint32_t own = sbase + (L::BUFS - 1) * L::STAGE;
  {
    TcPart<HP * KC, PL> rows;
    const int c = lane % (HP * KC);
    const bool have = (c % KC) * 8 < p.dk;
    rows.init(static_cast<const T*>(p.a.q), p.H * p.dk, (head0 + c / KC) * p.dk + (have ? c % KC : 0) * 8, t.row0, L::QK, L::RK);
    rows.template load<L::RK>(L::BUFS == 2 ? own : own + L::STAGE, t.rows, have);
    tc_commit();
    if constexpr (L::BUFS == 1) {
      tc_wait<0>();
      rows.template split<L::RK>(own, own + L::STAGE, t.rows);
    }
  }
  TcLoader<NT, KC, HP, PL> ld;
  if (k_begin < k_end) {
    ld.init(p, p.a.k, p.a.hp, p.a.posk, head0, k_begin);
    ld.load(sbase, k_end - k_begin);
  }
  tc_commit();

  uint32_t qf[HP][PL][KC][2];
  tc_wait<1>();
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h)
    tc_frag_rows<KC, PL>(own + L::QK + rw * 16 * L::RK + h * KC * 16 + tc_lane_t(L::RK, 16), 16, L::PK, qf[h]);
  f32x2 px[2] = {}, py[2] = {}, pz[2] = {}, slope[HP] = {};   // minus the rows' positions
  if constexpr (BIAS) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (r ? lB : lA) {
        const float* x = p.a.posq + (r ? rowB : rowA) * 3;
        px[r] = f2_set(-x[0]);
        py[r] = f2_set(-x[1]);
        pz[r] = f2_set(-x[2]);
      }
#pragma unroll
    for (int h = 0; h < HP; ++h) slope[h] = f2_set(-p.a.slope[head0 + h] * kLog2e);
  }
  const f32x2 c_in = f2_set(CAP ? p.scale * p.inv_cap : p.scale * kLog2e), c_cap = f2_set(p.cap * kLog2e);

  float acc[HP][NT][4] = {};
  // minus the rows' references (NaN: none yet, which no score passes), and the
  // normaliser by lane
  f32x2 ref[HP][2], sum[HP][2] = {};
#pragma unroll
  for (int h = 0; h < HP; ++h) ref[h][0] = ref[h][1] = f2_set(__int_as_float(0x7fffffff));

  __syncthreads();   // the loop fills that stage
  int buf = 0;
  bool first = true;
  for (int k0 = k_begin; k0 < k_end; k0 += kTcStage, buf ^= L::BUFS - 1) {
    if constexpr (L::BUFS == 2) {
      if (k0 + kTcStage < k_end) ld.load(sbase + (buf ^ 1) * L::STAGE, k_end - k0 - kTcStage);
      tc_commit();
      tc_wait<1>();
    } else {
      tc_wait<0>();
      ld.split(sbase, k_end - k0);
      if (k0 + kTcStage < k_end) ld.load(sbase, k_end - k0 - kTcStage);
      tc_commit();
    }
    __syncthreads();
    const uint32_t st = sbase + buf * L::STAGE;
    const float* sp = reinterpret_cast<const float*>(tsm + buf * L::STAGE + L::POS);
    const int n = min(kTcStage, k_end - k0);
    if (warp_live)
#pragma unroll 1
      for (int j = kw * 16; j < n; j += kws * 16) {
        f32x2 d[2][2] = {}, unused[2][2];
        if constexpr (BIAS) tc_dists<false>(sp + j + t2, px, py, pz, d, unused);
        // base-2 scores of head h plus (n0, n1) by row: w[8-key tile][row]
        auto scores = [&](int h, f32x2 n0, f32x2 n1, f32x2 (&w)[4]) {
          float s[2][4] = {};
          tc_dot<KC, PL>(s, qf[h], st + L::QK + j * L::RK + h * KC * 16 + tc_lane_n(L::RK, 16), 0, 16, L::PK);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            w[2 * c] = f2_pack(s[c][0], s[c][1]);
            w[2 * c + 1] = f2_pack(s[c][2], s[c][3]);
          }
          if constexpr (CAP) {
            f32x2 none[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = f2_mul(w[i], c_in);
            tc_cap<4, false>(w, none);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = f2_fma(w[i], CAP ? c_cap : c_in, (i & 1) ? n1 : n0);
            if constexpr (BIAS) w[i] = f2_fma(d[i >> 1][i & 1], slope[h], w[i]);
          }
        };
        f32x2 w[HP][4];
        // once with the references and, where one has to move (the first step's always
        // do), once without: one copy of the code
        bool move = first;
#pragma unroll 1
        for (;;) {
          bool pass = false;
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            scores(h, move ? 0ull : ref[h][0], move ? 0ull : ref[h][1], w[h]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float v[4];
              f2_unpack(w[h][r], v[0], v[1]);
              f2_unpack(w[h][2 + r], v[2], v[3]);
              // all NaN without a reference
              pass |= !(fmaxf(tc_max3(v[0], v[1], v[2]), v[3]) <= 8.f);
            }
            if (j + 16 > n)   // keys past the molecule
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float a, b;
                f2_unpack(w[h][i], a, b);
                if (j + 8 * (i >> 1) + t2 >= n) a = -INFINITY;
                if (j + 8 * (i >> 1) + t2 + 1 >= n) b = -INFINITY;
                w[h][i] = f2_pack(a, b);
              }
          }
          if (move) break;
          move = __any_sync(~0u, pass);
          if (!move) break;
        }
        if (move) {
#pragma unroll
          for (int h = 0; h < HP; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float v[4], old, unused1;
              f2_unpack(w[h][r], v[0], v[1]);
              f2_unpack(w[h][2 + r], v[2], v[3]);
              f2_unpack(ref[h][r], old, unused1);
              const float top = quad_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
              const float up = fmaxf(-old, top);   // a NaN reference drops out
              // all -inf so far: no reference, no weights
              const bool none = up == -INFINITY;
              const float f = none || isnan(old) ? 0.f : fast_exp2(-old - up);
              ref[h][r] = f2_set(none ? __int_as_float(0x7fffffff) : -up);
              sum[h][r] = f2_mul(sum[h][r], f2_set(f));
              if (!first)
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                  acc[h][x][2 * r] *= f;
                  acc[h][x][2 * r + 1] *= f;
                }
              const f32x2 shift = f2_set(none ? 0.f : -up);
              w[h][r] = f2_add(w[h][r], shift);
              w[h][2 + r] = f2_add(w[h][2 + r], shift);
            }
        }
        first = false;
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          uint32_t pf[WP][2][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(w[h][i], a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[h][i & 1] = f2_add(sum[h][i & 1], f2_pack(a, b));
            tc_put<WP>(pf, i >> 1, i & 1, a, b);
          }
          tc_apply<NT, WP>(acc[h], pf, st + L::VAL + j * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16,
                           L::PV);
        }
      }
    __syncthreads();
  }

  tc_wait<0>();
  if (kws == 1) {
    // rows of its own: normalised in registers, through shared memory for whole chunks
    T* rows = reinterpret_cast<T*>(tsm) + warp * 16 * L::OUTROW;   // this warp's [16][OUTROW]
#pragma unroll
    for (int h = 0; h < HP; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float lo, hi, mr;
        f2_unpack(sum[h][r], lo, hi);
        const float l = quad_sum(lo + hi), inv = l == 0.f ? 0.f : 1.f / l;
        f2_unpack(ref[h][r], mr, hi);
        const size_t row = r ? rowB : rowA;
        if (t2 == 0 && p.lse && (r ? lB : lA)) p.lse[row * p.H + head0 + h] = l == 0.f ? -INFINITY : -mr * kLn2 + logf(l);
#pragma unroll
        for (int x = 0; x < NT; ++x)
          tc_store2(rows + (g + 8 * r) * L::OUTROW + (x * HP + h) * 8 + t2, acc[h][x][2 * r] * inv, acc[h][x][2 * r + 1] * inv);
      }
    __syncwarp();
    tc_write_vals<NT, HP, L::OUTROW>(p, rows, p.m, head0, size_t(t.row0) + rw * 16, min(16, t.rows - rw * 16));
    return;
  }
  // join the warps that shared rows, and write whole 16-byte chunks
  float* oacc = reinterpret_cast<float*>(tsm);                  // [4 warps][16][OUTROW]
  float* oml = oacc + 4 * 16 * L::OUTROW;                        // [4 warps][16][HP][2]
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = warp * 16 + g + 8 * r;
      float lo, hi, mr;
      f2_unpack(sum[h][r], lo, hi);
      const float l = quad_sum(lo + hi);
      f2_unpack(ref[h][r], mr, hi);
      if (t2 == 0) {
        oml[(row * HP + h) * 2] = isnan(mr) ? -INFINITY : -mr;
        oml[(row * HP + h) * 2 + 1] = l;
      }
#pragma unroll
      for (int x = 0; x < NT; ++x)
        *reinterpret_cast<float2*>(oacc + row * L::OUTROW + (x * HP + h) * 8 + t2) =
            make_float2(acc[h][x][2 * r], acc[h][x][2 * r + 1]);
    }
  __syncthreads();
  const int rws = 1 << p.rwlog;
  const size_t total = size_t(p.nq) * p.H;
  for (int i = threadIdx.x; i < t.rows * HP * NT; i += kTcThreads) {
    const int row = i / (HP * NT), c = i % (HP * NT), x = c / HP, h = c % HP;
    float top = -INFINITY, l = 0.f, f[4], o[8] = {};
    for (int w = 0; w < kws; ++w) top = fmaxf(top, oml[(((w * rws) * 16 + row) * HP + h) * 2]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kws; ++w) {
      const float* ml = oml + (((w * rws) * 16 + row) * HP + h) * 2;
      f[w & 3] = fast_exp2(ml[0] - ref);
      l = fmaf(f[w & 3], ml[1], l);
      const float* a = oacc + ((w * rws) * 16 + row) * L::OUTROW + c * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(f[w & 3], a[e], o[e]);
    }
    const size_t at = size_t(t.row0) + row, rh = at * p.H + head0 + h;
    if (p.splits > 1) {
      const size_t z = blockIdx.z * total + rh;
      if (x == 0) {
        p.part_ml[2 * z] = top;
        p.part_ml[2 * z + 1] = l;
      }
      float4* to = reinterpret_cast<float4*>(p.part_o + z * p.dv + x * 8);
      to[0] = make_float4(o[0], o[1], o[2], o[3]);
      to[1] = make_float4(o[4], o[5], o[6], o[7]);
      continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (x == 0 && p.lse) p.lse[rh] = l == 0.f ? -INFINITY : top * kLn2 + logf(l);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    tc_store8(static_cast<T*>(p.m) + at * (p.D * p.C) + tc_val_off(p, head0 + h, x), o);
  }
}

template <int PL>
int tc_forward(const MolParams& p, cudaStream_t st) {
  return tc_dispatch<PL, 2>(p.dv / 8, p.dk, [&](auto nt, auto kc, auto hp) {
    constexpr int NT = decltype(nt)::value, KC = decltype(kc)::value, HP = decltype(hp)::value;
    using L = TcLay<NT, KC, HP, PL>;
    const size_t shm = std::max(L::BYTES, 4 * 16 * (L::OUTROW + 2 * HP) * 4);
    const dim3 grid(p.slots, p.H / HP, p.splits);
    return mol_flags(p.cap > 0.f, p.a.slope != nullptr, [&](auto cap, auto bias) {
      return tc_launch(mol_fwd_tc_kernel<NT, KC, HP, PL, decltype(cap)::value, decltype(bias)::value>, grid, shm, p, st);
    });
  });
}

}  // namespace
}  // namespace egat
