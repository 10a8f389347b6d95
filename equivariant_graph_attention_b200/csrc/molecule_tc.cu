// Attention within each molecule on tensor cores (bf16 storage): the forward
// pass, and the rules of the tensor-core path.
#include "molecule_tc.cuh"

namespace egat {
namespace {

// Per 16 x 16 pairs and head: S = Q K^T (one k-step of 16, two at dk 32), base-2
// scores in packed float32 pairs, the online softmax, and m += P H' with P
// rounded once to bf16 (the normaliser adds the unrounded weights).  The running
// maximum is a reference: it moves only when a score passes it by 2^8, so most
// steps need no exchange between lanes and no rescaling.
template <int NT, int KC, int HP>
__global__ void __launch_bounds__(kTcThreads) mol_fwd_tc_kernel(MolParams p) {
  using L = TcLay<NT, KC, HP>;
  extern __shared__ __align__(128) unsigned char tsm[];
  const int head0 = blockIdx.y * HP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const MolTile t = mol_tile(4 + p.rwlog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) return;
  const int rw = warp & ((1 << p.rwlog) - 1), kw = warp >> p.rwlog, kws = 4 >> p.rwlog;
  const int rA = rw * 16 + g, rB = rA + 8;
  const bool warp_live = rw * 16 < t.rows, lA = rA < t.rows, lB = rB < t.rows;
  const size_t rowA = size_t(t.row0) + rA, rowB = rowA + 8;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q);
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.a.k);
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.a.hp);

  // this split's share of the molecule's stages
  const int stages = (t.o1 - t.o0 + kTcStage - 1) / kTcStage, per = (stages + p.splits - 1) / p.splits;
  const int k_begin = t.o0 + int(blockIdx.z) * per * kTcStage;
  const int k_end = min(t.o1, k_begin + per * kTcStage);
  const uint32_t sbase = tc_smem(tsm);
  if (k_begin < k_end) tc_load_stage<NT, KC, HP>(p, k, v, p.a.posk, head0, k_begin, k_end, sbase);
  tc_commit();

  uint32_t qf[HP][KC][2];
#pragma unroll
  for (int h = 0; h < HP; ++h) tc_frag_qk<KC>(p, q, rowA, rowB, lA, lB, head0 + h, qf[h]);
  f32x2 px[2] = {}, py[2] = {}, pz[2] = {}, slope[HP] = {};   // minus the rows' positions
  if (p.a.slope) {
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
  const bool capped = p.cap > 0.f;
  const f32x2 c_in = f2_set(capped ? p.scale * p.inv_cap : p.scale * kLog2e), c_cap = f2_set(p.cap * kLog2e);

  float acc[HP][NT][4] = {};
  float mx[HP][2], sum[HP][2];
#pragma unroll
  for (int h = 0; h < HP; ++h) mx[h][0] = mx[h][1] = -INFINITY, sum[h][0] = sum[h][1] = 0.f;

  int buf = 0;
  for (int k0 = k_begin; k0 < k_end; k0 += kTcStage, buf ^= 1) {
    if (k0 + kTcStage < k_end)
      tc_load_stage<NT, KC, HP>(p, k, v, p.a.posk, head0, k0 + kTcStage, k_end, sbase + (buf ^ 1) * L::STAGE);
    tc_commit();
    tc_wait<1>();
    __syncthreads();
    const uint32_t st = sbase + buf * L::STAGE;
    const float* sp = reinterpret_cast<const float*>(tsm + buf * L::STAGE + L::POS);
    const int n = min(kTcStage, k_end - k0);
    if (warp_live)
#pragma unroll 1
      for (int j = kw * 16; j < n; j += kws * 16) {
        f32x2 d[2][2] = {};   // distances: [8-key tile][row]
        if (p.a.slope) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const f32x2* at = reinterpret_cast<const f32x2*>(sp + j + 8 * c + t2);
            const f32x2 x = at[0], y = at[kTcStage / 2], z = at[kTcStage];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const f32x2 dx = f2_add(x, px[r]), dy = f2_add(y, py[r]), dz = f2_add(z, pz[r]);
              float a, b;
              f2_unpack(f2_fma(dx, dx, f2_fma(dy, dy, f2_mul(dz, dz))), a, b);
              d[c][r] = f2_pack(mol_sqrt(a), mol_sqrt(b));
            }
          }
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          float s[2][4] = {};
          tc_dot<KC>(s, qf[h], st + L::QK + j * L::RK + h * KC * 16 + tc_lane_n(L::RK, 16), 0, 16);
          f32x2 x[2][2];   // scores in base 2, before the reference is taken off
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            x[c][0] = f2_pack(s[c][0], s[c][1]);
            x[c][1] = f2_pack(s[c][2], s[c][3]);
          }
          if (capped) {
            f32x2 unused;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              x[c][0] = f2_mul(x[c][0], c_in);
              x[c][1] = f2_mul(x[c][1], c_in);
              tc_cap<false>(x[c][0], x[c][1], unused, unused);
            }
          }
          float w[2][4];
          auto score = [&](float m0, float m1) {
            const f32x2 cm = capped ? c_cap : c_in;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              f32x2 a = f2_fma(x[c][0], cm, f2_set(-m0)), b = f2_fma(x[c][1], cm, f2_set(-m1));
              if (p.a.slope) {
                a = f2_fma(d[c][0], slope[h], a);
                b = f2_fma(d[c][1], slope[h], b);
              }
              f2_unpack(a, w[c][0], w[c][1]);
              f2_unpack(b, w[c][2], w[c][3]);
              if (j + 16 > n) {   // keys past the molecule
                if (j + 8 * c + t2 >= n) w[c][0] = w[c][2] = -INFINITY;
                if (j + 8 * c + t2 + 1 >= n) w[c][1] = w[c][3] = -INFINITY;
              }
            }
          };
          score(mx[h][0], mx[h][1]);
          const float top0 = fmaxf(fmaxf(w[0][0], w[0][1]), fmaxf(w[1][0], w[1][1]));
          const float top1 = fmaxf(fmaxf(w[0][2], w[0][3]), fmaxf(w[1][2], w[1][3]));
          // a row without a finite reference yet takes this way too: its w may be NaN from inf - inf
          if (__any_sync(~0u, !(top0 <= 8.f) || !(top1 <= 8.f) || fminf(mx[h][0], mx[h][1]) == -INFINITY)) {
            score(0.f, 0.f);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float up = fmaxf(mx[h][r], quad_max(fmaxf(fmaxf(w[0][2 * r], w[0][2 * r + 1]),
                                                              fmaxf(w[1][2 * r], w[1][2 * r + 1]))));
              const float f = up == -INFINITY ? 1.f : fast_exp2(mx[h][r] - up);
              const float ref = up == -INFINITY ? 0.f : up;
              mx[h][r] = up;
              sum[h][r] *= f;
#pragma unroll
              for (int x8 = 0; x8 < NT; ++x8) {
                acc[h][x8][2 * r] *= f;
                acc[h][x8][2 * r + 1] *= f;
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                w[c][2 * r] -= ref;
                w[c][2 * r + 1] -= ref;
              }
            }
          }
          uint32_t pf[2][2];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float a = fast_exp2(w[c][2 * r]), b = fast_exp2(w[c][2 * r + 1]);
              sum[h][r] += a + b;
              pf[c][r] = tc_pack(a, b);
            }
          tc_apply<NT>(acc[h], pf, st + L::VAL + j * L::RV + h * 16 + tc_lane_t(L::RV, HP * 16), HP * 16);
        }
      }
    __syncthreads();
  }

  // join the warps that shared rows, and write whole 16-byte chunks
  float* oacc = reinterpret_cast<float*>(tsm);                  // [4 warps][16][OUTROW]
  float* oml = oacc + 4 * 16 * L::OUTROW;                        // [4 warps][16][HP][2]
  tc_wait<0>();
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HP; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = warp * 16 + g + 8 * r;
      const float l = quad_sum(sum[h][r]);
      if (t2 == 0) {
        oml[(row * HP + h) * 2] = mx[h][r];
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
    uint4 u;
    u.x = tc_pack(o[0] * inv, o[1] * inv);
    u.y = tc_pack(o[2] * inv, o[3] * inv);
    u.z = tc_pack(o[4] * inv, o[5] * inv);
    u.w = tc_pack(o[6] * inv, o[7] * inv);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.m) + at * (p.D * p.C) + tc_val_off(p, head0 + h, x)) = u;
  }
}

int value_tiles(const egat_mol_shape& s) { return (s.lmax + 1) * (s.lmax + 1) * (s.C / s.H) / 8; }

}  // namespace

int mol_tc_heads(const egat_mol_shape& s) { return value_tiles(s) <= 9 ? 2 : 1; }

// bf16 rows with up to 256 value columns a head (the accumulators of 16 rows fill
// half of a warp's registers there), and two heads where two are taken together.
bool mol_tc_supported(const egat_mol_shape& s) {
  const int nt = value_tiles(s);
  return s.dtype == EGAT_BF16 && s.H >= mol_tc_heads(s) &&
         (nt == 1 || nt == 2 || nt == 4 || nt == 8 || nt == 9 || nt == 16 || nt == 18 || nt == 32);
}

int mol_tc_forward(const MolParams& p, cudaStream_t st) {
  return tc_dispatch(p.dv / 8, p.dk, [&](auto nt, auto kc, auto hp) {
    constexpr int NT = decltype(nt)::value, KC = decltype(kc)::value, HP = decltype(hp)::value;
    using L = TcLay<NT, KC, HP>;
    const size_t shm = std::max(2 * L::STAGE, 4 * 16 * (L::OUTROW + 2 * HP) * 4);
    return tc_launch(mol_fwd_tc_kernel<NT, KC, HP>, dim3(p.slots, p.H / HP, p.splits), shm, p, st);
  });
}

}  // namespace egat
