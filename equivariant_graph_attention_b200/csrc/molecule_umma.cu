// Attention within each molecule on the fifth-generation tensor cores: the
// forward pass over long molecules (bf16 storage).
//
// A CTA takes one head and 128 G query rows of a molecule, in G groups of four
// warps whose lanes are rows, and passes over the keys in stages of 64:
//  * one warp brings the stages in (bulk copies, one per chunk, three stages in
//    flight) and writes their positions;
//  * one thread issues the products: S = Q K^T into one of a group's two
//    64-column score buffers in tensor memory, and m += P H' with P from tensor
//    memory, where it replaces the scores;
//  * a thread of a group reads the 64 scores of its row, applies cap, bias and
//    exponential, and writes its weights back as bf16.  A row is one thread's:
//    maximum and normaliser need no exchange.  The row's reference moves only when
//    a score passes it by 2^8; then the accumulator is rescaled in place.
// While a group works on one stage, the tensor core forms its next scores and
// the other group's products.  Work per pair and head is one exponential (and one
// root with a bias) on the special-function unit, which is what bounds it: the
// products take a quarter of that at 16 + 72 columns.  Every wait is bounded.
#include "molecule_umma.cuh"

namespace egat {
namespace {

// [n][row] bf16 tensors into [head][chunk][n] chunks of 8 columns, 64 rows and up
// to 16 chunks a block through shared memory, read and written in whole runs.
struct PackJob {
  const uint4* src;
  uint4* dst;
  int n, row_chunks;   // rows, chunks of a row
  int head_chunks;     // chunks of a head in a run of heads (its channels / 8, or dk / 8)
  int run_chunks;      // chunks of one run of heads (C / 8, or a whole row)
  int dst_chunks;      // chunks of a head in dst
  int slices;          // blocks over a row: 16 chunks each
  int blocks;          // 64-row blocks
};
struct PackArgs {
  PackJob job[3];
};
__global__ void __launch_bounds__(256) mol_pack_kernel(PackArgs args) {
  __shared__ uint4 sm[64][17];
  int b = blockIdx.x, which = 0;
  while (b >= args.job[which].slices * args.job[which].blocks) b -= args.job[which].slices * args.job[which++].blocks;
  const PackJob& j = args.job[which];
  const int row0 = (b / j.slices) * 64, c0 = (b % j.slices) * 16;
  const int c = threadIdx.x & 15;
  for (int r = threadIdx.x >> 4; r < 64; r += 16)
    if (row0 + r < j.n && c0 + c < j.row_chunks) sm[r][c] = __ldg(j.src + size_t(row0 + r) * j.row_chunks + c0 + c);
  __syncthreads();
  const int r = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < 16; i += 4)
    if (row0 + r < j.n && c0 + i < j.row_chunks) {
      const int x = c0 + i, run = x / j.run_chunks, in = x - run * j.run_chunks;
      const int head = in / j.head_chunks, chunk = run * j.head_chunks + in - head * j.head_chunks;
      j.dst[(size_t(head) * j.dst_chunks + chunk) * j.n + row0 + r] = sm[r][i];
    }
}

constexpr int kUmStages = 3;

// Shared memory of a CTA, in bytes; the numbers of chunks are those of the shape.
template <int G>
struct UmLay {
  static constexpr int NBARS = 2 * kUmStages + 1 + 6 * G;
  static constexpr int COLS = 256 * G;   // per group: scores 2 x 64, accumulator up to 128
  int nt, nv;      // value chunks, and to a multiple of 16 columns (the last chunk zeros)
  int ks;          // k-steps of 16 of a score
  int v, pos, stage, q, bars, slot, flag, total;
  __host__ __device__ UmLay(int dv, int dk) {
    nt = dv >> 3;
    nv = (nt + 1) & ~1;
    ks = dk > 16 ? 2 : 1;
    v = 2 * ks * kUmStage * 16;               // after keys [2 ks chunks][64][16 B]: values [nv][64][16 B]
    pos = v + nv * kUmStage * 16;             // x[64], y[64], z[64]
    stage = pos + kUmStage * 16;
    q = kUmStages * stage;                    // [G][2 ks chunks][128][16 B]
    bars = q + G * 2 * ks * kUmRows * 16;
    slot = bars + 8 * NBARS;
    flag = slot + 4;
    total = flag + 12;
  }
};

template <int G, bool CAP, bool BIAS>
__global__ void __launch_bounds__((4 * G + 2) * 32, G == 1 ? 2 : 1) mol_fwd_umma_kernel(MolParams p) {
  const UmLay<G> L(p.dv, p.dk);
  extern __shared__ __align__(128) unsigned char um[];
  const int head = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const MolTile t = mol_tile(G == 2 ? 8 : 7, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) return;   // whole CTA
  const uint32_t base = tc_smem(um), bars = base + L.bars;
  auto full = [&](int s) { return bars + 8 * s; };
  auto freed = [&](int s) { return bars + 8 * (kUmStages + s); };
  const uint32_t qfull = bars + 8 * 2 * kUmStages;
  // Two of each by stage parity: a warp may be done with the next stage before
  // another is with this one, and a wait on one barrier for both stages would take
  // the phase before this one for the phase after it.
  auto sfull = [&](int g, int b) { return bars + 8 * (2 * kUmStages + 1 + 6 * g + b); };
  auto pready = [&](int g, int b) { return bars + 8 * (2 * kUmStages + 1 + 6 * g + 2 + b); };
  auto pvdone = [&](int g, int b) { return bars + 8 * (2 * kUmStages + 1 + 6 * g + 4 + b); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(um + L.flag);
  const int n = t.o1 - t.o0, stages = (n + kUmStage - 1) / kUmStage;
  const int groups = (t.rows + kUmRows - 1) / kUmRows;   // groups with rows

  // rows that no copy fills are zeros, not what was there before
  for (int i = threadIdx.x; i < L.bars / 16; i += blockDim.x) reinterpret_cast<uint4*>(um)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kUmStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(freed(s), 1);
    }
    mbar_init(qfull, 1);
    for (int g = 0; g < G; ++g) {
      mbar_init(sfull(g, 0), 1);
      mbar_init(sfull(g, 1), 1);
      mbar_init(pready(g, 0), 4);
      mbar_init(pready(g, 1), 4);
      mbar_init(pvdone(g, 0), 1);
      mbar_init(pvdone(g, 1), 1);
    }
    mbar_fence_init();
    *abort_flag = 0;
  }
  if (warp == 4 * G) um_alloc<UmLay<G>::COLS>(base + L.slot);
  fence_proxy_async_smem();
  um_before();
  __syncthreads();
  um_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(um + L.slot);

  if (warp == 4 * G + 1) {
    // ---- stages
    const int kc = p.dk >> 3;
    if (lane == 0 && stages > 0) {
      mbar_arrive_expect_tx(qfull, uint32_t(t.rows * kc * 16));
      for (int g = 0; g < groups; ++g) {
        const int rows = min(kUmRows, t.rows - g * kUmRows);
        for (int c = 0; c < kc; ++c)
          bulk_g2s(base + L.q + (g * 2 * L.ks + c) * kUmRows * 16,
                   p.qp + (size_t(head) * kc + c) * p.nq + t.row0 + g * kUmRows, rows * 16, qfull);
      }
    }
    for (int i = 0; i < stages; ++i) {
      const int s = i % kUmStages, k0 = t.o0 + i * kUmStage, rows = min(kUmStage, t.o1 - k0);
      if (i >= kUmStages && !bounded_wait(freed(s), (i / kUmStages - 1) & 1, kWaitPolls, abort_flag)) break;
      if (BIAS) {
        float* sp = reinterpret_cast<float*>(um + s * L.stage + L.pos);
        for (int r = lane; r < rows; r += 32)
#pragma unroll
          for (int c = 0; c < 3; ++c) sp[c * kUmStage + r] = __ldg(p.a.posk + size_t(k0 + r) * 3 + c);
      }
      __syncwarp();
      if (lane == 0) {
        const uint32_t st = base + s * L.stage;
        mbar_arrive_expect_tx(full(s), uint32_t((kc + L.nt) * rows * 16));
        for (int c = 0; c < kc; ++c)
          bulk_g2s(st + c * kUmStage * 16, p.kp + (size_t(head) * kc + c) * p.nk + k0, rows * 16, full(s));
        for (int c = 0; c < L.nt; ++c)
          bulk_g2s(st + L.v + c * kUmStage * 16, p.vp + (size_t(head) * L.nt + c) * p.nk + k0, rows * 16, full(s));
      }
      __syncwarp();
    }
    if (*abort_flag && lane == 0) {   // copies in flight land before the memory is given up
      volatile int none = 0;
      if (stages > 0) bounded_wait(qfull, 0, kDrainPolls, &none);
      for (int s = 0; s < kUmStages; ++s) {
        int last = stages - 1;
        while (last >= 0 && last % kUmStages != s) --last;
        if (last >= 0) bounded_wait(full(s), (last / kUmStages) & 1, kDrainPolls, &none);
      }
    }
  } else if (warp == 4 * G) {
    // ---- products
    if (lane == 0 && stages > 0) {
      bool ok = bounded_wait(qfull, 0, kWaitPolls, abort_flag);
      auto scores = [&](int i, int g) {
        const uint32_t st = base + (i % kUmStages) * L.stage;
#pragma unroll
        for (int k = 0; k < L.ks; ++k)
          um_mma_ss(tmem + g * 256 + (i & 1) * kUmStage,
                    um_k_major<kUmRows>(base + L.q + (g * 2 * L.ks + 2 * k) * kUmRows * 16),
                    um_k_major<kUmStage>(st + 2 * k * kUmStage * 16), um_idesc(kUmStage, false), k > 0);
        um_commit(sfull(g, i & 1));
      };
      ok = ok && bounded_wait(full(0), 0, kWaitPolls, abort_flag);
      um_after();
      if (ok)
        for (int g = 0; g < groups; ++g) scores(0, g);
      for (int i = 0; ok && i < stages; ++i) {
        if (i + 1 < stages) ok = bounded_wait(full((i + 1) % kUmStages), ((i + 1) / kUmStages) & 1, kWaitPolls, abort_flag);
        for (int g = 0; ok && g < groups; ++g) {
          // its score buffer holds the weights of stage i - 1 until that product is through
          if (i > 0) ok = bounded_wait(pvdone(g, (i - 1) & 1), ((i - 1) >> 1) & 1, kWaitPolls, abort_flag);
          if (!ok) break;
          um_after();
          if (i + 1 < stages) scores(i + 1, g);
          ok = bounded_wait(pready(g, i & 1), (i >> 1) & 1, kWaitPolls, abort_flag);
          if (!ok) break;
          um_after();
          const uint32_t st = base + (i % kUmStages) * L.stage;
#pragma unroll
          for (int k = 0; k < kUmStage / 16; ++k)
            um_mma_ts(tmem + g * 256 + 2 * kUmStage, tmem + g * 256 + (i & 1) * kUmStage + k * 8,
                      um_mn_major<kUmStage>(st + L.v + k * 256), um_idesc(L.nv * 8, true), i > 0 || k > 0);
          um_commit(pvdone(g, i & 1));
        }
        if (ok) um_commit(freed(i % kUmStages));
      }
    }
    __syncwarp();
  } else if ((warp >> 2) < groups) {
    // ---- softmax: a thread is a row
    const int g = warp >> 2, own = g * kUmRows + (warp & 3) * 32 + lane;
    const bool live = own < t.rows;
    const size_t row = size_t(t.row0) + (live ? own : 0);
    const uint32_t tm = tmem + (uint32_t((warp & 3) * 32) << 16) + g * 256;
    f32x2 px = 0, py = 0, pz = 0, slope = 0;
    if (BIAS) {
      const float* x = p.a.posq + row * 3;
      px = f2_set(-x[0]);
      py = f2_set(-x[1]);
      pz = f2_set(-x[2]);
      slope = f2_set(-p.a.slope[head] * kLog2e);
    }
    const f32x2 c_in = f2_set(CAP ? p.scale * p.inv_cap : p.scale * kLog2e), c_cap = f2_set(p.cap * kLog2e);
    const float none = __int_as_float(0x7fffffff);
    float ref = none;   // minus the reference; NaN: none yet
    f32x2 sum = 0;
    bool ok = true;
    for (int i = 0; i < stages; ++i) {
      ok = um_wait(sfull(g, i & 1), (i >> 1) & 1, abort_flag);
      if (BIAS) ok = ok && um_wait(full(i % kUmStages), (i / kUmStages) & 1, abort_flag);   // its positions
      if (!ok) break;
      um_after();
      const uint32_t ts = tm + (i & 1) * kUmStage;
      const int left = n - i * kUmStage;
      const float* sp = reinterpret_cast<const float*>(um + (i % kUmStages) * L.stage + L.pos);
      f32x2 w[32];
      // base-2 scores of the row plus r
      auto scores = [&](float r) {
        uint32_t s[64];
        um_ld64(ts, s);
        const f32x2 rr = f2_set(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
        if constexpr (CAP) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f32x2 x[8], unused[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = f2_mul(w[8 * k + e], c_in);
            tc_cap<8, false>(x, unused);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[8 * k + e] = x[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = f2_fma(w[e], CAP ? c_cap : c_in, rr);
        if constexpr (BIAS) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sp + 2 * e);
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sp + kUmStage + 2 * e);
            const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(sp + 2 * kUmStage + 2 * e);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const f32x2 dx = f2_add(k ? x.y : x.x, px), dy = f2_add(k ? y.y : y.x, py), dz = f2_add(k ? z.y : z.x, pz);
              float a, b;
              f2_unpack(f2_fma(dx, dx, f2_fma(dy, dy, f2_mul(dz, dz))), a, b);
              w[e + k] = f2_fma(f2_pack(mol_sqrt(a), mol_sqrt(b)), slope, w[e + k]);
            }
          }
        }
      };
      auto row_max = [&]() {
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float a, b;
          f2_unpack(w[e], a, b);
          m[e & 3] = tc_max3(m[e & 3], a, b);
        }
        return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      };
      auto mask = [&]() {   // keys past the molecule
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float a, b;
          f2_unpack(w[e], a, b);
          w[e] = f2_pack(2 * e < left ? a : -INFINITY, 2 * e + 1 < left ? b : -INFINITY);
        }
      };
      // once with the reference and, where that has to move, once without: one
      // copy of the code, which would not fit the instruction cache twice
      bool move = i == 0;
#pragma unroll 1
      for (;;) {
        scores(move ? 0.f : ref);
        if (left < kUmStage) mask();
        if (move) break;
        move = __any_sync(~0u, !(row_max() <= 8.f) || isnan(ref));
        if (!move) break;
      }
      if (__builtin_expect(move, 0)) {
        const float up = fmaxf(-ref, row_max());   // a NaN reference drops out
        const bool empty = up == -INFINITY;        // all -inf so far
        const float f = empty || isnan(ref) ? 0.f : fast_exp2(-ref - up);
        ref = empty ? none : -up;
        sum = f2_mul(sum, f2_set(f));
        const f32x2 shift = f2_set(empty ? 0.f : -up);
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = f2_add(w[e], shift);
        if (i > 0) {   // rescale the accumulator, once the last stage's product is in it
          ok = um_wait(pvdone(g, (i - 1) & 1), ((i - 1) >> 1) & 1, abort_flag);
          if (!ok) break;
          um_after();
#pragma unroll 1
          for (int c = 0; c < L.nt; ++c) {
            uint32_t o[8];
            um_ld8(tm + 2 * kUmStage + c * 8, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            um_st8(tm + 2 * kUmStage + c * 8, o);
          }
          um_st_wait();
        }
      }
      uint32_t pk[32];
      f32x2 part[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float a, b;
        f2_unpack(w[e], a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        part[e & 3] = f2_add(part[e & 3], f2_pack(a, b));
        pk[e] = tc_pack(a, b);
      }
      sum = f2_add(sum, f2_add(f2_add(part[0], part[1]), f2_add(part[2], part[3])));
      um_st32(ts, pk);
      um_st_wait();
      um_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready(g, i & 1));
    }
    if (ok && stages > 0) ok = um_wait(pvdone(g, (stages - 1) & 1), ((stages - 1) >> 1) & 1, abort_flag);
    um_after();
    float l0, l1;
    f2_unpack(sum, l0, l1);
    const float l = l0 + l1, inv = l == 0.f ? 0.f : 1.f / l;
    if (live && p.lse) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : -ref * kLn2 + logf(l);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.m) + row * (p.D * p.C);
    if (ok)
#pragma unroll 1
      for (int c = 0; c < L.nt; ++c) {
        uint32_t o[8] = {};
        if (stages > 0) {
          um_ld8(tm + 2 * kUmStage + c * 8, o);
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
        if (live)
          *reinterpret_cast<uint4*>(out + tc_val_off(p, head, c)) =
              make_uint4(tc_pack(v[0], v[1]), tc_pack(v[2], v[3]), tc_pack(v[4], v[5]), tc_pack(v[6], v[7]));
      }
  }
  if (*abort_flag && warp == 4 * G && lane == 0) {   // products in flight end before tensor memory is freed
    volatile int none = 0;
    um_commit(qfull);   // its second phase: everything issued so far
    bounded_wait(qfull, 1, kDrainPolls, &none);
  }
  um_before();
  __syncthreads();
  if (warp == 4 * G) {
    um_after();
    um_dealloc<UmLay<G>::COLS>(tmem);
  }
}

PackJob pack_job(const void* src, void* dst, int n, int row, int head, int run, int heads) {
  PackJob j;
  j.src = static_cast<const uint4*>(src);
  j.dst = static_cast<uint4*>(dst);
  j.n = n;
  j.row_chunks = row / 8;
  j.head_chunks = head / 8;
  j.run_chunks = run / 8;
  j.dst_chunks = j.row_chunks / heads;
  j.slices = (j.row_chunks + 15) / 16;
  j.blocks = (n + 63) / 64;
  return j;
}

}  // namespace

int mol_umma_pack(const MolParams& p, cudaStream_t st) {
  PackArgs a;
  a.job[0] = pack_job(p.a.q, const_cast<uint4*>(p.qp), p.nq, p.H * p.dk, p.dk, p.H * p.dk, p.H);
  a.job[1] = pack_job(p.a.k, const_cast<uint4*>(p.kp), p.nk, p.H * p.dk, p.dk, p.H * p.dk, p.H);
  a.job[2] = pack_job(p.a.hp, const_cast<uint4*>(p.vp), p.nk, p.D * p.C, p.ch, p.C, p.H);
  long long blocks = 0;
  for (const PackJob& j : a.job) blocks += (long long)j.slices * j.blocks;
  if (blocks > 0) mol_pack_kernel<<<unsigned(blocks), 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA;
}

// up to 128 value columns a head: a group's accumulator beside its scores in 256
// columns of tensor memory
bool mol_umma_supported(const egat_mol_shape& s) {
  return s.dtype == EGAT_BF16 && (s.lmax + 1) * (s.lmax + 1) * (s.C / s.H) <= 128;
}

int mol_umma_forward(const MolParams& p, int groups, cudaStream_t st) {
  return mol_flags(p.cap > 0.f, p.a.slope != nullptr, [&](auto cap, auto bias) {
    constexpr bool CAP = decltype(cap)::value, BIAS = decltype(bias)::value;
    const dim3 grid(p.slots, p.H);
    return groups == 2 ? mol_launch(mol_fwd_umma_kernel<2, CAP, BIAS>, grid, 320, UmLay<2>(p.dv, p.dk).total, p, st)
                       : mol_launch(mol_fwd_umma_kernel<1, CAP, BIAS>, grid, 192, UmLay<1>(p.dv, p.dk).total, p, st);
  });
}

int take_wait_timeouts_molecule(cudaStream_t st, unsigned int* count) {
  return take_unit_wait_timeouts(st, count) == 0 ? EGAT_OK : EGAT_ERR_CUDA;
}

}  // namespace egat
