// Attention within each molecule on the fifth-generation tensor cores: the
// forward pass over long molecules (bf16 storage).
//
// A CTA takes one head and 128 query rows of a molecule, eight warps of them, and
// passes over the keys in stages of 64; two CTAs share an SM (one CTA of twice the rows
// is slower: 2.21 instead of 1.69 ms for 16,384 atoms at lmax 3):
//  * one warp brings the stages in (bulk copies, one per chunk, three stages in
//    flight) and writes their positions;
//  * one thread issues the products: S = Q K^T into one of two
//    64-column score buffers in tensor memory, and m += P H' with P from tensor
//    memory, where it replaces the scores;
//  * a row is two threads', of two warps that share its lanes: each
//    reads 32 of its 64 scores, applies cap, bias and exponential, and writes its
//    weights back as the sum of two bf16 numbers, one behind the other over the 64
//    columns of the scores.  (One thread with all 64 leaves two warps a scheduler to
//    hide each other's latency: 0.40 instead of 0.37 ms at 4,096 capped atoms.)  The row's
//    reference moves only when a score passes it by 2^8; only then do the two
//    exchange their maxima, and the accumulator is rescaled in place.
// While the warps work on one stage, the tensor core forms the next scores and the
// other CTA's products.  Work per pair and head is one exponential (and one
// root with a bias) on the special-function unit (8,191 atoms, lmax 3: 0.24 of 0.64 ms);
// cap and bias add 13 operations on the FMA pipe and bound it there (4,096 atoms, lmax 2:
// 0.17 of 0.37 ms).  The products take 0.05 ms at the measured rate in the second case and
// 0.35 ms in the first (16 + 2 x 128 columns a pair), where they bound it.  One plane of the weights took 0.46 and 0.35 ms for these
// two, with an error of m up to 1.4 times that of its own rounding.  Every wait is bounded.
#include <algorithm>

#include "molecule_umma.cuh"

namespace egat {
namespace {

// Operand blocks of a shape, in bytes; one of them is one bulk copy.
struct UmBlocks {
  int nt, nv;        // value chunks, and to a multiple of 16 columns (the last chunk zeros)
  int ks;            // k-steps of 16 of a score
  int v, pos, key;   // key block: [2 ks chunks][64][16 B], values [nv][64][16 B], x[64], y[64], z[64]
  int query;         // query block: [2 ks chunks][128][16 B]
  __host__ __device__ UmBlocks(int dv, int dk) {
    nt = dv >> 3;
    nv = (nt + 1) & ~1;
    ks = dk > 16 ? 2 : 1;
    v = 2 * ks * kUmStage * 16;
    pos = v + nv * kUmStage * 16;
    key = pos + kUmStage * 16;
    query = 2 * ks * kUmRows * 16;
  }
};

// q, k, the values and the key positions into those blocks, by head and tile (64
// keys; 128 query rows): 64 rows and up to 16 chunks a block through shared
// memory, read and written in whole runs.  Rows past a tile are zeros.
__global__ void __launch_bounds__(256) mol_pack_kernel(MolParams p, int key_slots, int query_slots) {
  const UmBlocks B(p.dv, p.dk);
  __shared__ uint4 sm[64][17];
  const bool keys = int(blockIdx.x) < key_slots;
  const int slot = keys ? blockIdx.x : blockIdx.x - key_slots;
  const MolTile t = keys ? mol_tile(6, p.a.kptr, p.a.kptr, p.nmol, p.nk, p.nk, slot)
                         : mol_tile(kUmRowsLog, p.a.qptr, p.a.qptr, p.nmol, p.nq, p.nq, slot);
  if (t.rows <= 0) return;
  const int qk_chunks = p.H * p.dk / 8, qk_slices = (qk_chunks + 15) / 16;
  const int val_chunks = p.D * p.C / 8, val_slices = (val_chunks + 15) / 16;
  int y = blockIdx.y, sub = 0;
  if (!keys) {   // 64 rows of the tile, slices of q
    sub = y & 1;
    y >>= 1;
  }
  const int last = keys ? qk_slices + val_slices : qk_slices;
  if (y > last) return;
  const int row0 = t.row0 + sub * 64, rows = min(64, t.rows - sub * 64);   // may be below one: zeros
  // logarithms of a run's chunks: a head's part of a query or key, of a degree, a degree
  const int kc = p.dk >> 3, klog = __ffs(kc) - 1, runlog = __ffs(p.C >> 3) - 1;
  unsigned char* const out = static_cast<unsigned char*>(keys ? p.kv : p.qp);
  const size_t block = keys ? B.key : B.query, slots = keys ? key_slots : query_slots;
  const size_t in_block = keys ? 0 : sub * 64 * 16;
  const int chunk_bytes = keys ? kUmStage * 16 : kUmRows * 16;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (y == last) {   // what no tensor fills, and positions
    for (int h = 0; h < p.H; ++h) {
      unsigned char* o = out + (h * slots + slot) * block + in_block;
      for (int r = threadIdx.x; r < 64; r += blockDim.x) {
        if (kc == 1) *reinterpret_cast<uint4*>(o + chunk_bytes + r * 16) = zero;
        if (keys && B.nv > B.nt) *reinterpret_cast<uint4*>(o + B.v + B.nt * chunk_bytes + r * 16) = zero;
        if (keys && p.a.slope)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            *reinterpret_cast<float*>(o + B.pos + (c * kUmStage + r) * 4) =
                r < rows ? p.a.posk[size_t(row0 + r) * 3 + c] : 0.f;
      }
    }
    return;
  }
  const bool val = y >= qk_slices;
  const int c0 = (val ? y - qk_slices : y) * 16, chunks = val ? val_chunks : qk_chunks;
  const uint4* src = static_cast<const uint4*>(val ? p.a.hp : keys ? p.a.k : p.a.q);
  const int c = threadIdx.x & 15;
  for (int r = threadIdx.x >> 4; r < 64; r += 16)
    if (c0 + c < chunks) sm[r][c] = r < rows ? __ldg(src + size_t(row0 + r) * chunks + c0 + c) : zero;
  __syncthreads();
  const int r = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < 16; i += 4) {
    const int x = c0 + i;
    if (x >= chunks) break;
    const int d = val ? x >> runlog : 0, in = val ? x & ((1 << runlog) - 1) : x, plog = val ? p.ch8log : klog;
    const int head = in >> plog, chunk = (d << plog) + (in & ((1 << plog) - 1));
    *reinterpret_cast<uint4*>(out + (head * slots + slot) * block + in_block + (val ? B.v : 0) + chunk * chunk_bytes +
                              r * 16) = sm[r][i];
  }
}

constexpr int kUmStages = 3;
constexpr int kUmThreads = 10 * 32;   // eight warps of rows, one of products, one of copies

// Shared memory of a CTA
struct UmLay : UmBlocks {
  static constexpr int NBARS = 2 * kUmStages + 8;
  static constexpr int COLS = 256;       // tensor memory: scores 2 x 64, accumulator up to 128
  int q, pair, bars, slot, flag, total;  // after the stages
  __host__ __device__ UmLay(int dv, int dk) : UmBlocks(dv, dk) {
    q = kUmStages * key;
    pair = q + query;                      // [4 pairs of warps][2][32] maxima or sums, then [..][2][2] flags
    bars = pair + 4 * (64 + 4) * 4;
    slot = bars + 8 * NBARS;
    flag = slot + 4;
    total = flag + 12;
  }
};

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kUmThreads, 2) mol_fwd_umma_kernel(MolParams p) {
  const UmLay L(p.dv, p.dk);
  extern __shared__ __align__(128) unsigned char um[];
  const int head = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const MolTile t = mol_tile(kUmRowsLog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) return;   // whole CTA
  const uint32_t base = tc_smem(um), bars = base + L.bars;
  auto full = [&](int s) { return bars + 8 * s; };
  auto freed = [&](int s) { return bars + 8 * (kUmStages + s); };
  const uint32_t qfull = bars + 8 * 2 * kUmStages, drained = qfull + 8;
  // Two of each by stage parity: a warp may be done with the next stage before
  // another is with this one, and a wait on one barrier for both stages would take
  // the phase before this one for the phase after it.
  auto sfull = [&](int b) { return bars + 8 * (2 * kUmStages + 2 + b); };
  auto pready = [&](int b) { return bars + 8 * (2 * kUmStages + 4 + b); };
  auto pvdone = [&](int b) { return bars + 8 * (2 * kUmStages + 6 + b); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(um + L.flag);
  const int n = t.o1 - t.o0, stages = (n + kUmStage - 1) / kUmStage;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kUmStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(freed(s), 1);
    }
    mbar_init(qfull, 1);
    mbar_init(drained, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(sfull(b), 1);
      mbar_init(pready(b), 8);
      mbar_init(pvdone(b), 1);
    }
    mbar_fence_init();
    *abort_flag = 0;
  }
  if (warp == 8) um_alloc<UmLay::COLS>(base + L.slot);
  um_before();
  __syncthreads();
  um_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(um + L.slot);

  int issued = 0;   // stages whose copies were issued (the copying thread's)
  if (warp == 9) {
    // ---- stages
    const unsigned char* kv = static_cast<const unsigned char*>(p.kv) +
                              (size_t(head) * p.kv_slots + (t.o0 >> 6) + t.seg) * L.key;
    if (lane == 0 && stages > 0) {
      mbar_arrive_expect_tx(qfull, L.query);
      bulk_g2s(base + L.q, static_cast<const unsigned char*>(p.qp) + (size_t(head) * p.slots + blockIdx.x) * L.query,
               L.query, qfull);
      for (int i = 0; i < stages; ++i) {
        const int s = i % kUmStages;
        if (i >= kUmStages && !bounded_wait(freed(s), (i / kUmStages - 1) & 1, kWaitPolls, abort_flag)) break;
        mbar_arrive_expect_tx(full(s), L.key);
        bulk_g2s(base + s * L.key, kv + size_t(i) * L.key, L.key, full(s));
        issued = i + 1;
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---- products
    if (lane == 0 && stages > 0) {
      bool ok = bounded_wait(qfull, 0, kWaitPolls, abort_flag);
      auto scores = [&](int i) {
        const uint32_t st = base + (i % kUmStages) * L.key;
#pragma unroll
        for (int k = 0; k < L.ks; ++k)
          um_mma_ss(tmem + (i & 1) * kUmStage,
                    um_k_major<kUmRows>(base + L.q + 2 * k * kUmRows * 16),
                    um_k_major<kUmStage>(st + 2 * k * kUmStage * 16), um_idesc(kUmStage, false), k > 0);
        um_commit(sfull(i & 1));
      };
      ok = ok && bounded_wait(full(0), 0, kWaitPolls, abort_flag);
      um_after();
      if (ok) scores(0);
      for (int i = 0; ok && i < stages; ++i) {
        if (i + 1 < stages) ok = bounded_wait(full((i + 1) % kUmStages), ((i + 1) / kUmStages) & 1, kWaitPolls, abort_flag);
        // the next score buffer holds the weights of stage i - 1 until that product is through
        if (ok && i > 0) ok = bounded_wait(pvdone((i - 1) & 1), ((i - 1) >> 1) & 1, kWaitPolls, abort_flag);
        if (!ok) break;
        um_after();
        if (i + 1 < stages) scores(i + 1);
        ok = bounded_wait(pready(i & 1), (i >> 1) & 1, kWaitPolls, abort_flag);
        if (!ok) break;
        um_after();
        const uint32_t st = base + (i % kUmStages) * L.key;
#pragma unroll
        for (int k = 0; k < kUmStage / 16; ++k)
          for (int w = 0; w < 2; ++w)   // the weights' planes
            um_mma_ts(tmem + 2 * kUmStage, tmem + (i & 1) * kUmStage + w * 32 + k * 8,
                      um_mn_major<kUmStage>(st + L.v + k * 256), um_idesc(L.nv * 8, true), i > 0 || k > 0 || w > 0);
        um_commit(pvdone(i & 1));
        // only for a stage that will come: an arrival that nothing waits for could land in
        // shared memory that the CTA has given up
        if (i + kUmStages < stages) um_commit(freed(i % kUmStages));
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: a row is two threads'
    const int half = warp >> 2, own = (warp & 3) * 32 + lane;
    const bool live = own < t.rows;
    const size_t row = size_t(t.row0) + (live ? own : 0);
    const uint32_t tm = tmem + (uint32_t((warp & 3) * 32) << 16);
    const int pair = warp & 3;
    volatile float* shared_row = reinterpret_cast<float*>(um + L.pair) + pair * 64 + lane;   // [half] * 32
    volatile int* flags = reinterpret_cast<int*>(um + L.pair) + 4 * 64 + pair * 4;         // [stage & 1][half]
    auto sync_pair = [&]() { asm volatile("bar.sync %0, 64;\n" ::"r"(1 + pair) : "memory"); };
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
    // a wait that gave up does not end the loop: the pair's barriers need both warps,
    // and later waits return at once
    bool ok = true;
    for (int i = 0; i < stages; ++i) {
      ok = um_wait(sfull(i & 1), (i >> 1) & 1, abort_flag) && ok;
      if (BIAS) ok = um_wait(full(i % kUmStages), (i / kUmStages) & 1, abort_flag) && ok;   // its positions
      um_after();
      const uint32_t ts = tm + (i & 1) * kUmStage;
      const int left = n - i * kUmStage - half * 32;
      const float* sp = reinterpret_cast<const float*>(um + (i % kUmStages) * L.key + L.pos) + half * 32;
      f32x2 w[16];
      // once with the reference and, where that has to move, once without: one
      // copy of the code, which would not fit the instruction cache twice
      bool move = i == 0;
#pragma unroll 1
      for (;;) {
        uint32_t s[32];
        um_ld32(ts + half * 32, s);
        const f32x2 rr = f2_set(move ? 0.f : ref);
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
        if constexpr (CAP) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            f32x2 x[8], unused[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = f2_mul(w[8 * k + e], c_in);
            tc_cap<8, false>(x, unused);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[8 * k + e] = x[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = f2_fma(w[e], CAP ? c_cap : c_in, rr);
        if constexpr (BIAS) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
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
        if (left < 32) {   // keys past the molecule
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b;
            f2_unpack(w[e], a, b);
            w[e] = f2_pack(2 * e < left ? a : -INFINITY, 2 * e + 1 < left ? b : -INFINITY);
          }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          f2_unpack(w[e], a, b);
          top[e & 1] = tc_max3(top[e & 1], a, b);
        }
        const float mx = fmaxf(top[0], top[1]);
        if (!move) {
          move = __any_sync(~0u, !(mx <= 8.f) || isnan(ref));
          if (lane == 0) flags[(i & 1) * 2 + half] = move;
          sync_pair();   // both have read their scores, too: the weights may replace them
          move = flags[(i & 1) * 2] | flags[(i & 1) * 2 + 1];
          if (!move) break;
          continue;
        }
        shared_row[half * 32] = mx;
        sync_pair();
        const float up = fmaxf(-ref, fmaxf(shared_row[0], shared_row[32]));   // a NaN reference drops out
        const bool empty = up == -INFINITY;                                    // all -inf so far
        const float f = empty || isnan(ref) ? 0.f : fast_exp2(-ref - up);
        ref = empty ? none : -up;
        sum = f2_mul(sum, f2_set(f));
        const f32x2 shift = f2_set(empty ? 0.f : -up);
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = f2_add(w[e], shift);
        if (i > 0) {   // rescale the accumulator, once the last stage's product is in it
          ok = um_wait(pvdone((i - 1) & 1), ((i - 1) >> 1) & 1, abort_flag) && ok;
          um_after();
#pragma unroll 1
          for (int c = half; c < L.nt; c += 2) {
            uint32_t o[8];
            um_ld8(tm + 2 * kUmStage + c * 8, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            um_st8(tm + 2 * kUmStage + c * 8, o);
          }
          um_st_wait();
        }
        break;
      }
      uint32_t pk[2][16];   // the weights as the sum of two bf16 numbers
      f32x2 part[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float a, b;
        f2_unpack(w[e], a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        part[e & 1] = f2_add(part[e & 1], f2_pack(a, b));
        uint32_t w2[2];
        tc_planes<2>(a, b, w2);
        pk[0][e] = w2[0];
        pk[1][e] = w2[1];
      }
      sum = f2_add(sum, f2_add(part[0], part[1]));
      um_st16(ts + half * 16, pk[0]);
      um_st16(ts + 32 + half * 16, pk[1]);
      um_st_wait();
      um_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready(i & 1));
    }
    if (ok && stages > 0) ok = um_wait(pvdone((stages - 1) & 1), ((stages - 1) >> 1) & 1, abort_flag);
    um_after();
    float l0, l1;
    f2_unpack(sum, l0, l1);
    sync_pair();   // the maxima have been read
    shared_row[half * 32] = l0 + l1;
    sync_pair();
    const float l = shared_row[0] + shared_row[32], inv = l == 0.f ? 0.f : 1.f / l;
    if (live && half == 0 && p.lse) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : -ref * kLn2 + logf(l);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.m) + row * (p.D * p.C);
    if (ok)
#pragma unroll 1
      for (int c = half; c < L.nt; c += 2) {
        uint32_t o[8] = {};
        if (stages > 0) um_ld8(tm + 2 * kUmStage + c * 8, o);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
        if (live)
          *reinterpret_cast<uint4*>(out + tc_val_off(p, head, c)) =
              make_uint4(tc_pack(v[0], v[1]), tc_pack(v[2], v[3]), tc_pack(v[4], v[5]), tc_pack(v[6], v[7]));
      }
  }
  um_release<UmLay::COLS>(abort_flag, 9, 8, drained, tmem, [&](volatile int* none) {
    if (issued > 0) bounded_wait(qfull, 0, kDrainPolls, none);
    for (int i = max(0, issued - kUmStages); i < issued; ++i)
      bounded_wait(full(i % kUmStages), (i / kUmStages) & 1, kDrainPolls, none);
  });
}

// The way out of a wait that gives up: a copy is on its way, and a wait for an
// arrival that never comes runs out of its polls.
__device__ uint4 g_selftest_source[64];
__global__ void __launch_bounds__(64) mol_wait_timeout_selftest_kernel(int polls) {
  __shared__ __align__(128) uint4 to[64];
  __shared__ __align__(8) uint64_t bar[3];
  __shared__ uint32_t slot;
  __shared__ int flag;
  const uint32_t full = smem_u32(bar), never = smem_u32(bar + 1), drained = smem_u32(bar + 2);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(full, 1);
    mbar_init(never, 1);
    mbar_init(drained, 1);
    mbar_fence_init();
    flag = 0;
  }
  if (warp == 0) um_alloc<32>(smem_u32(&slot));
  um_before();
  __syncthreads();
  um_after();
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&slot);
  if (warp == 1 && lane == 0) {
    mbar_arrive_expect_tx(full, sizeof(to));
    bulk_g2s(smem_u32(to), g_selftest_source, sizeof(to), full);
  } else if (warp == 0 && lane == 0) {
    bounded_wait(never, 0, polls, &flag);
  }
  __syncwarp();
  um_release<32>(&flag, 1, 0, drained, tmem, [&](volatile int* none) { bounded_wait(full, 0, kDrainPolls, none); });
}

}  // namespace

size_t mol_umma_key_bytes(const egat_mol_shape& s) {
  return size_t(mol_slots(s.nk, s.n_mol, kUmStage)) * s.H *
         UmBlocks((s.lmax + 1) * (s.lmax + 1) * (s.C / s.H), s.dk).key;
}
size_t mol_umma_query_bytes(const egat_mol_shape& s) {
  return size_t(mol_slots(s.nq, s.n_mol, kUmRows)) * s.H * UmBlocks(8, s.dk).query;
}

int mol_umma_pack(const MolParams& p, cudaStream_t st) {
  const int qk = (p.H * p.dk / 8 + 15) / 16, val = (p.D * p.C / 8 + 15) / 16;
  const dim3 grid(p.kv_slots + p.slots, std::max(qk + val + 1, (qk + 1) * 2));
  mol_pack_kernel<<<grid, 256, 0, st>>>(p, p.kv_slots, p.slots);
  return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA;
}

// up to 128 value columns a head: the accumulator beside the scores in 256
// columns of tensor memory
bool mol_umma_supported(const egat_mol_shape& s) {
  return s.dtype == EGAT_BF16 && (s.lmax + 1) * (s.lmax + 1) * (s.C / s.H) <= 128;
}

int mol_umma_forward(const MolParams& p, cudaStream_t st) {
  return mol_flags(p.cap > 0.f, p.a.slope != nullptr, [&](auto cap, auto bias) {
    return mol_launch(mol_fwd_umma_kernel<decltype(cap)::value, decltype(bias)::value>, dim3(p.slots, p.H), kUmThreads,
                      UmLay(p.dv, p.dk).total, p, st);
  });
}

int launch_molecule_wait_timeout_selftest(int polls, cudaStream_t st) {
  mol_wait_timeout_selftest_kernel<<<1, 64, 0, st>>>(polls);
  return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA;
}
int take_wait_timeouts_molecule(cudaStream_t st, unsigned int* count) {
  return take_unit_wait_timeouts(st, count) == 0 ? EGAT_OK : EGAT_ERR_CUDA;
}

}  // namespace egat
