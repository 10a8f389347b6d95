// Building blocks of the tensor-core kernels of the attention within molecules.
//
// A CTA has four warps; a warp owns 16 rows and HP heads of them, and meets the
// other side's rows 16 at a time from shared-memory stages of 64 rows.  The
// warps stand side by side over rows (RW of them, a tile has 16 RW rows) and,
// where rows are few, over the stage's rows (4 / RW), whose sums are joined
// through shared memory at the end.  HP = 2 where the accumulators allow: two
// heads share the distances of a pair, and their rows of a degree are 32
// contiguous bytes, a whole memory sector.
//
// Products are mma.sync m16n8k16 with float32 accumulators that stay in
// registers with the online softmax.  A staged row is HP * KC chunks (16 bytes)
// of queries or keys and HP * NT chunks of values, each part padded to an odd
// number of chunks, so that the eight rows of an 8 x 8 ldmatrix hit different
// banks.  Rows past the molecule are zero-filled: NaN of a neighbour cannot
// enter a product.
//
// float32 storage takes the same kernels with PL = 3 planes: every operand, the
// weights and dS too, is the sum of three bf16 numbers (24 bits), and a product is
// the six bf16 products whose planes add up to two at most; what is left out is
// below 2^-25 of the terms.  Six products at the tensor rate are four thirds of the
// FMA pipe's rate, without its shared-memory reads (216-water box: 107 us on that
// pipe).  A stage is copied as it is while the last one is worked on, and each lane then
// splits what it copied; a warp takes one head.
#pragma once

#include <algorithm>

#include "molecule.cuh"

namespace egat {
namespace {

constexpr int kTcThreads = 128;
constexpr int kTcStage = 64;   // rows of a stage

template <int PL>
struct TcStorage { using T = __nv_bfloat16; };
template <>
struct TcStorage<3> { using T = float; };

template <int NT, int KC, int HP, int PL>
struct TcLay {
  using T = typename TcStorage<PL>::T;
  static_assert(PL == 1 || (PL == 3 && HP == 1), "float32: three planes, one head");
  static constexpr int PK = HP * KC * 16, PV = HP * NT * 16;   // bytes of a row's plane
  static constexpr int RK = (HP * KC * PL | 1) * 16;           // bytes of a staged query/key row
  static constexpr int RV = (HP * NT * PL | 1) * 16;           // bytes of a staged value row
  static constexpr int QK = 0;
  static constexpr int VAL = QK + kTcStage * RK;
  static constexpr int POS = VAL + kTcStage * RV;    // x[64], y[64], z[64]
  static constexpr int ROW = POS + kTcStage * 12;    // per head: lse2[64], delta[64]
  static constexpr int STAGE = ROW + HP * kTcStage * 8;
  // float32: one split stage, and behind it what was copied: rows of both parts, then
  // positions and row numbers
  static constexpr int BUFS = PL == 1 ? 2 : 1;
  static constexpr int RAWV = STAGE + kTcStage * KC * 32, RAWP = RAWV + kTcStage * NT * 32;
  static constexpr int BYTES = PL == 1 ? 2 * STAGE : RAWP + kTcStage * 20;   // all stages
  static constexpr int OUTROW = HP * NT * 8 + 8;     // floats of a joined row (bank spread)
};

__device__ __forceinline__ uint32_t tc_smem(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }
// 16 bytes, or (ok false) nothing from src and zeros
__device__ __forceinline__ void tc_cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tc_cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void tc_move4(uint32_t to, uint32_t from) {
  asm volatile("{\n .reg .b32 x;\n ld.shared.b32 x, [%1];\n st.shared.b32 [%0], x;\n}\n" ::"r"(to), "r"(from) : "memory");
}
__device__ __forceinline__ void tc_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void tc_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

__device__ __forceinline__ void tc_ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void tc_ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void tc_ldsm2(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];\n" : "=r"(r0), "=r"(r1) : "r"(a));
}
__device__ __forceinline__ void tc_ldsm2t(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];\n" : "=r"(r0), "=r"(r1) : "r"(a));
}
// c += a b; fragment of a 16 x 8 chunk of A: rows g (index 0) and g + 8 (index 1)
__device__ __forceinline__ void tc_mma16(float (&c)[4], const uint32_t (&a0)[2], const uint32_t (&a1)[2],
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0[0]), "r"(a0[1]), "r"(a1[0]), "r"(a1[1]), "r"(b0), "r"(b1));
}
// c = a b
__device__ __forceinline__ void tc_mma16_first(float (&c)[4], const uint32_t (&a0)[2], const uint32_t (&a1)[2],
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0[0]), "r"(a0[1]), "r"(a1[0]), "r"(a1[1]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void tc_mma8(float (&c)[4], const uint32_t (&a)[2], uint32_t b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(b));
}
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// (a, b) as pairs of the PL planes
template <int PL>
__device__ __forceinline__ void tc_planes(float a, float b, uint32_t (&w)[PL]) {
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    w[i] = tc_pack(a, b);
    if (i + 1 < PL) {
      a -= __uint_as_float(w[i] << 16);
      b -= __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// max(a, b, c) in one instruction (the three-input form of sm_100); drops NaN
// operands unless all are NaN
__device__ __forceinline__ float tc_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ f32x2 f2_set(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(~0u, x, 1);
  return x + __shfl_xor_sync(~0u, x, 2);
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}

// offset of value chunk x (8 columns) of head h inside a row of [D][C]
__device__ __forceinline__ int tc_val_off(const MolParams& p, int h, int x) {
  return (x >> p.ch8log) * p.C + h * p.ch + ((x & ((1 << p.ch8log) - 1)) << 3);
}

// Copies consecutive stages of 64 rows of heads head0...  A row's W chunks are
// copied by W lanes, 32 / W rows at a time, so a lane keeps its chunk and advances
// by whole rows.  Rows from `end` on arrive as zeros.
template <int W, int PL>
struct TcPart {
  using T = typename TcStorage<PL>::T;
  static_assert(W <= 32, "a row's chunks are one warp's");
  static constexpr int ROWS = 32 / W, STEP = ROWS * (kTcThreads / 32), ITS = (kTcStage + STEP - 1) / STEP;
  const T* src;   // this lane's chunk of its first row
  int ld;         // elements from row to row
  uint32_t dst;
  int row;        // its first row in a stage; past the stage: nothing to copy
  __device__ __forceinline__ void init(const T* base, int ld_, int off, int r0, uint32_t at, int rs) {
    const int lane = threadIdx.x & 31, r = (threadIdx.x >> 5) * ROWS + lane / W;
    row = lane < ROWS * W ? r : kTcStage;
    ld = ld_;
    src = base + size_t(r0 + r) * ld + off;
    dst = at + r * rs + (lane % W) * 16;
  }
  // bf16: into a stage; float32: as it is, 32 bytes a chunk, to `st`
  template <int RS>
  __device__ __forceinline__ void load(uint32_t st, int left, bool have) {
    const int need = (left + 15) & ~15;   // rows that the last step of 16 meets
    if (row < kTcStage) {
      if (PL == 1 && left >= kTcStage && have) {
#pragma unroll
        for (int i = 0; i < ITS; ++i)
          if (kTcStage % STEP == 0 || row + i * STEP < kTcStage)
            tc_cp16(st + dst + i * STEP * RS, src + size_t(i) * STEP * ld, true);
      } else {
#pragma unroll
        for (int i = 0; i < ITS; ++i)
          if (i * STEP < need && (kTcStage % STEP == 0 || row + i * STEP < kTcStage)) {
            const bool ok = have && row + i * STEP < left;
            const T* x = src + size_t(i) * STEP * ld;
            if constexpr (PL == 1) {
              tc_cp16(st + dst + i * STEP * RS, x, ok);
            } else {
              const uint32_t to = st + ((row + i * STEP) * W + (threadIdx.x & 31) % W) * 32;
              tc_cp16(to, x, ok);
              tc_cp16(to + 16, x + 4, ok);
            }
          }
      }
    }
    src += size_t(kTcStage) * ld;
  }
  // float32: what this lane copied to `raw`, split, into the stage at st
  template <int RS>
  __device__ __forceinline__ void split(uint32_t st, uint32_t raw, int left) const {
    const int need = (left + 15) & ~15;
    if (row < kTcStage)
#pragma unroll 2
      for (int i = 0; i < ITS; ++i) {
        if (i * STEP >= need || row + i * STEP >= kTcStage) break;
        const uint32_t from = raw + ((row + i * STEP) * W + (threadIdx.x & 31) % W) * 32;
        float v[8];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(from) : "memory");
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(from + 16) : "memory");
        uint32_t w[4][PL];
#pragma unroll
        for (int e = 0; e < 4; ++e) tc_planes<PL>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
        for (int k = 0; k < PL; ++k)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(st + dst + i * STEP * RS + k * W * 16),
                       "r"(w[0][k]), "r"(w[1][k]), "r"(w[2][k]), "r"(w[3][k])
                       : "memory");
      }
  }
};
template <int NT, int KC, int HP, int PL>
struct TcLoader {
  using L = TcLay<NT, KC, HP, PL>;
  using T = typename L::T;
  TcPart<HP * KC, PL> qk;
  TcPart<HP * NT, PL> val;
  const float* pos;
  bool have;   // at dk 8 the second chunk is zeros
  // the first stage starts at row r0 (r0 < end)
  __device__ __forceinline__ void init(const MolParams& p, const void* q, const void* v, const float* positions,
                                       int head0, int r0) {
    const int lane = threadIdx.x & 31, cq = lane % (HP * KC), cv = lane % (HP * NT);
    have = (cq % KC) * 8 < p.dk;
    qk.init(static_cast<const T*>(q), p.H * p.dk, (head0 + cq / KC) * p.dk + (have ? cq % KC : 0) * 8, r0, L::QK, L::RK);
    val.init(static_cast<const T*>(v), p.D * p.C, tc_val_off(p, head0 + cv % HP, cv / HP), r0, L::VAL, L::RV);
    pos = p.a.slope ? positions + size_t(r0) * 3 : nullptr;
  }
  // bf16: the next stage to st; float32: to the copies' place behind the stage at st
  __device__ __forceinline__ void load(uint32_t st, int left) {
    qk.template load<L::RK>(PL == 1 ? st : st + L::STAGE, left, have);
    val.template load<L::RV>(PL == 1 ? st : st + L::RAWV, left, true);
    if (pos) {
      const int c = threadIdx.x >> 5;
      if (c < 3)
#pragma unroll
        for (int r = threadIdx.x & 31; r < kTcStage; r += 32)
          tc_cp4(st + (PL == 1 ? L::POS : L::RAWP) + c * (kTcStage * 4) + r * 4, r < left ? pos + r * 3 + c : pos, r < left);
      pos += kTcStage * 3;
    }
  }
  // float32: the copies (complete for this thread) into the stage at st
  __device__ __forceinline__ void split(uint32_t st, int left) const {
    if constexpr (PL == 3) {
      qk.template split<L::RK>(st, st + L::STAGE, left);
      val.template split<L::RV>(st, st + L::RAWV, left);
      if (pos && threadIdx.x < 96)
#pragma unroll
        for (int r = threadIdx.x & 31; r < kTcStage; r += 32)
          tc_move4(st + L::POS + (threadIdx.x >> 5) * (kTcStage * 4) + r * 4,
                   st + L::RAWP + (threadIdx.x >> 5) * (kTcStage * 4) + r * 4);
    }
  }
};

// Two elements as pairs of the planes
__device__ __forceinline__ void tc_load2(const __nv_bfloat16* x, bool ok, uint32_t (&w)[1]) {
  w[0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(x)) : 0u;
}
__device__ __forceinline__ void tc_load2(const float* x, bool ok, uint32_t (&w)[3]) {
  const float2 v = ok ? __ldg(reinterpret_cast<const float2*>(x)) : make_float2(0.f, 0.f);
  tc_planes<3>(v.x, v.y, w);
}
__device__ __forceinline__ void tc_store2(__nv_bfloat16* x, float a, float b) {
  *reinterpret_cast<uint32_t*>(x) = tc_pack(a, b);
}
__device__ __forceinline__ void tc_store2(float* x, float a, float b) { *reinterpret_cast<float2*>(x) = make_float2(a, b); }
// Eight elements of a row
__device__ __forceinline__ void tc_store8(__nv_bfloat16* x, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(x) =
      make_uint4(tc_pack(v[0], v[1]), tc_pack(v[2], v[3]), tc_pack(v[4], v[5]), tc_pack(v[6], v[7]));
}
__device__ __forceinline__ void tc_store8(float* x, const float (&v)[8]) {
  reinterpret_cast<float4*>(x)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(x)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A fragments of this lane's rows (r0 = row g, r1 = row g + 8) from global memory
template <int NT, int PL>
__device__ __forceinline__ void tc_frag_val(const MolParams& p, const void* src, size_t r0, size_t r1, bool l0, bool l1,
                                            int head, uint32_t (&f)[PL][NT][2], int c0 = 0) {
  const typename TcStorage<PL>::T* x = static_cast<const typename TcStorage<PL>::T*>(src);
  const int t2 = (threadIdx.x & 3) * 2;
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t w[PL];
      tc_load2(x + (r ? r1 : r0) * (p.D * p.C) + tc_val_off(p, head, c0 + c) + t2, r ? l1 : l0, w);
#pragma unroll
      for (int k = 0; k < PL; ++k) f[k][c][r] = w[k];
    }
}

// ... and from shared memory: base is the lane's address of chunk 0 of its rows (row
// by lane & 15, chunk by lane / 16)
template <int NC, int PL>
__device__ __forceinline__ void tc_frag_rows(uint32_t base, int step, int plane, uint32_t (&f)[PL][NC][2]) {
#pragma unroll
  for (int k = 0; k < PL; ++k) {
#pragma unroll
    for (int c = 0; c + 1 < NC; c += 2) {
      uint32_t b[4];
      tc_ldsm4(base + k * plane + c * step, b);
      f[k][c][0] = b[0], f[k][c][1] = b[1], f[k][c + 1][0] = b[2], f[k][c + 1][1] = b[3];
    }
    if constexpr (NC & 1) tc_ldsm2(base + k * plane + (NC - 1) * step, f[k][NC - 1][0], f[k][NC - 1][1]);
  }
}
// the numbers of a pair, from its planes
template <int PL>
__device__ __forceinline__ float2 tc_value(const uint32_t (&w)[PL]) {
  float2 v = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = PL - 1; k >= 0; --k) {
    v.x += __uint_as_float(w[k] << 16);
    v.y += __uint_as_float(w[k] & 0xffff0000u);
  }
  return v;
}

// Sums of the warps that share rows: visit(f) calls f on a thread's N sums; the
// first of the warps ends with the total.  The other threads only take part.
template <int N, typename V>
__device__ __forceinline__ void tc_join(float* sm, int rw, int rws, int kw, int kws, V&& visit) {
  const int lane = threadIdx.x & 31;
  if (kw > 0) {
    float* o = sm + size_t((kw - 1) * rws + rw) * N * 32 + lane;
    visit([&](float& x) {
      *o = x;
      o += 32;
    });
  }
  __syncthreads();
  if (kw == 0)
    for (int w = 1; w < kws; ++w) {
      const float* o = sm + size_t((w - 1) * rws + rw) * N * 32 + lane;
      visit([&](float& x) {
        x += *o;
        o += 32;
      });
    }
  __syncthreads();
}
constexpr int tc_join_bytes(int n) { return 3 * n * 32 * 4; }   // at most three warps' sums

// A warp's 16 rows of values, or of queries or keys, from shared memory (rows of
// OUT elements) to global memory in 16-byte pieces: a lane keeps its piece and
// advances by whole rows.
template <int CH, int OUT, typename T, typename F>
__device__ __forceinline__ void tc_write_rows(const T* rows, T* out, size_t ld, int live, F&& offset) {
  constexpr int PER = 16 / int(sizeof(T)), ROWS = CH <= 32 ? 32 / CH : 1;
  const int lane = threadIdx.x & 31;
  for (int piece = CH <= 32 ? lane % CH : lane; piece < CH; piece += 32) {
    const int off = offset(piece * PER);
    if (off < 0) continue;
    int row = CH <= 32 ? lane / CH : 0;
    if (row >= ROWS) continue;
    const T* from = rows + row * OUT + piece * PER;
    T* to = out + row * ld + off;
    for (; row < live; row += ROWS, from += ROWS * OUT, to += ROWS * ld)
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
  }
}
template <int NT, int HP, int OUT, typename T>
__device__ __forceinline__ void tc_write_vals(const MolParams& p, const T* rows, void* out, int head0, size_t row0, int live) {
  const size_t ld = p.D * p.C;
  tc_write_rows<HP * NT * 8 * int(sizeof(T)) / 16, OUT>(rows, static_cast<T*>(out) + row0 * ld, ld, live, [&](int e) {
    const int c = e >> 3;
    return tc_val_off(p, head0 + c % HP, c / HP) + (e & 7);
  });
}
template <int KC, int HP, int OUT, typename T>
__device__ __forceinline__ void tc_write_qk(const MolParams& p, const T* rows, void* out, int head0, size_t row0, int live) {
  const size_t ld = p.H * p.dk;
  tc_write_rows<HP * KC * 8 * int(sizeof(T)) / 16, OUT>(rows, static_cast<T*>(out) + row0 * ld, ld, live, [&](int e) {
    const int h = e / (KC * 8), d = e % (KC * 8);
    return d < p.dk ? (head0 + h) * p.dk + d : -1;
  });
}

// acc (16 rows x 16 other rows) = (or, with ADD, +=) A (16 rows x NC chunks) . (other rows)^T:
// base is the lane's address of chunk 0 for a non-transposed x4 load (rows by
// lane & 7 and lane / 16, chunk by bit 3), base2 that of an x2 load of a last odd
// chunk; step and plane: bytes from a chunk, a plane to the next.
template <int NC, int PL, bool ADD = false>
__device__ __forceinline__ void tc_dot(float (&acc)[2][4], const uint32_t (&a)[PL][NC][2], uint32_t base, uint32_t base2,
                                       int step, int plane) {
  if constexpr (NC == 1 && !ADD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] = 0.f;
  }
  // small products first: a tensor-core sum drops bits below its largest term
#pragma unroll
  for (int q = PL - 1; q >= 0; --q) {
#pragma unroll
    for (int c = 0; c + 1 < NC; c += 2) {
      uint32_t b[4];
      tc_ldsm4(base + q * plane + c * step, b);
#pragma unroll
      for (int k = PL - 1 - q; k >= 0; --k) {
        if (c == 0 && q == PL - 1 && !ADD) {
          tc_mma16_first(acc[0], a[k][c], a[k][c + 1], b[0], b[1]);
          tc_mma16_first(acc[1], a[k][c], a[k][c + 1], b[2], b[3]);
        } else {
          tc_mma16(acc[0], a[k][c], a[k][c + 1], b[0], b[1]);
          tc_mma16(acc[1], a[k][c], a[k][c + 1], b[2], b[3]);
        }
      }
    }
    if constexpr (NC & 1) {
      uint32_t b0, b1;
      tc_ldsm2(base2 + q * plane + (NC - 1) * step, b0, b1);
#pragma unroll
      for (int k = PL - 1 - q; k >= 0; --k) {
        tc_mma8(acc[0], a[k][NC - 1], b0);
        tc_mma8(acc[1], a[k][NC - 1], b1);
      }
    }
  }
}
// acc[NC chunks of columns] += w (16 rows x 16 other rows) . other rows; base is
// the lane's address of chunk 0 for a transposed x4 load (row by lane & 15,
// chunk by lane / 16).  PW planes of w; of the rows as many for float32, one for bf16.
// For float32 a step's products are summed apart, small ones first, and added to
// the accumulator by the FMA pipe, which rounds where the tensor core truncates:
// the many steps of a long molecule added up to 2e-6 of the result otherwise.
template <int NC, int PW>
__device__ __forceinline__ void tc_apply(float (&acc)[NC][4], const uint32_t (&w)[PW][2][2], uint32_t base, int step,
                                         int plane) {
  if constexpr (PW < 3) {
#pragma unroll
    for (int c = 0; c + 1 < NC; c += 2) {
      uint32_t b[4];
      tc_ldsm4t(base + c * step, b);
#pragma unroll
      for (int k = PW - 1; k >= 0; --k) {
        tc_mma16(acc[c], w[k][0], w[k][1], b[0], b[1]);
        tc_mma16(acc[c + 1], w[k][0], w[k][1], b[2], b[3]);
      }
    }
    if constexpr (NC & 1) {
      uint32_t b0, b1;
      tc_ldsm2t(base + (NC - 1) * step, b0, b1);
#pragma unroll
      for (int k = PW - 1; k >= 0; --k) tc_mma16(acc[NC - 1], w[k][0], w[k][1], b0, b1);
    }
  } else {
#pragma unroll
    for (int c = 0; c + 1 < NC; c += 2) {
      float t[2][4];
#pragma unroll
      for (int q = 2; q >= 0; --q) {
        uint32_t b[4];
        tc_ldsm4t(base + q * plane + c * step, b);
#pragma unroll
        for (int k = 2 - q; k >= 0; --k) {
          if (q == 2) {
            tc_mma16_first(t[0], w[k][0], w[k][1], b[0], b[1]);
            tc_mma16_first(t[1], w[k][0], w[k][1], b[2], b[3]);
          } else {
            tc_mma16(t[0], w[k][0], w[k][1], b[0], b[1]);
            tc_mma16(t[1], w[k][0], w[k][1], b[2], b[3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[c + (i >> 2)][i & 3] += t[i >> 2][i & 3];
    }
    if constexpr (NC & 1) {
      float t[4];
#pragma unroll
      for (int q = 2; q >= 0; --q) {
        uint32_t b0, b1;
        tc_ldsm2t(base + q * plane + (NC - 1) * step, b0, b1);
#pragma unroll
        for (int k = 2 - q; k >= 0; --k) {
          if (q == 2)
            tc_mma16_first(t, w[k][0], w[k][1], b0, b1);
          else
            tc_mma16(t, w[k][0], w[k][1], b0, b1);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[NC - 1][i] += t[i];
    }
  }
}
// (a, b), columns 2t and 2t + 1 of 8-row tile c and row r, into A fragments
template <int PL>
__device__ __forceinline__ void tc_put(uint32_t (&f)[PL][2][2], int c, int r, float a, float b) {
  uint32_t w[PL];
  tc_planes<PL>(a, b, w);
#pragma unroll
  for (int k = 0; k < PL; ++k) f[k][c][r] = w[k];
}
// Lane offsets of those loads inside a stage part with rows of RS bytes.
__device__ __forceinline__ uint32_t tc_lane_n(int RS, int step) {
  const int lane = threadIdx.x & 31;
  return uint32_t(((lane & 7) + (lane >> 4) * 8) * RS + ((lane >> 3) & 1) * step);
}
__device__ __forceinline__ uint32_t tc_lane_t(int RS, int step) {
  const int lane = threadIdx.x & 31;
  return uint32_t((lane & 15) * RS + (lane >> 4) * step);
}
__device__ __forceinline__ uint32_t tc_lane_n2(int RS) { return uint32_t((threadIdx.x & 15) * RS); }

// tanh on pairs for |x| <= 1: x P(x^2), P a degree-6 fit of tanh(sqrt z) / sqrt z on
// [0, 1] with relative error 1.4e-7 in float32.  On the FMA pipe: logits below
// the cap cost no special-function work.
__device__ __forceinline__ f32x2 tc_tanh_small(f32x2 x) {
  const f32x2 z = f2_mul(x, x);
  f32x2 r = f2_fma(z, f2_set(1.041022467e-03f), f2_set(-6.203378603e-03f));
  r = f2_fma(z, r, f2_set(2.028997986e-02f));
  r = f2_fma(z, r, f2_set(-5.345702927e-02f));
  r = f2_fma(z, r, f2_set(1.332520407e-01f));
  r = f2_fma(z, r, f2_set(-3.333283915e-01f));
  r = f2_fma(z, r, f2_set(9.999999502e-01f));
  return f2_mul(x, r);
}
// tanh of a step's logits (units of the cap) in place, and the derivative if wanted
template <int N, bool WANT>
__device__ __forceinline__ void tc_cap(f32x2 (&x)[N], f32x2 (&fx)[WANT ? N : 1]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a, b;
    f2_unpack(x[i], a, b);
    top = tc_max3(top, fabsf(a), fabsf(b));
  }
  if (__builtin_expect(top > 1.f, 0)) {   // a NaN logit stays NaN either way
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float a, b, da, db;
      f2_unpack(x[i], a, b);
      a = mol_tanh(a, da);
      b = mol_tanh(b, db);
      x[i] = f2_pack(a, b);
      if (WANT) fx[i] = f2_pack(da, db);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = tc_tanh_small(x[i]);
    if (WANT) fx[i] = f2_fma(f2_mul(x[i], f2_set(-1.f)), x[i], f2_set(1.f));
  }
}

// Two distances from their squares and, with RECIP, their reciprocals (any finite
// number at distance zero, where the direction is zero).
template <bool RECIP>
__device__ __forceinline__ void tc_dist(float a, float b, f32x2& d, f32x2& ri) {
  if (!RECIP) {
    d = f2_pack(mol_sqrt(a), mol_sqrt(b));
    return;
  }
  float ra, rb;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(fminf(fmaxf(a, 1e-37f), 3.4e38f)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(fminf(fmaxf(b, 1e-37f), 3.4e38f)));
  ri = f2_pack(ra, rb);
  d = f2_mul(f2_pack(a, b), ri);   // NaN and inf of the squares stay
}

// Distances of this lane's two rows (px.. = minus their positions) to the keys
// 2t, 2t + 1 of both 8-key tiles at sp: [tile][row], and with RECIP their reciprocals
template <bool RECIP>
__device__ __forceinline__ void tc_dists(const float* sp, const f32x2 (&px)[2], const f32x2 (&py)[2],
                                         const f32x2 (&pz)[2], f32x2 (&d)[2][2], f32x2 (&ri)[2][2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const f32x2* at = reinterpret_cast<const f32x2*>(sp + 8 * c);
    const f32x2 x = at[0], y = at[kTcStage / 2], z = at[kTcStage];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const f32x2 dx = f2_add(x, px[r]), dy = f2_add(y, py[r]), dz = f2_add(z, pz[r]);
      float a, b;
      f2_unpack(f2_fma(dx, dx, f2_fma(dy, dy, f2_mul(dz, dz))), a, b);
      tc_dist<RECIP>(a, b, d[c][r], ri[c][r]);
    }
  }
}

// Whether any distance of a warp's step is infinite
__device__ __forceinline__ bool tc_far(const f32x2 (&d)[2][2]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_unpack(d[i >> 1][i & 1], a, b);
    top = tc_max3(top, a, b);
  }
  return __any_sync(~0u, top == INFINITY);
}
// g += f (r_j - r_i) by component; FAR: a direction may be infinite, where f is zero
template <bool FAR>
__device__ __forceinline__ void tc_pull(const f32x2* at, f32x2 px, f32x2 py, f32x2 pz, f32x2 f, f32x2 (&g)[3]) {
  f32x2 v[3] = {f2_add(at[0], px), f2_add(at[kTcStage / 2], py), f2_add(at[kTcStage], pz)};
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    if (FAR) {
      float a, b;
      f2_unpack(v[e], a, b);
      v[e] = f2_pack(mol_finite(a), mol_finite(b));
    }
    g[e] = f2_fma(f, v[e], g[e]);
  }
}
// ... by a flag that is the same for the whole warp and nearly always false
__device__ __forceinline__ void tc_pull(bool far, const f32x2* at, f32x2 px, f32x2 py, f32x2 pz, f32x2 f, f32x2 (&g)[3]) {
  if (__builtin_expect(far, 0))
    tc_pull<true>(at, px, py, pz, f, g);
  else
    tc_pull<false>(at, px, py, pz, f, g);
}

// Calls f with the value tiles, the query chunks and the heads of a warp: two for up
// to 64 value columns, HP9 for 72, and one where the registers would not hold two.
template <int PL, int HP9, typename F>
int tc_dispatch(int nt, int dk, F&& f) {
#define EGAT_TC(N_, HP_)                                                                                   \
  case N_:                                                                                                 \
    if (dk <= 16) return f(std::integral_constant<int, N_>{}, std::integral_constant<int, 2>{},            \
                           std::integral_constant<int, PL == 1 ? HP_ : 1>{});                              \
    return f(std::integral_constant<int, N_>{}, std::integral_constant<int, 4>{},                          \
             std::integral_constant<int, PL == 1 ? HP_ : 1>{})
  switch (nt) {
    EGAT_TC(1, 2);
    EGAT_TC(2, 2);
    EGAT_TC(4, 2);
    EGAT_TC(8, 2);
    EGAT_TC(9, HP9);
    EGAT_TC(16, 1);
    EGAT_TC(18, 1);
    case 32:
      if constexpr (PL == 1) {
        if (dk <= 16) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
        return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
      }
      return EGAT_ERR_UNSUPPORTED;
    default: return EGAT_ERR_UNSUPPORTED;
  }
#undef EGAT_TC
}

// ... and f with two flags
template <typename F>
int mol_flags(bool a, bool b, F&& f) {
  if (a) return b ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  return b ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

template <typename K>
int tc_launch(K* kernel, dim3 grid, size_t shm, const MolParams& p, cudaStream_t st) {
  return mol_launch(kernel, grid, kTcThreads, shm, p, st);
}

}  // namespace
}  // namespace egat
