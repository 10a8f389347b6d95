// Building blocks of the tensor-core kernels of the attention within
// molecules (bf16 storage).
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
#pragma once

#include "molecule.cuh"

namespace egat {
namespace {

constexpr int kTcThreads = 128;
constexpr int kTcStage = 64;   // rows of a stage

template <int NT, int KC, int HP>
struct TcLay {
  static constexpr int RK = ((HP * KC) | 1) * 16;    // bytes of a staged query/key row
  static constexpr int RV = ((HP * NT) | 1) * 16;    // bytes of a staged value row
  static constexpr int QK = 0;
  static constexpr int VAL = QK + kTcStage * RK;
  static constexpr int POS = VAL + kTcStage * RV;    // x[64], y[64], z[64]
  static constexpr int ROW = POS + kTcStage * 12;    // per head: lse2[64], delta[64]
  static constexpr int STAGE = ROW + HP * kTcStage * 8;
  static constexpr int OUTROW = HP * NT * 8 + 8;     // floats of a joined row (bank spread)
};

__device__ __forceinline__ uint32_t tc_smem(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void tc_cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tc_cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
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
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
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

// Rows [r0, r0 + 64) of heads head0.. into a stage; rows from `end` on as zeros.
template <int NT, int KC, int HP>
__device__ __forceinline__ void tc_load_stage(const MolParams& p, const __nv_bfloat16* qk, const __nv_bfloat16* val,
                                              const float* pos, int head0, int r0, int end, uint32_t st) {
  using L = TcLay<NT, KC, HP>;
  const int kc = p.dk >> 3;   // below KC at dk 8: the second chunk is zeros
#pragma unroll
  for (int i = threadIdx.x; i < kTcStage * HP * KC; i += kTcThreads) {
    const int r = i / (HP * KC), c = i % (HP * KC), hp = c / KC, cc = c % KC;
    const bool ok = r0 + r < end && cc < kc;
    tc_cp16(st + L::QK + r * L::RK + c * 16,
            ok ? qk + (size_t(r0 + r) * p.H + head0 + hp) * p.dk + cc * 8 : qk, ok);
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < kTcStage * HP * NT; i += kTcThreads) {
    const int r = i / (HP * NT), c = i % (HP * NT), x = c / HP, hp = c % HP;
    const bool ok = r0 + r < end;
    tc_cp16(st + L::VAL + r * L::RV + c * 16,
            ok ? val + size_t(r0 + r) * (p.D * p.C) + tc_val_off(p, head0 + hp, x) : val, ok);
  }
  if (p.a.slope)
    for (int i = threadIdx.x; i < 3 * kTcStage; i += kTcThreads) {
      const int r = i / 3, c = i % 3;
      const bool ok = r0 + r < end;
      tc_cp4(st + L::POS + c * (kTcStage * 4) + r * 4, ok ? pos + size_t(r0) * 3 + i : pos, ok);
    }
}

// A fragments of this lane's rows (r0 = row g, r1 = row g + 8) from global memory
template <int KC>
__device__ __forceinline__ void tc_frag_qk(const MolParams& p, const __nv_bfloat16* x, size_t r0, size_t r1, bool l0,
                                           bool l1, int head, uint32_t (&f)[KC][2]) {
  const int kc = p.dk >> 3, t2 = (threadIdx.x & 3) * 2;
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    f[c][0] = l0 && c < kc ? __ldg(reinterpret_cast<const uint32_t*>(x + (r0 * p.H + head) * p.dk + c * 8 + t2)) : 0u;
    f[c][1] = l1 && c < kc ? __ldg(reinterpret_cast<const uint32_t*>(x + (r1 * p.H + head) * p.dk + c * 8 + t2)) : 0u;
  }
}
template <int NT>
__device__ __forceinline__ void tc_frag_val(const MolParams& p, const __nv_bfloat16* x, size_t r0, size_t r1, bool l0,
                                            bool l1, int head, uint32_t (&f)[NT][2]) {
  const int t2 = (threadIdx.x & 3) * 2;
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int o = tc_val_off(p, head, c) + t2;
    f[c][0] = l0 ? __ldg(reinterpret_cast<const uint32_t*>(x + r0 * (p.D * p.C) + o)) : 0u;
    f[c][1] = l1 ? __ldg(reinterpret_cast<const uint32_t*>(x + r1 * (p.D * p.C) + o)) : 0u;
  }
}

// acc[16 rows x 16 other rows] = A (16 rows x NC chunks) . (other rows)^T:
// base is the lane's address of chunk 0 for a non-transposed x4 load (rows by
// lane & 7 and lane / 16, chunk by bit 3), base2 that of an x2 load of a last odd
// chunk; step: bytes from a chunk to the next.
template <int NC>
__device__ __forceinline__ void tc_dot(float (&acc)[2][4], const uint32_t (&a)[NC][2], uint32_t base, uint32_t base2,
                                       int step) {
#pragma unroll
  for (int c = 0; c + 1 < NC; c += 2) {
    uint32_t b[4];
    tc_ldsm4(base + c * step, b);
    tc_mma16(acc[0], a[c], a[c + 1], b[0], b[1]);
    tc_mma16(acc[1], a[c], a[c + 1], b[2], b[3]);
  }
  if constexpr (NC & 1) {
    uint32_t b0, b1;
    tc_ldsm2(base2 + (NC - 1) * step, b0, b1);
    tc_mma8(acc[0], a[NC - 1], b0);
    tc_mma8(acc[1], a[NC - 1], b1);
  }
}
// acc[NC chunks of columns] += w (16 rows x 16 other rows) . other rows; base is
// the lane's address of chunk 0 for a transposed x4 load (row by lane & 15,
// chunk by lane / 16).
template <int NC>
__device__ __forceinline__ void tc_apply(float (&acc)[NC][4], const uint32_t (&w)[2][2], uint32_t base, int step) {
#pragma unroll
  for (int c = 0; c + 1 < NC; c += 2) {
    uint32_t b[4];
    tc_ldsm4t(base + c * step, b);
    tc_mma16(acc[c], w[0], w[1], b[0], b[1]);
    tc_mma16(acc[c + 1], w[0], w[1], b[2], b[3]);
  }
  if constexpr (NC & 1) {
    uint32_t b0, b1;
    tc_ldsm2t(base + (NC - 1) * step, b0, b1);
    tc_mma16(acc[NC - 1], w[0], w[1], b0, b1);
  }
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
// x = cap tanh of 4 logits (an accumulator fragment), in units of 1 / cap, and f' if wanted
template <bool WANT>
__device__ __forceinline__ void tc_cap(f32x2& a, f32x2& b, f32x2& fa, f32x2& fb) {
  float v[4];
  f2_unpack(a, v[0], v[1]);
  f2_unpack(b, v[2], v[3]);
  const float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
  if (!(top <= 1.f)) {
    float d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mol_tanh(v[i], d[i]);
    a = f2_pack(v[0], v[1]);
    b = f2_pack(v[2], v[3]);
    if (WANT) {
      fa = f2_pack(d[0], d[1]);
      fb = f2_pack(d[2], d[3]);
    }
    return;
  }
  a = tc_tanh_small(a);
  b = tc_tanh_small(b);
  if (WANT) {
    const f32x2 one = f2_set(1.f);
    fa = f2_fma(f2_mul(a, f2_set(-1.f)), a, one);
    fb = f2_fma(f2_mul(b, f2_set(-1.f)), b, one);
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
  const float ra = rsqrtf(fminf(fmaxf(a, 1e-37f), 3.4e38f)), rb = rsqrtf(fminf(fmaxf(b, 1e-37f), 3.4e38f));
  ri = f2_pack(ra, rb);
  d = f2_mul(f2_pack(a, b), ri);   // NaN and inf of the squares stay
}

// Calls f with the value tiles, the query chunks and the heads of a warp.
template <typename F>
int tc_dispatch(int nt, int dk, F&& f) {
#define EGAT_TC(N_, HP_)                                                                                   \
  case N_:                                                                                                 \
    if (dk <= 16) return f(std::integral_constant<int, N_>{}, std::integral_constant<int, 2>{},            \
                           std::integral_constant<int, HP_>{});                                            \
    return f(std::integral_constant<int, N_>{}, std::integral_constant<int, 4>{},                          \
             std::integral_constant<int, HP_>{})
  switch (nt) {
    EGAT_TC(1, 2);
    EGAT_TC(2, 2);
    EGAT_TC(4, 2);
    EGAT_TC(8, 2);
    EGAT_TC(9, 2);
    EGAT_TC(16, 1);
    EGAT_TC(18, 1);
    EGAT_TC(32, 1);
    default: return EGAT_ERR_UNSUPPORTED;
  }
#undef EGAT_TC
}

template <typename K>
int tc_launch(K* kernel, dim3 grid, size_t shm, const MolParams& p, cudaStream_t st) {
  if (shm > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shm)) != cudaSuccess)
    return EGAT_ERR_CUDA;
  kernel<<<grid, kTcThreads, shm, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA;
}

}  // namespace
}  // namespace egat
