// Building blocks of the tcgen05 kernels of the attention within molecules:
// operands laid out by head, descriptors, tensor-memory access.
//
// The products read their operands from shared memory as 16-byte chunks (8
// columns of one row), consecutive rows 16 bytes apart: with rows as the
// contraction's outer index that is the canonical K-major layout without
// swizzle, and with rows as the contraction index the canonical MN-major one,
// so one staged copy of a tensor serves both kinds of product.  A packing kernel
// lays the operands out as whole stages by head and tile, once a call: a stage is
// then one contiguous bulk copy (one copy per chunk, 18 at lmax 3, took the issuing
// thread 2,500 cycles a stage, twice the exponentials), and every 32-byte sector
// is used whole, where a head's chunk alone is half a sector of an atom's row.
#pragma once

#include "egat_async.cuh"
#include "molecule_tc.cuh"

namespace egat {
namespace {

constexpr int kUmRowsLog = 7, kUmRows = 128;   // rows of a tile (lanes of tensor memory)
constexpr int kUmStage = 64;                   // rows of the other side of a stage

// Shared-memory matrix descriptor without swizzle (leading and stride byte offsets).
__device__ __forceinline__ uint64_t um_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46);
}
// Rows of R-row chunks as K-major operand: 8-row groups 128 bytes apart, the two
// chunks of a k-step R * 16 bytes apart.
template <int R>
__device__ __forceinline__ uint64_t um_k_major(uint32_t saddr) { return um_desc(saddr, R * 16, 128); }
// The same rows as the contraction index (16 from the start on): 8-row groups 128
// bytes apart, column chunks R * 16 bytes apart.
template <int R>
__device__ __forceinline__ uint64_t um_mn_major(uint32_t saddr) { return um_desc(saddr, 128, R * 16); }

// Instruction descriptor, kind::f16: float32 accumulator, bf16 operands, M = 128
constexpr uint32_t um_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
         (uint32_t(kUmRows >> 4) << 24);
}
__device__ __forceinline__ void um_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(uint32_t(add))
      : "memory");
}
// A from tensor memory
__device__ __forceinline__ void um_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void um_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void um_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void um_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void um_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
#define EGAT_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define EGAT_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// Consecutive 32-bit columns of this thread's lane; the wait is part of the load,
// so that nothing can read them early.
__device__ __forceinline__ void um_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : EGAT_R8(r, 0), EGAT_R8(r, 8), EGAT_R8(r, 16), EGAT_R8(r, 24)
      : "r"(t) : "memory");
}
__device__ __forceinline__ void um_ld8(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : EGAT_R8(r, 0) : "r"(t) : "memory");
}
__device__ __forceinline__ void um_st8(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::EGAT_I8(r, 0), "r"(t)
               : "memory");
}
__device__ __forceinline__ void um_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};\n" ::EGAT_I8(r, 0), EGAT_I8(r, 8), "r"(t)
      : "memory");
}
#undef EGAT_R8
#undef EGAT_I8
// A whole warp's wait: its lanes leave together, as the tensor-memory accesses
// that follow need them.
__device__ __forceinline__ bool um_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(~0u, bounded_wait(bar, parity, kWaitPolls, abort_flag));
}
template <int COLS>
__device__ __forceinline__ void um_alloc(uint32_t slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot), "r"(COLS) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void um_dealloc(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(COLS) : "memory");
}

// The end of a CTA.  A wait that gave up left copies or products in flight; behind the
// barrier every role is past its last wait, so the flag no longer changes, and the threads
// that issued them (lane 0 of two warps; `land` waits for the copies) see them land before
// shared and tensor memory are given up.  `issuer` is the warp that allocated.
template <int COLS, typename F>
__device__ __forceinline__ void um_release(volatile int* abort_flag, int copier, int issuer, uint32_t drained, uint32_t tmem,
                                           F&& land) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  um_before();
  __syncthreads();
  if (*abort_flag) {
    volatile int none = 0;
    if (warp == copier && lane == 0) {
      land(&none);
    } else if (warp == issuer && lane == 0) {
      um_commit(drained);
      bounded_wait(drained, 0, kDrainPolls, &none);
    }
    __syncthreads();
  }
  if (warp == issuer) {
    um_after();
    um_dealloc<COLS>(tmem);
  }
}

}  // namespace
}  // namespace egat
