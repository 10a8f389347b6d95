// Shared by the kernels of the attention within each molecule: the rows of a
// batch cut into tiles that never cross a molecule, the score functions, and
// the launch parameters.
#pragma once

#include "egat_device.cuh"
#include "egat_host.h"

namespace egat {

struct MolParams {
  MolArgs a;
  MolGrads g;
  void* m;
  float* lse;
  float* part_o;       // [splits][nq][H][dv] unnormalised sums of a key split
  float* part_ml;      // [splits][nq][H][2] its maximum (base 2) and normaliser
  float* delta;        // [nq][H] sum_j a_ij dP_ij (minus that on the tensor-core path)
  float* nlse2;        // [nq][H] minus lse in base 2, -inf for rows without weights (tensor-core path)
  float* part_dq;      // [groups][nq][3] dL/dr of the query atoms, by group of heads
  float* part_dk;      // [groups_k][nk][3] dL/dr of the key atoms
  float* part_ds;      // [H][slots] dL/dslope, by query tile
  void *qp, *kv;       // operand blocks of the tcgen05 kernels
  int kv_slots;        // key blocks of a head
  int nq, nk, nmol, D, C, H, dk;
  int ch;              // channels of a head, C / H
  int ch8log;          // log2(ch / 8)
  int dv;              // value columns of a head, D * ch
  int splits;          // key splits (grid z)
  int slots;           // query tile slots
  int kb;              // keys per staged tile (generic kernels)
  int rwlog;           // log2 of the warps side by side over rows (tensor-core kernels)
  int groups, groups_k;   // groups of heads with position sums of their own, by side
  float scale;         // 1 / sqrt(dk)
  float cap, inv_cap;  // 0: none
  bool exact_delta;    // delta from a float32 sweep instead of G . m
  bool want_pos;       // any of dL/dr, dL/dslope
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- rows of a batch in tiles of at most M rows of one molecule
//
// With a run of rows in front of the first molecule and one behind the last
// (rows of no molecule, which have no keys), segment b starts at row P(b),
// P(0) = 0, and takes the tile slots from P(b) / M + b on: since
// ceil(n / M) <= (P + n) / M - P / M + 1, slots of different segments never
// meet, n / M + segments of them suffice, and a slot's segment is found by
// bisection over P(b) / M + b.  So tiles need no table, no extra launch and
// no lengths on the host.
__host__ __device__ inline int mol_slots(int n, int nmol, int M) { return n / M + nmol + 2; }

__device__ __forceinline__ int mol_clamp(int x, int n) { return min(max(x, 0), n); }
// first row of segment b, 0 <= b <= nmol + 2 (segment b is molecule b - 1)
__device__ __forceinline__ int mol_start(const int32_t* ptr, int nmol, int n, int b) {
  if (b == 0) return 0;
  return b == nmol + 2 ? n : mol_clamp(__ldg(ptr + b - 1), n);
}

struct MolTile {
  int row0, rows;    // own rows; rows <= 0: nothing to do
  int o0, o1;        // rows of the other side it meets
  int seg;           // its segment
};
// The tile of a slot (M = 2^mlog); called by whole warps (32-way bisection).
__device__ __forceinline__ MolTile mol_tile(int mlog, const int32_t* ptr, const int32_t* optr, int nmol,
                                            int n, int on, int slot) {
  const int M = 1 << mlog;
  const int lane = threadIdx.x & 31;
  int lo = 0, len = nmol + 2;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int b = lo + lane * step;
    const bool in = lane * step < len && (lane == 0 || (mol_start(ptr, nmol, n, b) >> mlog) + b <= slot);
    const int c = 31 - __clz(int(__ballot_sync(~0u, in)));   // lane 0 is always in
    lo += c * step;
    len = min(step, len - c * step);
  }
  MolTile t;
  const int s = mol_start(ptr, nmol, n, lo), e = mol_start(ptr, nmol, n, lo + 1);
  // pointers that descend give a segment more slots than it has rows: those stay empty
  const int off = slot - ((s >> mlog) + lo);
  const bool some = e > s && off <= ((e - s) >> mlog);
  t.row0 = some ? s + (off << mlog) : 0;
  t.rows = some ? min(M, e - t.row0) : 0;
  t.seg = lo;
  const bool mol = lo > 0 && lo <= nmol;
  t.o0 = mol ? mol_start(optr, nmol, on, lo) : 0;
  t.o1 = mol ? max(t.o0, mol_start(optr, nmol, on, lo + 1)) : 0;
  return t;
}

// tanh(x) and its derivative.  With u = 1 / (exp(2|x|) + 1), tanh is 1 - 2u
// with x's sign, whose absolute error is near one rounding of 1, and below
// 0.3, where that would be a large share of x, the first five terms of the
// Taylor series (the sixth is below 2^-24 there).  So cap tanh(x / cap) is
// right to a few roundings of itself for every cap.  1 - tanh^2 = 4 u (1 - u)
// keeps its relative accuracy where tanh saturates.  No overflow: u is 0 there.
__device__ __forceinline__ float mol_tanh(float x, float& slope) {
  const float u = __fdividef(1.f, fast_exp2(fabsf(x) * (2.f * kLog2e)) + 1.f);
  slope = 4.f * u * (1.f - u);
  const float y = x * x;
  float r = fmaf(y, 62.f / 2835.f, -17.f / 315.f);
  r = fmaf(y, r, 2.f / 15.f);
  r = fmaf(y, r, -1.f / 3.f);
  return fabsf(x) < 0.3f ? fmaf(x * y, r, x) : copysignf(fmaf(-2.f, u, 1.f), x);
}
// squares below 2^-126 count as zero
__device__ __forceinline__ float mol_sqrt(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// An infinite distance masks its pair, whose position gradient is then zero times
// the direction: a direction of infinite components would make that NaN.
__device__ __forceinline__ float mol_finite(float x) { return copysignf(fminf(fabsf(x), 3.4e38f), x); }

// Tensor-core kernels in tiles of 16 << p.rwlog rows: whether they take the shape,
// the heads that a warp takes together, and their launches.
bool mol_tc_supported(const egat_mol_shape& s);
int mol_tc_heads(const egat_mol_shape& s, bool query_gradients);
int mol_tc_forward_bf16(const MolParams& p, cudaStream_t st);
int mol_tc_forward_f32(const MolParams& p, cudaStream_t st);
int mol_tc_backward_q_bf16(const MolParams& p, cudaStream_t st);
int mol_tc_backward_q_f32(const MolParams& p, cudaStream_t st);
int mol_tc_backward_k_bf16(const MolParams& p, cudaStream_t st);
int mol_tc_backward_k_f32(const MolParams& p, cudaStream_t st);
// tcgen05 kernels: whether they take the shape, the sizes of the operand blocks
// and their packing, and the forward pass in tiles of 128 rows.
bool mol_umma_supported(const egat_mol_shape& s);
size_t mol_umma_key_bytes(const egat_mol_shape& s);
size_t mol_umma_query_bytes(const egat_mol_shape& s);
int mol_umma_pack(const MolParams& p, cudaStream_t st);
int mol_umma_forward(const MolParams& p, cudaStream_t st);

template <typename K>
int mol_launch(K* kernel, dim3 grid, int threads, size_t shm, const MolParams& p, cudaStream_t st) {
  if (shm > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shm)) != cudaSuccess)
    return EGAT_ERR_CUDA;
  kernel<<<grid, threads, shm, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA;
}
}  // namespace egat
