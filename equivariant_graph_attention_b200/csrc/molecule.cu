// Attention within each molecule, forward and backward: the host side (which
// kernels a shape takes, tiles, key splits, workspaces), the join of key splits,
// the position and slope sums, and the kernels on the FMA pipe in float32 for the
// shapes that the tensor-core kernels leave (more than 256 value columns a head of
// bf16, 144 of float32; one head of bf16 with few columns).
//
//   x_ij = q_i.k_j / sqrt(dk),  s_ij = f(x_ij) - slope |r_i - r_j|,
//   f(x) = x or cap tanh(x / cap),  m_i = sum_j softmax_j(s_ij) h'_j
//
// In the FMA kernels the rows of one head are taken in tiles of one molecule
// (molecule.cuh); a group of LP lanes holds a row: its query, its accumulators and,
// backward, its gradient, split over the lanes in float4 vectors.  Key (or, for
// the gradients of the keys, query) rows pass through shared memory as float32 and
// are read by broadcast, so a warp's read serves 32 / LP rows.  The softmax runs
// online with base-2 exponents: one running maximum and sum per row, rescaled only
// when the maximum grows.  They are bound by shared-memory reads: a 16-byte read
// feeds four products, a quarter of what the FMA pipe could take.
#include <cmath>

#include "molecule.cuh"

namespace egat {
namespace {

constexpr int kMolThreads = 128;
constexpr int kMolWarps = kMolThreads / 32;
constexpr int kMolBatch = 4;   // keys taken together by the online softmax

template <int NV, int LP>
struct MolRows {
  static constexpr int WLOG = LP == 1 ? 5 : LP == 2 ? 4 : LP == 4 ? 3 : LP == 8 ? 2 : LP == 16 ? 1 : 0;
  static constexpr int W = 1 << WLOG;                // rows of a warp (of one row a lane group)
  static constexpr int DV = 4 * NV * LP;             // value columns
};

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void axpy4(float s, float4 b, float4& c) {
  c.x = fmaf(s, b.x, c.x);
  c.y = fmaf(s, b.y, c.y);
  c.z = fmaf(s, b.z, c.z);
  c.w = fmaf(s, b.w, c.w);
}
__device__ __forceinline__ void scale4(float s, float4& c) {
  c.x *= s;
  c.y *= s;
  c.z *= s;
  c.w *= s;
}
template <int LP>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// offset of value vector x (4 columns) of a head inside a row of [D][C]
__device__ __forceinline__ int val_off(const MolParams& p, int head, int x) {
  const int vlog = p.ch8log + 1;   // vectors of a head's channels: ch / 4
  return (x >> vlog) * p.C + head * p.ch + ((x & ((1 << vlog) - 1)) << 2);
}

// A tile of `kb` rows [r0, end) of one head into shared memory as float32:
// the query/key part, the value part and the positions.  Rows from `end` on
// are zeros, so nothing of another molecule enters a product.
template <int DV, typename T>
__device__ __forceinline__ void stage_rows(const MolParams& p, int head, const T* qk, const T* val,
                                           const float* pos, int r0, int end, float* sk, float* sv,
                                           float* sp) {
  const int kvlog = p.dk == 8 ? 1 : p.dk == 16 ? 2 : 3;   // vectors of a query or key
  for (int i = threadIdx.x; i < p.kb << kvlog; i += kMolThreads) {
    const int r = i >> kvlog, x = i & ((1 << kvlog) - 1);
    const bool in = r0 + r < end;
    const float4 v = in ? load4(qk + (size_t(r0 + r) * p.H + head) * p.dk + 4 * x)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(sk + r * p.dk + 4 * x) = v;
  }
  for (int i = threadIdx.x; i < p.kb * (DV / 4); i += kMolThreads) {
    const int r = i / (DV / 4), x = i - r * (DV / 4);
    const bool in = r0 + r < end;
    const float4 v = in ? load4(val + size_t(r0 + r) * p.D * p.C + val_off(p, head, x))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(sv + r * DV + 4 * x) = v;
  }
  if (p.a.slope)
    for (int i = threadIdx.x; i < p.kb; i += kMolThreads) {
      const bool in = r0 + i < end;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        const float* r = pos + size_t(r0 + i) * 3;
        v = make_float4(r[0], r[1], r[2], 0.f);
      }
      *reinterpret_cast<float4*>(sp + 4 * i) = v;
    }
}

// ---- forward

template <int NV, int LP, int KV, typename T>
__global__ void __launch_bounds__(kMolThreads) mol_fwd_kernel(MolParams p) {
  using G = MolRows<NV, LP>;
  extern __shared__ __align__(16) float msm[];
  float* sk = msm;
  float* sv = sk + p.kb * p.dk;
  float* sp = sv + p.kb * G::DV;
  const int head = blockIdx.y, lane = threadIdx.x & 31, l = lane & (LP - 1), warp = threadIdx.x >> 5;
  const int rws = 1 << p.rwlog, kws = kMolWarps >> p.rwlog, rw = warp & (rws - 1), kw = warp >> p.rwlog;
  const MolTile t = mol_tile(G::WLOG + p.rwlog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) return;
  const int own = rw * G::W + lane / LP;
  const bool live = own < t.rows;
  const bool warp_live = rw * G::W < t.rows;
  const size_t row = size_t(t.row0) + (live ? own : 0);
  const int kv = p.dk / 4;
  float4 q[KV];
#pragma unroll
  for (int i = 0; i < KV; ++i) {
    const int x = l + LP * i;
    q[i] = x < kv ? load4(static_cast<const T*>(p.a.q) + (row * p.H + head) * p.dk + 4 * x)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float rx = 0.f, ry = 0.f, rz = 0.f, slope = 0.f;
  if (p.a.slope) {
    rx = p.a.posq[row * 3];
    ry = p.a.posq[row * 3 + 1];
    rz = p.a.posq[row * 3 + 2];
    slope = p.a.slope[head] * kLog2e;
  }
  float4 o[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float mx = -INFINITY, sum = 0.f;
  // this split's share of the molecule's key tiles
  const int tiles = (t.o1 - t.o0 + p.kb - 1) / p.kb, per = (tiles + p.splits - 1) / p.splits;
  const int k_begin = t.o0 + int(blockIdx.z) * per * p.kb;
  const int k_end = min(t.o1, k_begin + per * p.kb);
  for (int k0 = k_begin; k0 < k_end; k0 += p.kb) {
    __syncthreads();
    stage_rows<G::DV, T>(p, head, static_cast<const T*>(p.a.k), static_cast<const T*>(p.a.hp), p.a.posk,
                         k0, k_end, sk, sv, sp);
    __syncthreads();
    if (!warp_live) continue;
    const int nk = min(p.kb, k_end - k0);
    for (int j0 = kw * kMolBatch; j0 < nk; j0 += kws * kMolBatch) {
      float s[kMolBatch];
#pragma unroll
      for (int b = 0; b < kMolBatch; ++b) {
        float x = 0.f, unused;
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv)
            x = dot4(q[i], *reinterpret_cast<const float4*>(sk + (j0 + b) * p.dk + 4 * (l + LP * i)), x);
        x = group_sum<LP>(x) * p.scale;
        if (p.cap > 0.f) x = p.cap * mol_tanh(x * p.inv_cap, unused);
        x *= kLog2e;
        if (p.a.slope) {
          const float4 r = *reinterpret_cast<const float4*>(sp + 4 * (j0 + b));
          const float dx = rx - r.x, dy = ry - r.y, dz = rz - r.z;
          x -= slope * mol_sqrt(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
        }
        s[b] = j0 + b < nk ? x : -INFINITY;
      }
      const float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
      if (__any_sync(~0u, top > mx)) {
        const float up = fmaxf(mx, top);
        const float f = up == -INFINITY ? 1.f : fast_exp2(mx - up);
        mx = up;
        sum *= f;
#pragma unroll
        for (int i = 0; i < NV; ++i) scale4(f, o[i]);
      }
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int b = 0; b < kMolBatch; ++b) {
        const float w = fast_exp2(s[b] - ref);
        sum += w;
        const float* v = sv + (j0 + b) * G::DV + 4 * l;
#pragma unroll
        for (int i = 0; i < NV; ++i) axpy4(w, *reinterpret_cast<const float4*>(v + 4 * LP * i), o[i]);
      }
    }
  }
  // join the warps that shared rows: the first of them adds the others' rows
  if (kws > 1) {
    float* oj = msm;                           // [rws][W][DV]
    float* mj = msm + rws * G::W * G::DV;      // [rws][W][2]
    const int at = rw * G::W + lane / LP;
    for (int w = 1; w < kws; ++w) {
      __syncthreads();
      if (kw == w) {
        if (l == 0) mj[2 * at] = mx, mj[2 * at + 1] = sum;
#pragma unroll
        for (int i = 0; i < NV; ++i) store4(oj + at * G::DV + 4 * (l + LP * i), o[i]);
      }
      __syncthreads();
      if (kw == 0) {
        const float m1 = mj[2 * at], up = fmaxf(mx, m1), ref = up == -INFINITY ? 0.f : up;
        const float f0 = fast_exp2(mx - ref), f1 = fast_exp2(m1 - ref);
        mx = up;
        sum = fmaf(sum, f0, f1 * mj[2 * at + 1]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          scale4(f0, o[i]);
          axpy4(f1, *reinterpret_cast<const float4*>(oj + at * G::DV + 4 * (l + LP * i)), o[i]);
        }
      }
    }
  }
  if (!live || kw != 0) return;
  if (p.splits > 1) {
    const size_t at = (size_t(blockIdx.z) * p.nq + row) * p.H + head;
    if (l == 0) {
      p.part_ml[2 * at] = mx;
      p.part_ml[2 * at + 1] = sum;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) store4(p.part_o + at * p.dv + 4 * (l + LP * i), o[i]);
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (l == 0 && p.lse) p.lse[row * p.H + head] = sum == 0.f ? -INFINITY : mx * kLn2 + logf(sum);
  T* out = static_cast<T*>(p.m) + row * p.D * p.C;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    scale4(inv, o[i]);
    store4(out + val_off(p, head, l + LP * i), o[i]);
  }
}

// Joins the key splits: a block per row and head, whose warps take every fourth
// split and whose lanes take the columns; the warps' sums are joined in order.
constexpr int kJoinCols = 32;   // float4 columns at a time
template <typename T>
__global__ void __launch_bounds__(128) mol_join_kernel(MolParams p) {
  __shared__ float4 part[4][kJoinCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t rh = blockIdx.x, total = size_t(p.nq) * p.H, row = rh / p.H;
  const int head = int(rh - row * p.H);
  // maximum and normaliser of up to 64 splits: two a lane
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + rh;
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 a = lane < p.splits ? ml[lane * total] : none, b = lane + 32 < p.splits ? ml[(lane + 32) * total] : none;
  float mx = fmaxf(a.x, b.x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  const float wa = fast_exp2(a.x - ref), wb = fast_exp2(b.x - ref);
  float sum = fmaf(wa, a.y, wb * b.y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (threadIdx.x == 0 && p.lse) p.lse[rh] = sum == 0.f ? -INFINITY : mx * kLn2 + logf(sum);
  T* out = static_cast<T*>(p.m) + row * p.D * p.C;
  const int cols = p.dv / 4;
  for (int x0 = 0; x0 < cols; x0 += kJoinCols) {
    const int x = min(x0 + lane, cols - 1);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = warp; s < p.splits; s += 4) {
      const float w = __shfl_sync(~0u, s < 32 ? wa : wb, s & 31);
      axpy4(w, *reinterpret_cast<const float4*>(p.part_o + (s * total + rh) * p.dv + 4 * x), acc);
    }
    __syncthreads();
    part[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && x0 + lane < cols) {
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float4 v = part[w][lane];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      scale4(inv, acc);
      store4(out + val_off(p, head, x), acc);
    }
  }
}

// ---- backward

// The softmax weight and the score's derivative dx of one pair: x = q.k (not
// yet scaled), d = distance, lse2 = the row's log-sum-exp in base 2.
__device__ __forceinline__ float pair_weight(const MolParams& p, float x, float bias2, float lse2,
                                             float& slope_x) {
  x *= p.scale;
  slope_x = p.scale;
  if (p.cap > 0.f) {
    float d;
    x = p.cap * mol_tanh(x * p.inv_cap, d);
    slope_x *= d;
  }
  return lse2 == -INFINITY ? 0.f : fast_exp2(fmaf(x, kLog2e, -bias2) - lse2);
}

// dL/dq, the row sums delta, and the query side of dL/dr and dL/dslope.
template <int NV, int LP, int KV, typename T>
__global__ void __launch_bounds__(kMolThreads) mol_bwd_q_kernel(MolParams p) {
  using G = MolRows<NV, LP>;
  extern __shared__ __align__(16) float msm[];
  float* sk = msm;
  float* sv = sk + p.kb * p.dk;
  float* sp = sv + p.kb * G::DV;
  __shared__ float warp_ds[kMolWarps];
  const int head = blockIdx.y, lane = threadIdx.x & 31, l = lane & (LP - 1);
  const MolTile t = mol_tile(G::WLOG + p.rwlog, p.a.qptr, p.a.kptr, p.nmol, p.nq, p.nk, blockIdx.x);
  if (t.rows <= 0) {
    if (p.want_pos && threadIdx.x == 0) p.part_ds[size_t(head) * p.slots + blockIdx.x] = 0.f;
    return;
  }
  const int warp = threadIdx.x >> 5, rws = 1 << p.rwlog, kws = kMolWarps >> p.rwlog;
  const int rw = warp & (rws - 1), kw = warp >> p.rwlog;
  const int own = rw * G::W + lane / LP;
  const bool live = own < t.rows;
  const bool warp_live = rw * G::W < t.rows;
  const size_t row = size_t(t.row0) + (live ? own : 0);
  const int kv = p.dk / 4;
  float4 q[KV], dq[KV], g[NV];
  float delta = 0.f;
#pragma unroll
  for (int i = 0; i < KV; ++i) {
    const int x = l + LP * i;
    q[i] = x < kv ? load4(static_cast<const T*>(p.a.q) + (row * p.H + head) * p.dk + 4 * x)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    dq[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const size_t at = row * p.D * p.C + val_off(p, head, l + LP * i);
    g[i] = load4(static_cast<const T*>(p.g.g) + at);
    if (!p.exact_delta) delta = dot4(g[i], load4(static_cast<const T*>(p.g.m) + at), delta);
  }
  delta = group_sum<LP>(delta);
  const float lse2 = p.g.lse[row * p.H + head] * kLog2e;
  float rx = 0.f, ry = 0.f, rz = 0.f, slope = 0.f;
  if (p.a.slope) {
    rx = p.a.posq[row * 3];
    ry = p.a.posq[row * 3 + 1];
    rz = p.a.posq[row * 3 + 2];
    slope = p.a.slope[head];
  }
  float gx = 0.f, gy = 0.f, gz = 0.f, ds_sum = 0.f;
  for (int sweep = p.exact_delta ? 0 : 1; sweep < 2; ++sweep) {
    for (int k0 = t.o0; k0 < t.o1; k0 += p.kb) {
      __syncthreads();
      stage_rows<G::DV, T>(p, head, static_cast<const T*>(p.a.k), static_cast<const T*>(p.a.hp), p.a.posk,
                           k0, t.o1, sk, sv, sp);
      __syncthreads();
      if (!warp_live) continue;
      const int nk = min(p.kb, t.o1 - k0);
      for (int j = kw; j < nk; j += kws) {
        float x = 0.f, dp = 0.f;
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv)
            x = dot4(q[i], *reinterpret_cast<const float4*>(sk + j * p.dk + 4 * (l + LP * i)), x);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          dp = dot4(g[i], *reinterpret_cast<const float4*>(sv + j * G::DV + 4 * (l + LP * i)), dp);
        x = group_sum<LP>(x);
        dp = group_sum<LP>(dp);
        float d = 0.f, dx = 0.f, dy = 0.f, dz = 0.f, slope_x;
        if (p.a.slope) {
          const float4 r = *reinterpret_cast<const float4*>(sp + 4 * j);
          dx = rx - r.x, dy = ry - r.y, dz = rz - r.z;
          d = mol_sqrt(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
          if (d == INFINITY) dx = mol_finite(dx), dy = mol_finite(dy), dz = mol_finite(dz);
        }
        const float w = pair_weight(p, x, slope * kLog2e * d, lse2, slope_x);
        if (sweep == 0) {
          delta = fmaf(w, dp, delta);
          continue;
        }
        const float ds = w * (dp - delta);
        if (p.want_pos) {
          ds_sum -= ds != 0.f ? ds * d : 0.f;   // d may be inf where the weight is 0
          const float u = d > 0.f ? __fdividef(-slope * ds, d) : 0.f;
          gx = fmaf(u, dx, gx);
          gy = fmaf(u, dy, gy);
          gz = fmaf(u, dz, gz);
        }
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv)
            axpy4(ds * slope_x, *reinterpret_cast<const float4*>(sk + j * p.dk + 4 * (l + LP * i)), dq[i]);
      }
    }
    if (sweep == 0 && kws > 1) {   // the row's delta over the warps that share it
      const int at = rw * G::W + lane / LP;
      __syncthreads();
      if (l == 0) msm[kw * rws * G::W + at] = delta;
      __syncthreads();
      delta = 0.f;
      for (int w = 0; w < kws; ++w) delta += msm[w * rws * G::W + at];
      __syncthreads();
    }
  }
  if (kws > 1) {   // and its gradients
    const int at = rw * G::W + lane / LP;
    for (int w = 1; w < kws; ++w) {
      float* oj = msm + at * (p.dk + 4);
      __syncthreads();
      if (kw == w) {
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv) store4(oj + 4 * (l + LP * i), dq[i]);
        if (l == 0) store4(oj + p.dk, make_float4(gx, gy, gz, ds_sum));
      }
      __syncthreads();
      if (kw == 0) {
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv) axpy4(1.f, *reinterpret_cast<const float4*>(oj + 4 * (l + LP * i)), dq[i]);
        const float4 g = *reinterpret_cast<const float4*>(oj + p.dk);
        gx += g.x;
        gy += g.y;
        gz += g.z;
        ds_sum += g.w;
      }
    }
  }
  const bool writer = live && kw == 0;
  if (writer) {
#pragma unroll
    for (int i = 0; i < KV; ++i)
      if (l + LP * i < kv)
        store4(static_cast<T*>(p.g.dq) + (row * p.H + head) * p.dk + 4 * (l + LP * i), dq[i]);
    if (l == 0) {
      p.delta[row * p.H + head] = delta;
      if (p.want_pos) {
        float* at = p.part_dq + (size_t(head) * p.nq + row) * 3;
        at[0] = gx;
        at[1] = gy;
        at[2] = gz;
      }
    }
  }
  if (p.want_pos) {
    float v = writer && l == 0 ? ds_sum : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (lane == 0) warp_ds[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.f;
      for (int i = 0; i < kMolWarps; ++i) sum += warp_ds[i];
      p.part_ds[size_t(head) * p.slots + blockIdx.x] = sum;
    }
  }
}

// dL/dk, dL/dh' and the key side of dL/dr: a lane group owns a key row and
// meets the molecule's query rows.
template <int NV, int LP, int KV, typename T>
__global__ void __launch_bounds__(kMolThreads) mol_bwd_k_kernel(MolParams p) {
  using G = MolRows<NV, LP>;
  extern __shared__ __align__(16) float msm[];
  float* sq = msm;
  float* sg = sq + p.kb * p.dk;
  float* sp = sg + p.kb * G::DV;
  float* sl = sp + 4 * p.kb;   // lse2, delta
  const int head = blockIdx.y, lane = threadIdx.x & 31, l = lane & (LP - 1);
  const MolTile t = mol_tile(G::WLOG + p.rwlog, p.a.kptr, p.a.qptr, p.nmol, p.nk, p.nq, blockIdx.x);
  if (t.rows <= 0) return;
  const int warp = threadIdx.x >> 5, rws = 1 << p.rwlog, kws = kMolWarps >> p.rwlog;
  const int rw = warp & (rws - 1), kw = warp >> p.rwlog;
  const int own = rw * G::W + lane / LP;
  const bool live = own < t.rows;
  const bool warp_live = rw * G::W < t.rows;
  const size_t row = size_t(t.row0) + (live ? own : 0);
  const int kv = p.dk / 4;
  float4 k[KV], dk[KV], v[NV], dv[NV];
#pragma unroll
  for (int i = 0; i < KV; ++i) {
    const int x = l + LP * i;
    k[i] = x < kv ? load4(static_cast<const T*>(p.a.k) + (row * p.H + head) * p.dk + 4 * x)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    dk[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = load4(static_cast<const T*>(p.a.hp) + row * p.D * p.C + val_off(p, head, l + LP * i));
    dv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float rx = 0.f, ry = 0.f, rz = 0.f, slope = 0.f;
  if (p.a.slope) {
    rx = p.a.posk[row * 3];
    ry = p.a.posk[row * 3 + 1];
    rz = p.a.posk[row * 3 + 2];
    slope = p.a.slope[head];
  }
  float gx = 0.f, gy = 0.f, gz = 0.f;
  for (int q0 = t.o0; q0 < t.o1; q0 += p.kb) {
    __syncthreads();
    stage_rows<G::DV, T>(p, head, static_cast<const T*>(p.a.q), static_cast<const T*>(p.g.g), p.a.posq, q0,
                         t.o1, sq, sg, sp);
    for (int i = threadIdx.x; i < p.kb; i += kMolThreads) {
      const bool in = q0 + i < t.o1;
      const size_t at = size_t(q0 + i) * p.H + head;
      sl[2 * i] = in ? p.g.lse[at] * kLog2e : -INFINITY;
      sl[2 * i + 1] = in ? p.delta[at] : 0.f;
    }
    __syncthreads();
    if (!warp_live) continue;
    const int nq = min(p.kb, t.o1 - q0);
    for (int j = kw; j < nq; j += kws) {
      float x = 0.f, dp = 0.f;
#pragma unroll
      for (int i = 0; i < KV; ++i)
        if (l + LP * i < kv)
          x = dot4(k[i], *reinterpret_cast<const float4*>(sq + j * p.dk + 4 * (l + LP * i)), x);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        dp = dot4(v[i], *reinterpret_cast<const float4*>(sg + j * G::DV + 4 * (l + LP * i)), dp);
      x = group_sum<LP>(x);
      dp = group_sum<LP>(dp);
      float d = 0.f, dx = 0.f, dy = 0.f, dz = 0.f, slope_x;
      if (p.a.slope) {
        const float4 r = *reinterpret_cast<const float4*>(sp + 4 * j);
        dx = rx - r.x, dy = ry - r.y, dz = rz - r.z;
        d = mol_sqrt(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
        if (d == INFINITY) dx = mol_finite(dx), dy = mol_finite(dy), dz = mol_finite(dz);
      }
      const float w = pair_weight(p, x, slope * kLog2e * d, sl[2 * j], slope_x);
      const float ds = w * (dp - sl[2 * j + 1]);
      if (p.want_pos) {
        const float u = d > 0.f ? __fdividef(-slope * ds, d) : 0.f;
        gx = fmaf(u, dx, gx);
        gy = fmaf(u, dy, gy);
        gz = fmaf(u, dz, gz);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        axpy4(w, *reinterpret_cast<const float4*>(sg + j * G::DV + 4 * (l + LP * i)), dv[i]);
#pragma unroll
      for (int i = 0; i < KV; ++i)
        if (l + LP * i < kv)
          axpy4(ds * slope_x, *reinterpret_cast<const float4*>(sq + j * p.dk + 4 * (l + LP * i)), dk[i]);
    }
  }
  if (kws > 1) {   // the warps that share a row
    float* oj = msm + (rw * G::W + lane / LP) * (G::DV + p.dk + 4);
    for (int w = 1; w < kws; ++w) {
      __syncthreads();
      if (kw == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i) store4(oj + 4 * (l + LP * i), dv[i]);
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv) store4(oj + G::DV + 4 * (l + LP * i), dk[i]);
        if (l == 0) store4(oj + G::DV + p.dk, make_float4(gx, gy, gz, 0.f));
      }
      __syncthreads();
      if (kw == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) axpy4(1.f, *reinterpret_cast<const float4*>(oj + 4 * (l + LP * i)), dv[i]);
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (l + LP * i < kv) axpy4(1.f, *reinterpret_cast<const float4*>(oj + G::DV + 4 * (l + LP * i)), dk[i]);
        const float4 g = *reinterpret_cast<const float4*>(oj + G::DV + p.dk);
        gx += g.x;
        gy += g.y;
        gz += g.z;
      }
    }
  }
  if (!live || kw != 0) return;
#pragma unroll
  for (int i = 0; i < KV; ++i)
    if (l + LP * i < kv)
      store4(static_cast<T*>(p.g.dk) + (row * p.H + head) * p.dk + 4 * (l + LP * i), dk[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    store4(static_cast<T*>(p.g.dhp) + row * p.D * p.C + val_off(p, head, l + LP * i), dv[i]);
  if (p.want_pos && l == 0) {
    float* at = p.part_dk + (size_t(head) * p.nk + row) * 3;
    at[0] = gx;
    at[1] = gy;
    at[2] = gz;
  }
}

// dL/dr summed over groups of heads (and, in the self form, over both roles of an
// atom); the last H blocks sum dL/dslope over query tiles, in a fixed order.
__global__ void mol_reduce_kernel(MolParams p, int pos_blocks) {
  if (int(blockIdx.x) < pos_blocks) {
    const long long nq3 = 3LL * p.nq, nk3 = 3LL * p.nk;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long j = p.a.self ? i : i - nq3;
    if (i < nq3 && p.g.dposq) {
      float s = 0.f;
      for (int h = 0; h < p.groups; ++h) s += p.part_dq[h * nq3 + i];
      if (p.a.self)
        for (int h = 0; h < p.groups_k; ++h) s += p.part_dk[h * nk3 + i];
      p.g.dposq[i] = s;
    }
    if (!p.a.self && j >= 0 && j < nk3 && p.g.dposk) {
      float s = 0.f;
      for (int h = 0; h < p.groups_k; ++h) s += p.part_dk[h * nk3 + j];
      p.g.dposk[j] = s;
    }
    return;
  }
  if (!p.g.dslope) return;
  __shared__ float part[256];
  const int h = blockIdx.x - pos_blocks;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.slots; i += 256) s += p.part_ds[size_t(h) * p.slots + i];
  part[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (int(threadIdx.x) < o) part[threadIdx.x] += part[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) p.g.dslope[h] = part[0];
}

// Value columns of a head as NV float4 vectors in each of LP lanes: dv / 4 is
// a power of two, or nine times one at lmax 2.  Up to nine vectors a lane
// keep the accumulators of a row in registers.
template <typename F>
int by_rows(int dv, F&& f) {
  switch (dv / 4) {
#define EGAT_ROWS(n, NV, LP) \
  case n: return f(std::integral_constant<int, NV>{}, std::integral_constant<int, LP>{})
    EGAT_ROWS(2, 2, 1);
    EGAT_ROWS(4, 4, 1);
    EGAT_ROWS(8, 8, 1);
    EGAT_ROWS(16, 8, 2);
    EGAT_ROWS(32, 8, 4);
    EGAT_ROWS(64, 8, 8);
    EGAT_ROWS(128, 8, 16);
    EGAT_ROWS(256, 8, 32);
    EGAT_ROWS(512, 16, 32);
    EGAT_ROWS(18, 9, 2);
    EGAT_ROWS(36, 9, 4);
    EGAT_ROWS(72, 9, 8);
    EGAT_ROWS(144, 9, 16);
    EGAT_ROWS(288, 9, 32);
#undef EGAT_ROWS
    default: return EGAT_ERR_UNSUPPORTED;
  }
}

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }
int ceil_log2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
int head_columns(const egat_mol_shape& s) { return (s.lmax + 1) * (s.lmax + 1) * (s.C / s.H); }
// ... and the query vectors of a lane
template <typename F>
int by_rows_dk(int dv, int dk, F&& f) {
  return by_rows(dv, [&](auto nv, auto lp) {
    constexpr int LP = decltype(lp)::value;
    if constexpr (LP < 8) {
      if (dk > 16) return f(nv, lp, std::integral_constant<int, 8 / LP>{});
    }
    if constexpr (LP < 4) {
      if (dk > 8) return f(nv, lp, std::integral_constant<int, 4 / LP>{});
    }
    return f(nv, lp, std::integral_constant<int, LP < 2 ? 2 : 1>{});
  });
}

// How a pass cuts a shape: rows of a tile and key splits.  Depends on the shape alone.
struct MolCut {
  bool tc;
  bool umma;    // forward on tcgen05, tiles of 128 rows
  int rwlog;    // log2 of the warps side by side over rows
  int rows;     // rows of a tile
  int groups;   // blocks side by side over heads
  int splits;
};
long long tile_blocks(int n, int n_mol, int rows, int groups) {
  return ((long long)n / rows + std::min(n_mol, n)) * groups;
}
// Tiles of four (two) warps' rows read the other side's rows a quarter (half) as often
// as tiles of one warp's, whose four warps share those rows instead: taken where
// `four` (`two`) blocks remain and the molecules are that long.
int wide_log(int n, int n_mol, int rows, int groups, int four, int two) {
  for (int l = 2; l > 0; --l)
    if (tile_blocks(n, n_mol, rows << l, groups) >= (l == 2 ? four : two) &&
        (long long)n >= (long long)(rows / 2 << l) * n_mol)
      return l;
  return 0;
}
MolCut tile_cut(const egat_mol_shape& s, int n, bool query_gradients = false) {
  MolCut c{};
  c.tc = mol_tc_supported(s);
  c.groups = c.tc ? s.H / mol_tc_heads(s, query_gradients) : s.H;
  c.splits = 1;
  if (c.tc) {
    // 64 rows from 1.2 blocks an SM on, 32 from half a block: at 192 blocks 64 rows are 7 %
    // faster than 32, at 176 12 % slower, at 128 9 %; at 80 blocks 32 rows are 30 % faster
    // than 16, whose batches of short molecules take 279 us in place of 124.  Rows of few
    // value columns cost little to read again: 110 blocks of 32 rows take 55 us, twice as
    // many of 16 rows 46
    c.rwlog = wide_log(n, s.n_mol, 16, c.groups, 180, head_columns(s) > 32 ? 74 : 148);
    c.rows = 16 << c.rwlog;
    return c;
  }
  int w = 1;
  by_rows(head_columns(s), [&](auto nv, auto lp) {
    w = MolRows<decltype(nv)::value, decltype(lp)::value>::W;
    return 0;
  });
  c.rwlog = wide_log(n, s.n_mol, w, s.H, 4 * 148, 4 * 148);
  c.rows = w << c.rwlog;
  return c;
}
MolCut forward_cut(const egat_mol_shape& s) {
  MolCut c = tile_cut(s, s.nq);
  // Long molecules: tcgen05 tiles of 128 rows, from 512 atoms on, where they fill most of
  // their last tile, and with 96 blocks.  Both sides measured, bf16 at lmax 2 with a bias:
  // one system of 500 atoms 24 against 22 us, of 700 27 against 33, of 2,000 75 against
  // 162; 64 molecules of 200 atoms 119 against 85, of 400 273 against 240; 56 blocks of
  // 8-column heads 74 against 44.
  if (mol_umma_supported(s) && s.n_mol > 0 && (long long)s.nq >= 512LL * s.n_mol && (long long)s.nk >= 512LL * s.n_mol) {
    if (tile_blocks(s.nq, s.n_mol, 128, s.H) >= 96) {
      c.umma = true;
      c.rows = 128;
      c.splits = 1;
      return c;
    }
  }
  // With fewer row tiles than two blocks an SM, each molecule's keys are cut, but not
  // below 128 keys a part on average: one wave of three blocks an SM for one molecule
  // (four are two waves: 45 instead of 37 us for one row against 32,768), finer for
  // several, whose lengths may differ.
  if (s.n_mol > 0 && s.nk > 0 && c.rwlog == 0) {
    const long long blocks = std::max(1LL, tile_blocks(s.nq, s.n_mol, c.rows, c.groups));
    const long long most = s.nk / s.n_mol / 128, want = (s.n_mol > 1 ? 8LL : 3LL) * 148 / blocks;
    if (blocks < 2 * 148) c.splits = int(std::max(1LL, std::min(std::min(most, want), 64LL)));
  }
  return c;
}

MolParams base_params(const egat_mol_shape& s, const MolArgs& a) {
  MolParams p{};
  p.a = a;
  p.nq = s.nq;
  p.nk = s.nk;
  p.nmol = s.n_mol;
  p.D = (s.lmax + 1) * (s.lmax + 1);
  p.C = s.C;
  p.H = s.H;
  p.dk = s.dk;
  p.ch = s.C / s.H;
  p.ch8log = ceil_log2(p.ch / 8);
  p.dv = p.D * p.ch;
  p.splits = 1;
  p.scale = 1.f / std::sqrt(float(s.dk));
  p.cap = s.cap;
  p.inv_cap = s.cap > 0.f ? 1.f / s.cap : 0.f;
  // rows of a staged tile: up to 32 within 40 KB
  p.kb = std::max(kMolBatch, std::min(32, int(40 * 1024 / (4 * (s.dk + p.dv + 6))) & ~(kMolBatch - 1)));
  return p;
}
// a staged tile, or the rows that the warps of a tile join
size_t stage_bytes(const MolParams& p, int w) {
  return size_t(std::max(p.kb, w << p.rwlog)) * (p.dk + p.dv + 6) * sizeof(float);
}
int launched() { return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA; }

template <typename T>
int forward_t(const MolParams& p, cudaStream_t st) {
  return by_rows_dk(p.dv, p.dk, [&](auto nv, auto lp, auto kv) {
    constexpr int NV = decltype(nv)::value, LP = decltype(lp)::value, KV = decltype(kv)::value;
    return mol_launch(mol_fwd_kernel<NV, LP, KV, T>, dim3(p.slots, p.H, p.splits), kMolThreads,
                      stage_bytes(p, MolRows<NV, LP>::W), p, st);
  });
}

template <typename T>
int backward_t(MolParams p, int k_rwlog, cudaStream_t st) {
  return by_rows_dk(p.dv, p.dk, [&](auto nv, auto lp, auto kv) {
    constexpr int NV = decltype(nv)::value, LP = decltype(lp)::value, KV = decltype(kv)::value;
    constexpr int W = MolRows<NV, LP>::W;
    int rc = EGAT_OK;
    if (p.nq > 0)
      rc = mol_launch(mol_bwd_q_kernel<NV, LP, KV, T>, dim3(p.slots, p.H), kMolThreads, stage_bytes(p, W), p, st);
    p.rwlog = k_rwlog;
    if (rc == EGAT_OK && p.nk > 0)
      rc = mol_launch(mol_bwd_k_kernel<NV, LP, KV, T>, dim3(mol_slots(p.nk, p.nmol, W << p.rwlog), p.H), kMolThreads,
                      stage_bytes(p, W), p, st);
    return rc;
  });
}

// Workspace of the backward pass: delta (and lse in base 2), then the partial sums of the
// position and slope gradients.
struct MolBwdWs {
  MolCut cut, cut_k;   // query and key side
  int slots;
  size_t delta, nlse2, dq, dk, ds, total;
};
MolBwdWs bwd_ws(const egat_mol_shape& s) {
  MolBwdWs w;
  w.cut = tile_cut(s, s.nq, true);
  w.cut_k = tile_cut(s, s.nk);
  w.slots = mol_slots(s.nq, s.n_mol, w.cut.rows);
  w.delta = 0;
  w.nlse2 = up256(sizeof(float) * size_t(s.nq) * s.H);
  w.dq = w.nlse2 + (w.cut.tc ? w.nlse2 : 0);
  w.dk = w.dq + up256(sizeof(float) * 3 * size_t(s.nq) * w.cut.groups);
  w.ds = w.dk + up256(sizeof(float) * 3 * size_t(s.nk) * w.cut_k.groups);
  w.total = w.ds + up256(sizeof(float) * size_t(w.slots) * s.H);
  return w;
}

}  // namespace

// Two heads a warp where the accumulators of two fit its registers, one of float32.
int mol_tc_heads(const egat_mol_shape& s, bool query_gradients) {
  return s.dtype == EGAT_BF16 && head_columns(s) <= (query_gradients ? 64 : 72) ? 2 : 1;
}
// Up to 256 value columns a head of bf16 and 144 of float32 (the accumulators of 16
// rows and the operands beside them fill a warp's registers there), and two heads
// where two are taken together.
bool mol_tc_supported(const egat_mol_shape& s) {
  const int nt = head_columns(s) / 8;
  return s.H >= mol_tc_heads(s, false) && (nt == 1 || nt == 2 || nt == 4 || nt == 8 || nt == 9 || nt == 16 || nt == 18 ||
                                    (nt == 32 && s.dtype == EGAT_BF16));
}

size_t molecule_ws_bytes(const egat_mol_shape& s) {
  const MolCut c = forward_cut(s);
  if (c.umma) return up256(mol_umma_key_bytes(s)) + up256(mol_umma_query_bytes(s));
  if (c.splits == 1) return 0;
  const size_t rows = size_t(c.splits) * s.nq * s.H;
  return up256(rows * head_columns(s) * sizeof(float)) + up256(rows * 2 * sizeof(float));
}

int launch_molecule_attention(const egat_mol_shape& s, const MolArgs& a, void* d_ws, void* d_m,
                              float* d_lse, cudaStream_t st) {
  MolParams p = base_params(s, a);
  p.m = d_m;
  p.lse = d_lse;
  const MolCut c = forward_cut(s);
  p.splits = c.splits;
  p.rwlog = c.rwlog;
  if (c.umma) {
    p.slots = mol_slots(s.nq, s.n_mol, c.rows);
    p.kv_slots = mol_slots(s.nk, s.n_mol, 64);
    p.kv = d_ws;
    p.qp = static_cast<char*>(d_ws) + up256(mol_umma_key_bytes(s));
    const int rc = mol_umma_pack(p, st);
    return rc != EGAT_OK ? rc : mol_umma_forward(p, st);
  }
  if (p.splits > 1) {
    p.part_o = static_cast<float*>(d_ws);
    p.part_ml = reinterpret_cast<float*>(static_cast<char*>(d_ws) +
                                         up256(size_t(p.splits) * s.nq * s.H * p.dv * sizeof(float)));
  }
  p.slots = mol_slots(s.nq, s.n_mol, c.rows);
  const bool bf16 = s.dtype == EGAT_BF16;
  const int rc = c.tc ? (bf16 ? mol_tc_forward_bf16(p, st) : mol_tc_forward_f32(p, st))
                      : bf16 ? forward_t<__nv_bfloat16>(p, st) : forward_t<float>(p, st);
  if (rc != EGAT_OK || p.splits == 1) return rc;
  const unsigned blocks = unsigned(size_t(p.nq) * p.H);
  if (bf16)
    mol_join_kernel<__nv_bfloat16><<<blocks, 128, 0, st>>>(p);
  else
    mol_join_kernel<float><<<blocks, 128, 0, st>>>(p);
  return launched();
}

size_t molecule_backward_ws_bytes(const egat_mol_shape& s) {
  return bwd_ws(s).total;
}

int launch_molecule_backward(const egat_mol_shape& s, const MolArgs& a, const MolGrads& g,
                             void* d_ws, cudaStream_t st) {
  MolParams p = base_params(s, a);
  p.g = g;
  const MolBwdWs w = bwd_ws(s);
  char* base = static_cast<char*>(d_ws);
  p.delta = reinterpret_cast<float*>(base + w.delta);
  p.nlse2 = reinterpret_cast<float*>(base + w.nlse2);
  p.part_dq = reinterpret_cast<float*>(base + w.dq);
  p.part_dk = reinterpret_cast<float*>(base + w.dk);
  p.part_ds = reinterpret_cast<float*>(base + w.ds);
  p.want_pos = g.dposq || g.dposk || g.dslope;
  // float32 m gives delta to float32; bf16 m would leave it bf16's error, which
  // showed as 1.6 times the rounding error of dq (4,096 atoms, 16 heads)
  p.exact_delta = s.dtype == EGAT_BF16;
  p.slots = w.slots;
  p.groups = w.cut.groups;
  p.groups_k = w.cut_k.groups;
  p.rwlog = w.cut.rwlog;
  const bool bf16 = s.dtype == EGAT_BF16;
  const int k_rwlog = w.cut_k.rwlog;
  int rc = EGAT_OK;
  if (w.cut.tc) {
    if (s.nq > 0) rc = bf16 ? mol_tc_backward_q_bf16(p, st) : mol_tc_backward_q_f32(p, st);
    p.rwlog = k_rwlog;
    if (rc == EGAT_OK && s.nk > 0) rc = bf16 ? mol_tc_backward_k_bf16(p, st) : mol_tc_backward_k_f32(p, st);
  } else {
    rc = bf16 ? backward_t<__nv_bfloat16>(p, k_rwlog, st) : backward_t<float>(p, k_rwlog, st);
  }
  if (rc != EGAT_OK || !p.want_pos) return rc;
  if (s.nq == 0) {   // no query tile ran
    if (g.dslope && cudaMemsetAsync(g.dslope, 0, sizeof(float) * s.H, st) != cudaSuccess)
      return EGAT_ERR_CUDA;
    if (!g.dposk) return EGAT_OK;
    p.g.dslope = nullptr;
  }
  const long long rows3 = 3LL * s.nq + (a.self ? 0 : 3LL * s.nk);
  const int pos_blocks = int((rows3 + 255) / 256);
  mol_reduce_kernel<<<pos_blocks + s.H, 256, 0, st>>>(p, pos_blocks);
  return launched();
}

}  // namespace egat
