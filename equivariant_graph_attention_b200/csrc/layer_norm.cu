// Layer norm of strided rows, forward and backward.
//
//   y = (x - mu) rstd w + b;  with xh = (x - mu) rstd and t = g w,
//   dx = rstd (t - mean t - xh mean(t xh)),  dw = sum_rows g xh,  db = sum_rows g
//
// Bound by memory: every row is read once, kept in registers for the centred
// second moment (taken about the mean, not as E x^2 - mu^2, which loses
// everything for rows far from zero) and the output, and written once.  TPR
// threads share a row: part of a warp up to 32 vectors, a warp up to 1,024
// columns, a block beyond.  Vectors are 16 bytes of bf16 (two of float32)
// where width, strides and pointers allow, pairs or single elements otherwise.
// A thread keeps its columns' weight and bias over the rows that it visits and has
// the next row on its way (100,000 x 1,000 bf16 rows: 74 us, 82 % of the measured copy
// rate; 209 us with both read again for every row, a block a row).
//
// The weight sums of the backward pass: each thread keeps its columns' sums
// over the rows its block visits, the block joins its rows' groups in a fixed
// order and writes one partial row, and a second kernel adds the partial rows
// in order.  No atomics: the same sums on every call.
#include "egat_device.cuh"
#include "egat_host.h"

namespace egat {
namespace {

// E consecutive elements, kept as stored
template <typename T, int E>
struct Vec;
template <>
struct Vec<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&o)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&o)[8]) const { bf16x8_to_f32(v, o); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&o)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void get(float (&o)[2]) const { o[0] = v.x, o[1] = v.y; }
  static __device__ __forceinline__ void store(float* p, const float (&o)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(o[0], o[1]);
  }
};
template <>
struct Vec<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = __uint_as_float(v << 16), o[1] = __uint_as_float(v & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&o)[2]) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(o[0], o[1]);
  }
};
template <typename T>
struct Vec<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = float(v); }
  static __device__ __forceinline__ void store(T* p, const float (&o)[1]) { store_one<T>(p, o[0]); }
};

struct NormParams {
  const void* x;
  const void* g;
  const float *w, *b, *stats;
  void* y;         // y, or dx
  float* stats_out;
  float* part;     // [blocks][2][width]
  long long ldx, ldg, ldy;
  int n, width;
  float eps, inv_width;
};

constexpr int kNormThreads = 256;
template <int TPR>
constexpr int norm_threads() { return TPR > 32 ? TPR : kNormThreads; }

// Sum over the TPR threads of a row (all of them get it).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if constexpr (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}

// E float32 parameters; VEC: their pointer is 16-byte aligned
template <int E, bool VEC>
__device__ __forceinline__ void load_f32(const float* p, int c, float dflt, float (&o)[E]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = dflt;
    return;
  }
  if constexpr (VEC && E == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + c)), b = __ldg(reinterpret_cast<const float4*>(p + c) + 1);
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __ldg(p + c + e);
  }
}

// A thread keeps its columns' parameters over the rows that it visits where they
// fit its registers, and reads them again for every row otherwise.
template <int E, int V>
constexpr bool norm_hold() { return E == 8 && V <= 4; }

// The warps' column sums lie side by side in shared memory up to 512 columns.
template <int E, int V>
constexpr bool norm_side() { return E == 8 && V <= 2; }

template <typename T, int E, int TPR, int V>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_fwd_kernel(NormParams p) {
  constexpr int NT = norm_threads<TPR>();
  constexpr bool HOLD = norm_hold<E, V>();
  __shared__ float red[32];
  const int lane = threadIdx.x % TPR;
  const long long stride = (long long)gridDim.x * (NT / TPR);
  float hw[HOLD ? V : 1][E], hb[HOLD ? V : 1][E];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width) {
        load_f32<E, true>(p.w, c, 1.f, hw[i]);
        load_f32<E, true>(p.b, c, 0.f, hb[i]);
      }
    }
  }
  Vec<T, E> raw[V], next[HOLD ? V : 1];
  auto fetch = [&](long long r0, Vec<T, E>(&v)[V]) {
    const long long row = r0 + threadIdx.x / TPR;
    const T* x = static_cast<const T*>(p.x) + (row < p.n ? row : r0) * p.ldx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width) v[i].load(x + c);
    }
  };
  // whole blocks stay in step: row_sum shuffles and, for TPR > 32, synchronises
  long long r0 = (long long)blockIdx.x * (NT / TPR);
  if (HOLD && r0 < p.n) fetch(r0, raw);
  for (; r0 < p.n; r0 += stride) {
    const long long row = r0 + threadIdx.x / TPR;
    const bool live = row < p.n;
    if constexpr (HOLD) {
      if (r0 + stride < p.n) fetch(r0 + stride, next);   // the next row is on its way meanwhile
    } else {
      fetch(r0, raw);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((lane + i * TPR) * E < p.width) {
        float v[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
      }
    const float mu = row_sum<TPR>(s, red) * p.inv_width;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((lane + i * TPR) * E < p.width) {
        float v[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(v[e] - mu, v[e] - mu, s);
      }
    const float rstd = rsqrtf(row_sum<TPR>(s, red) * p.inv_width + p.eps);
    if (live) {
      T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (lane + i * TPR) * E;
        if (c < p.width) {
          float v[E], w[E], b[E];
          raw[i].get(v);
          if constexpr (HOLD) {
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = hw[i][e], b[e] = hb[i][e];
          } else {
            load_f32<E, false>(p.w, c, 1.f, w);
            load_f32<E, false>(p.b, c, 0.f, b);
          }
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = fmaf((v[e] - mu) * rstd, w[e], b[e]);
          Vec<T, E>::store(y + c, v);
        }
      }
      if (lane == 0 && p.stats_out) {
        p.stats_out[2 * row] = mu;
        p.stats_out[2 * row + 1] = rstd;
      }
    }
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < V; ++i) raw[i] = next[i];
    }
  }
}

template <typename T, int E, int TPR, int V>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_bwd_kernel(NormParams p) {
  constexpr int NT = norm_threads<TPR>(), WARPS = NT / 32;
  constexpr bool HOLD = norm_hold<E, V>();
  extern __shared__ float sums[];   // [2][width], by warp where norm_side
  __shared__ float red[32];
  const int lane = threadIdx.x % TPR;
  float dw[V][E] = {}, db[V][E] = {}, hw[HOLD ? V : 1][E];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((lane + i * TPR) * E < p.width) load_f32<E, true>(p.w, (lane + i * TPR) * E, 1.f, hw[i]);
  }
  const long long stride = (long long)gridDim.x * (NT / TPR);
  for (long long r0 = (long long)blockIdx.x * (NT / TPR); r0 < p.n; r0 += stride) {
    const long long row = r0 + threadIdx.x / TPR;
    const bool live = row < p.n;
    const long long at = live ? row : r0;
    const T* x = static_cast<const T*>(p.x) + at * p.ldx;
    const T* g = static_cast<const T*>(p.g) + at * p.ldg;
    Vec<T, E> rx[V], rg[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width) {
        rx[i].load(x + c);
        rg[i].load(g + c);
      }
    }
    const float mu = p.stats[2 * at], rstd = p.stats[2 * at + 1];
    auto weight = [&](int i, float (&w)[E]) {
      if constexpr (HOLD) {
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = hw[i][e];
      } else {
        load_f32<E, false>(p.w, (lane + i * TPR) * E, 1.f, w);
      }
    };
    float st = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width) {
        float xv[E], gv[E], w[E];
        rx[i].get(xv);
        rg[i].get(gv);
        weight(i, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xh = (xv[e] - mu) * rstd, t = gv[e] * w[e];
          st += t;
          sx = fmaf(t, xh, sx);
          if (live) {
            dw[i][e] = fmaf(gv[e], xh, dw[i][e]);
            db[i][e] += gv[e];
          }
        }
      }
    }
    if (!p.y) continue;
    const float mt = row_sum<TPR>(st, red) * p.inv_width;
    const float mx = row_sum<TPR>(sx, red) * p.inv_width;
    if (!live) continue;
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width) {
        float xv[E], gv[E], w[E];
        rx[i].get(xv);
        rg[i].get(gv);
        weight(i, w);
#pragma unroll
        for (int e = 0; e < E; ++e)
          xv[e] = rstd * (gv[e] * w[e] - mt - (xv[e] - mu) * rstd * mx);
        Vec<T, E>::store(y + c, xv);
      }
    }
  }
  if (!p.part) return;
  float* part = p.part + size_t(blockIdx.x) * 2 * p.width;
  if constexpr (TPR > 32) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (lane + i * TPR) * E;
      if (c < p.width)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          part[c + e] = dw[i][e];
          part[p.width + c + e] = db[i][e];
        }
    }
  } else {
    // the groups of a warp by shuffles, then the warps in turn
#pragma unroll
    for (int o = 16; o >= TPR; o >>= 1)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dw[i][e] += __shfl_xor_sync(~0u, dw[i][e], o);
          db[i][e] += __shfl_xor_sync(~0u, db[i][e], o);
        }
    if constexpr (norm_side<E, V>()) {
      if (int(threadIdx.x % 32) < TPR) {
        float* own = sums + (threadIdx.x / 32) * 2 * p.width;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (lane + i * TPR) * E;
          if (c < p.width)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              own[c + e] = dw[i][e];
              own[p.width + c + e] = db[i][e];
            }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * p.width; c += NT) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) s += sums[k * 2 * p.width + c];
        part[c] = s;
      }
      return;
    }
    for (int k = 0; k < WARPS; ++k) {
      if (int(threadIdx.x / 32) == k && int(threadIdx.x % 32) < TPR) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (lane + i * TPR) * E;
          if (c < p.width)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              float* a = sums + c + e;
              a[0] = k ? a[0] + dw[i][e] : dw[i][e];
              a[p.width] = k ? a[p.width] + db[i][e] : db[i][e];
            }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.width; c += NT) part[c] = sums[c];
  }
}

// Adds the partial rows: 8 columns (a memory sector) a block, 64 threads down each
// column with four sums each, joined in a fixed order.
constexpr int kReduceCols = 8, kReduceRows = 64;
__global__ void __launch_bounds__(kReduceCols * kReduceRows)
    norm_reduce_kernel(const float* part, int blocks, int width, float* dw, float* db) {
  __shared__ float sm[kReduceCols][kReduceRows + 1];
  const int x = threadIdx.x % kReduceCols, y = threadIdx.x / kReduceCols, c = blockIdx.x * kReduceCols + x;
  float s[4] = {};
  if (c < 2 * width)
    for (int b = y; b < blocks; b += 4 * kReduceRows)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b + i * kReduceRows < blocks) s[i] += part[size_t(b + i * kReduceRows) * 2 * width + c];
  sm[x][y] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, col = blockIdx.x * kReduceCols + warp;
  if (warp >= kReduceCols) return;
  float v = sm[warp][lane] + sm[warp][lane + 32];   // a warp adds one column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (lane == 0 && col < 2 * width) {
    float* out = col < width ? dw : db;
    if (out) out[col < width ? col : col - width] = v;
  }
}

// Calls f with the vector width E, the threads of a row and their vectors.
template <int E, typename F>
int by_width_e(int width, F&& f) {
  const int nv = (width + E - 1) / E;
#define EGAT_NORM(T_, V_) \
  return f(std::integral_constant<int, E>{}, std::integral_constant<int, T_>{}, std::integral_constant<int, V_>{})
  if constexpr (E == 8) {
    if (nv <= 2) EGAT_NORM(2, 1);
    if (nv <= 4) EGAT_NORM(4, 1);
    if (nv <= 8) EGAT_NORM(8, 1);
    if (nv <= 16) EGAT_NORM(16, 1);
    if (nv <= 32) EGAT_NORM(32, 1);
    if (nv <= 64) EGAT_NORM(32, 2);
    if (nv <= 128) EGAT_NORM(32, 4);
    if (nv <= 256) EGAT_NORM(256, 1);
    if (nv <= 512) EGAT_NORM(256, 2);
    if (nv <= 1024) EGAT_NORM(256, 4);
    EGAT_NORM(512, 4);
  } else {
    constexpr int K = 2 / E;   // single elements need twice the vectors
    if (nv <= 32 * 2 * K) EGAT_NORM(32, 2 * K);
    if (nv <= 32 * 6 * K) EGAT_NORM(32, 6 * K);
    if (nv <= 32 * 16 * K) EGAT_NORM(32, 16 * K);
    if (nv <= 256 * 4 * K) EGAT_NORM(256, 4 * K);
    if (nv <= 256 * 8 * K) EGAT_NORM(256, 8 * K);
    EGAT_NORM(512, 16 * K);
  }
#undef EGAT_NORM
}
// The widest vectors that width, strides and pointers allow: 16-byte vectors
// of bf16 or 16-byte halves of float32, pairs, or elements.
template <typename T, typename F>
int by_width(int width, const float* w, const float* bias, const void* a, long long lda, const void* b,
             long long ldb, const void* c, long long ldc, F&& f) {
  auto fits = [&](int e, size_t bytes) {
    auto one = [&](const void* q, long long ld) {
      return !q || (reinterpret_cast<uintptr_t>(q) % bytes == 0 && ld * (long long)sizeof(T) % (long long)bytes == 0);
    };
    return width % e == 0 && one(a, lda) && one(b, ldb) && one(c, ldc);
  };
  const bool params = ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(bias)) & 15) == 0;
  if (fits(8, 16) && params) return by_width_e<8>(width, f);
  if (fits(2, 2 * sizeof(T))) return by_width_e<2>(width, f);
  return by_width_e<1>(width, f);
}

int launched() { return cudaGetLastError() == cudaSuccess ? EGAT_OK : EGAT_ERR_CUDA; }

template <typename T>
int norm_fwd_t(const NormParams& p, cudaStream_t st) {
  return by_width<T>(p.width, p.w, p.b, p.x, p.ldx, p.y, p.ldy, nullptr, 0, [&](auto e, auto tpr, auto v) {
    constexpr int E = decltype(e)::value, TPR = decltype(tpr)::value, V = decltype(v)::value;
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR;
    // up to eight blocks an SM; beyond, a block takes several rows with its
    // parameters in registers and the next row on its way
    const long long blocks = std::min<long long>(148 * 8, ((long long)p.n + ROWS - 1) / ROWS);
    norm_fwd_kernel<T, E, TPR, V><<<unsigned(blocks), NT, 0, st>>>(p);
    return launched();
  });
}

// Blocks of the backward pass: the partial rows are 2 * width floats each.
constexpr int kNormBlocks = 148 * 4;
int norm_blocks(int n, int rows_per_block) {
  return int(std::min<long long>(kNormBlocks, ((long long)n + rows_per_block - 1) / rows_per_block));
}

template <typename T>
int norm_bwd_t(NormParams p, bool want_w, float* d_dw, float* d_db, cudaStream_t st) {
  int blocks = 0;
  const int rc = by_width<T>(p.width, p.w, p.b, p.x, p.ldx, p.y, p.ldy, p.g, p.ldg, [&](auto e, auto tpr, auto v) {
    constexpr int E = decltype(e)::value, TPR = decltype(tpr)::value, V = decltype(v)::value;
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR;
    blocks = norm_blocks(p.n, ROWS);
    const size_t shm = TPR > 32 || !want_w ? 0 : 2 * size_t(p.width) * sizeof(float) * (norm_side<E, V>() ? NT / 32 : 1);
    norm_bwd_kernel<T, E, TPR, V><<<blocks, NT, shm, st>>>(p);
    return launched();
  });
  if (rc != EGAT_OK || !want_w) return rc;
  norm_reduce_kernel<<<(2 * p.width + kReduceCols - 1) / kReduceCols, kReduceCols * kReduceRows, 0, st>>>(
      p.part, blocks, p.width, d_dw, d_db);
  return launched();
}

}  // namespace

int launch_layer_norm(const void* d_x, long long ldx, int n, int width, int dtype,
                      const float* d_weight, const float* d_bias, float eps, void* d_y,
                      long long ldy, float* d_stats, cudaStream_t st) {
  NormParams p{};
  p.x = d_x;
  p.ldx = ldx;
  p.n = n;
  p.width = width;
  p.w = d_weight;
  p.b = d_bias;
  p.eps = eps;
  p.inv_width = 1.f / float(width);
  p.y = d_y;
  p.ldy = ldy;
  p.stats_out = d_stats;
  return dtype == EGAT_BF16 ? norm_fwd_t<__nv_bfloat16>(p, st) : norm_fwd_t<float>(p, st);
}

size_t layer_norm_backward_ws_bytes(int n, int width) {
  return n == 0 ? 0 : size_t(norm_blocks(n, 1)) * 2 * width * sizeof(float);
}

int launch_layer_norm_backward(const void* d_x, long long ldx, int n, int width, int dtype,
                               const float* d_weight, const float* d_stats, const void* d_grad,
                               long long ldg, void* d_ws, void* d_dx, long long lddx,
                               float* d_dweight, float* d_dbias, cudaStream_t st) {
  if (n == 0) {
    for (float* d : {d_dweight, d_dbias})
      if (d && cudaMemsetAsync(d, 0, sizeof(float) * size_t(width), st) != cudaSuccess)
        return EGAT_ERR_CUDA;
    return EGAT_OK;
  }
  const bool want_w = d_dweight || d_dbias;
  NormParams p{};
  p.x = d_x;
  p.ldx = ldx;
  p.g = d_grad;
  p.ldg = ldg;
  p.n = n;
  p.width = width;
  p.w = d_weight;
  p.stats = d_stats;
  p.inv_width = 1.f / float(width);
  p.y = d_dx;
  p.ldy = lddx;
  p.part = want_w ? static_cast<float*>(d_ws) : nullptr;
  return dtype == EGAT_BF16 ? norm_bwd_t<__nv_bfloat16>(p, want_w, d_dweight, d_dbias, st)
                            : norm_bwd_t<float>(p, want_w, d_dweight, d_dbias, st);
}

}  // namespace egat
