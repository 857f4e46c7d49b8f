// Layer norm and RMS norm over rows, forward and backward (sm_100a).
//
//   forward    mu = <x>,  rstd = 1/sqrt(<(x - mu)^2> + eps),  y = (x - mu) rstd w + b
//   backward   xh = (x - mu) rstd,  g = dy w
//              dx = rstd (g - <g> - xh <g xh>)
//              dw = sum_rows dy xh,  db = sum_rows dy
// < > is the mean over the row; the RMS norm has mu = 0 and no <g> term.
//
// Everything is bound by HBM: the forward pass reads x and writes y once, the
// backward pass reads dy and x and writes dx once.  A group of G threads (8
// lanes of a warp up to a block of 512) holds one row in registers, so a row is
// read once whatever the number of reductions over it, and loads its next row
// before it reduces the present one.  The weight is read from L1 for every row
// (kept in registers, it cost half of the rows in flight); backward, the dw/db
// sums of a thread's columns stay in registers.  Backward, the groups of a block join their sums in shared
// memory, each block writes one partial row, and a second small kernel adds the
// partial rows in a fixed order: no atomics, the same bits every time.  Rows
// wider than the registers hold (kWide) are walked over in global memory, and
// dw/db then come from a kernel of their own that walks down the columns.
//
// All sums are fp32: per thread over at most 16 elements of a row, then a tree.
#include <algorithm>
#include <cmath>

#include "muonh_common.cuh"

namespace muonh {
namespace {

constexpr int kNormThreads = 512;
constexpr int kMaxPack = 16;                        // elements of a row per thread
constexpr int kWide = kNormThreads * kMaxPack;      // widest row held in registers: 8192
constexpr int kMaxParts = 512;                      // partial rows of dw/db

struct NormParams {
  const void* x;
  const void* dy;
  void* out;                 // y, or dx
  const float* weight;       // may be null
  const float* bias;         // may be null
  float* mean;               // null: RMS norm
  float* rstd;
  float* part_w;             // backward: partial rows of dw (null: not wanted)
  float* part_b;
  int64_t rows, ldx, lddy, ldo;
  int32_t n, group;          // row width; threads per row
  float eps;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements from a 16-byte aligned address (V = 1: any address),
// as loaded and as fp32.
template <typename T, int V>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void to(float* v) const {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f(e[i]);
  }
};
template <typename T>
struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void zero() { u = from_f<T>(0.f); }
  __device__ __forceinline__ void to(float* v) const { v[0] = to_f(u); }
};
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float* v) {
  if constexpr (V == 1) {
    *p = from_f<T>(v[0]);
  } else {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = u;
  }
}
// V fp32 values of a weight-like array, 16-byte aligned where V > 1; `none` without one.
template <int V>
__device__ __forceinline__ void load_f32(const float* p, int64_t j, float none, float* v) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = none;
  } else if constexpr (V == 1) {
    v[0] = __ldg(p + j);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + j + i));
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  }
}

// Sums of a and b over the `group` threads of a row, in every thread of it.
// Groups within a warp use shuffles; wider groups add their warps' sums in
// shared memory behind a barrier of their own.  `buf` alternates between two
// slots, so that one barrier per call is enough.
struct GroupSum {
  float2* slots;             // [2][16] of this group's warps
  int group, bar, flip;
  __device__ __forceinline__ void operator()(float& a, float& b) {
    const int w = group < 32 ? group : 32;
    for (int o = w >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (group > 32) {
      const int warps = group >> 5, warp = (threadIdx.x % group) >> 5;
      float2* s = slots + flip * 16;
      flip ^= 1;
      if ((threadIdx.x & 31) == 0) s[warp] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(group) : "memory");
      a = b = 0.f;
      for (int i = 0; i < warps; ++i) {
        const float2 t = s[i];
        a += t.x;
        b += t.y;
      }
    }
  }
};

__device__ __forceinline__ GroupSum group_sum(float2* shared, int group) {
  const int g = threadIdx.x / group;
  // wider groups than a warp: at most 8 of 64 threads, barrier ids 1..8
  return GroupSum{group > 32 ? shared + 32 * g : shared, group, 1 + (group > 32 ? g : 0), 0};
}

template <typename T, int V, int P>
__global__ void __launch_bounds__(kNormThreads, V * P <= 8 ? 3 : 1) norm_forward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 sums[8 * 32];
  const int G = p.group, t = threadIdx.x % G, n = p.n;
  const int per_block = kNormThreads / G;
  GroupSum total = group_sum(sums, G);
  const float inv_n = 1.f / n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  float w[P * V], b[P * V];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int j = (k * G + t) * V;
    if (j < n) {
      load_f32<V>(p.weight, j, 1.f, w + k * V);
      load_f32<V>(p.bias, j, 0.f, b + k * V);
    }
  }
  Raw<T, V> next[P];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (row < p.rows && j < n)
        next[k].load(x + j);
      else
        next[k].zero();
    }
  };
  int64_t base = static_cast<int64_t>(blockIdx.x) * per_block;
  fetch(base + threadIdx.x / G);
  // the loop's bound is the block's, so that every lane takes part in the shuffles
  for (; base < p.rows; base += step) {
    const int64_t row = base + threadIdx.x / G;
    float v[P * V];
#pragma unroll
    for (int k = 0; k < P; ++k) next[k].to(v + k * V);
    fetch(row + step);
    float mu = 0.f, unused = 0.f;
    if (p.mean) {
#pragma unroll
      for (int i = 0; i < P * V; ++i) mu += v[i];
      total(mu, unused);
      mu *= inv_n;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if ((k * G + t) * V < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[k * V + i] -= mu;
          q = fmaf(v[k * V + i], v[k * V + i], q);
        }
      }
    }
    unused = 0.f;
    total(q, unused);
    const float rstd = 1.f / sqrtf(fmaf(q, inv_n, p.eps));
    if (row >= p.rows) continue;
    T* y = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(v[k * V + i] * rstd, w[k * V + i], b[k * V + i]);
        store_pack<T, V>(y + j, o);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
  }
}

// SUMS: also the partial rows of dw and db.
template <typename T, int V, int P, bool SUMS>
__global__ void __launch_bounds__(kNormThreads, SUMS ? 1 : 2) norm_backward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 sums[8 * 32];
  // [kNormThreads / G][n], where a block has several groups: at most kWide floats, 32 KB
  extern __shared__ float joined[];
  const int G = p.group, t = threadIdx.x % G, n = p.n;
  const int per_block = kNormThreads / G;
  GroupSum total = group_sum(sums, G);
  float dw[P * V], db[P * V];
#pragma unroll
  for (int i = 0; i < P * V; ++i) dw[i] = db[i] = 0.f;
  const float inv_n = 1.f / n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  Raw<T, V> next_x[P], next_dy[P];
  float next_mean = 0.f, next_rstd = 0.f;
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (row < p.rows && j < n) {
        next_x[k].load(x + j);
        next_dy[k].load(dy + j);
      } else {
        next_x[k].zero();
        next_dy[k].zero();
      }
    }
    next_rstd = row < p.rows ? p.rstd[row] : 0.f;
    next_mean = row < p.rows && p.mean ? p.mean[row] : 0.f;
  };
  int64_t base = static_cast<int64_t>(blockIdx.x) * per_block;
  fetch(base + threadIdx.x / G);
  for (; base < p.rows; base += step) {
    const int64_t row = base + threadIdx.x / G;
    const float rstd = next_rstd, mu = next_mean;
    float v[P * V], g[P * V];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      next_x[k].to(v + k * V);
      next_dy[k].to(g + k * V);
    }
    fetch(row + step);
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (row < p.rows && j < n) {
        float w[V];
        load_f32<V>(p.weight, j, 1.f, w);
#pragma unroll
        for (int i = k * V; i < (k + 1) * V; ++i) {
          v[i] = (v[i] - mu) * rstd;
          if (SUMS) {
            dw[i] = fmaf(g[i], v[i], dw[i]);
            db[i] += g[i];
          }
          g[i] *= w[i - k * V];
          sg += g[i];
          sgx = fmaf(g[i], v[i], sgx);
        }
      }
    }
    total(sg, sgx);
    if (row >= p.rows) continue;
    const float mg = p.mean ? sg * inv_n : 0.f, mgx = sgx * inv_n;
    T* dx = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = rstd * (g[k * V + i] - mg - v[k * V + i] * mgx);
        store_pack<T, V>(dx + j, o);
      }
    }
  }
  // one partial row of dw and of db per block
  for (int which = 0; which < (SUMS ? 2 : 0); ++which) {
    float* part = which ? p.part_b : p.part_w;
    if (!part) continue;
    part += static_cast<int64_t>(blockIdx.x) * n;
    if (per_block == 1) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int j = (k * G + t) * V;
        if (j < n) {
#pragma unroll
          for (int i = 0; i < V; ++i) part[j + i] = which ? db[k * V + i] : dw[k * V + i];
        }
      }
      continue;
    }
    __syncthreads();
    float* mine = joined + static_cast<int64_t>(threadIdx.x / G) * n;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) mine[j + i] = which ? db[k * V + i] : dw[k * V + i];
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kNormThreads) {
      float s = 0.f;
      for (int g = 0; g < per_block; ++g) s += joined[static_cast<int64_t>(g) * n + j];
      part[j] = s;
    }
  }
}

// Rows wider than kWide: one block per row, three (two) walks over it.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 sums[8 * 32];
  GroupSum total = group_sum(sums, kNormThreads);
  const float inv_n = 1.f / p.n;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    T* y = static_cast<T*>(p.out) + row * p.ldo;
    float mu = 0.f, s = 0.f, unused = 0.f, q = 0.f;
    if (p.mean) {
      for (int j = threadIdx.x; j < p.n; j += kNormThreads) s += to_f(x[j]);
      total(s, unused);
      mu = s * inv_n;
    }
    for (int j = threadIdx.x; j < p.n; j += kNormThreads) {
      const float d = to_f(x[j]) - mu;
      q = fmaf(d, d, q);
    }
    unused = 0.f;
    total(q, unused);
    const float rstd = 1.f / sqrtf(fmaf(q, inv_n, p.eps));
    for (int j = threadIdx.x; j < p.n; j += kNormThreads)
      y[j] = from_f<T>(fmaf((to_f(x[j]) - mu) * rstd, p.weight ? p.weight[j] : 1.f, p.bias ? p.bias[j] : 0.f));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_backward_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 sums[8 * 32];
  GroupSum total = group_sum(sums, kNormThreads);
  const float inv_n = 1.f / p.n;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    T* dx = static_cast<T*>(p.out) + row * p.ldo;
    const float rstd = p.rstd[row], mu = p.mean ? p.mean[row] : 0.f;
    float sg = 0.f, sgx = 0.f;
    for (int j = threadIdx.x; j < p.n; j += kNormThreads) {
      const float g = to_f(dy[j]) * (p.weight ? p.weight[j] : 1.f);
      sg += g;
      sgx = fmaf(g, (to_f(x[j]) - mu) * rstd, sgx);
    }
    total(sg, sgx);
    const float mg = p.mean ? sg * inv_n : 0.f, mgx = sgx * inv_n;
    for (int j = threadIdx.x; j < p.n; j += kNormThreads) {
      const float g = to_f(dy[j]) * (p.weight ? p.weight[j] : 1.f);
      dx[j] = from_f<T>(rstd * (g - mg - (to_f(x[j]) - mu) * rstd * mgx));
    }
  }
}

// Partial rows of dw and db, a thread per column and blockIdx.y-th slice of the rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormParams p) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= p.n) return;
  const int64_t first = p.rows * blockIdx.y / gridDim.y, last = p.rows * (blockIdx.y + 1) / gridDim.y;
  float sw = 0.f, sb = 0.f;
  for (int64_t row = first; row < last; ++row) {
    const float g = to_f(static_cast<const T*>(p.dy)[row * p.lddy + j]);
    const float xh = (to_f(static_cast<const T*>(p.x)[row * p.ldx + j]) - (p.mean ? p.mean[row] : 0.f)) * p.rstd[row];
    sw = fmaf(g, xh, sw);
    sb += g;
  }
  if (p.part_w) p.part_w[static_cast<int64_t>(blockIdx.y) * p.n + j] = sw;
  if (p.part_b) p.part_b[static_cast<int64_t>(blockIdx.y) * p.n + j] = sb;
}

// out[j] = sum over the partial rows, in their order within each of 16 slices
// and then over the slices.  blockIdx.y: dw or db.
constexpr int kJoinSlices = 16;
__global__ void __launch_bounds__(32 * kJoinSlices)
    norm_join_kernel(const float* part_w, const float* part_b, float* dw, float* db, int parts, int n) {
  __shared__ float s[kJoinSlices][33];
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float a = 0.f;
  if (j < n) {
#pragma unroll 4
    for (int i = slice; i < parts; i += kJoinSlices) a += part[static_cast<int64_t>(i) * n + j];
  }
  s[slice][lane] = a;
  __syncthreads();
  if (slice == 0 && j < n) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinSlices; ++i) sum += s[i][lane];
    out[j] = sum;
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

muonh_status norm_fail(muonh_status st, const char* msg) {
  set_error_message(msg);
  return st;
}

int elem_size(int32_t dtype) { return dtype == MUONH_DTYPE_F32 ? 4 : 2; }

// 16-byte packs: every row of the operand starts on a 16-byte boundary and
// holds whole packs.
bool packed(const void* p, int64_t ld, int64_t n, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * size) % 16 == 0 && (n * size) % 16 == 0;
}

// Threads per row: the fewest (a power of two) that hold the row with `most`
// elements each.
int group_for(int64_t n, int most) {
  int g = 8;
  while (static_cast<int64_t>(g) * most < n) g *= 2;
  return g;
}

bool bad_dtype(int32_t d) { return d != MUONH_DTYPE_F32 && d != MUONH_DTYPE_BF16 && d != MUONH_DTYPE_F16; }

enum Pass { kForward, kBackward, kBackwardRows };   // kBackwardRows: dx alone

template <typename T, int V, int P>
cudaError_t launch_row(const NormParams& p, Pass pass, int grid, size_t smem, cudaStream_t s) {
  if (pass == kForward)
    norm_forward_kernel<T, V, P><<<grid, kNormThreads, 0, s>>>(p);
  else if (pass == kBackward)
    norm_backward_kernel<T, V, P, true><<<grid, kNormThreads, smem, s>>>(p);
  else
    norm_backward_kernel<T, V, P, false><<<grid, kNormThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(NormParams p, Pass pass, bool vec, int elems, int grid, size_t smem, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    if (elems <= V) return launch_row<T, V, 1>(p, pass, grid, smem, s);
    if (elems <= 8) return launch_row<T, V, 8 / V>(p, pass, grid, smem, s);
    return launch_row<T, V, 16 / V>(p, pass, grid, smem, s);
  }
  if (elems <= 4) return launch_row<T, 1, 4>(p, pass, grid, smem, s);
  if (elems <= 8) return launch_row<T, 1, 8>(p, pass, grid, smem, s);
  return launch_row<T, 1, 16>(p, pass, grid, smem, s);
}

cudaError_t launch(const NormParams& p, int32_t dtype, Pass pass, bool vec, int elems, int grid, size_t smem,
                   cudaStream_t s) {
  if (dtype == MUONH_DTYPE_F32) return launch_typed<float>(p, pass, vec, elems, grid, smem, s);
  if (dtype == MUONH_DTYPE_BF16) return launch_typed<__nv_bfloat16>(p, pass, vec, elems, grid, smem, s);
  return launch_typed<__half>(p, pass, vec, elems, grid, smem, s);
}

// Partial rows of dw and db from x and dy: a thread per column, `slices` shares of the rows.
cudaError_t launch_columns(const NormParams& p, int32_t dtype, int slices, cudaStream_t s) {
  const dim3 grid((p.n + 255) / 256, slices);
  if (dtype == MUONH_DTYPE_F32)
    norm_columns_kernel<float><<<grid, 256, 0, s>>>(p);
  else if (dtype == MUONH_DTYPE_BF16)
    norm_columns_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else
    norm_columns_kernel<__half><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_wide(const NormParams& p, Pass pass, int grid, cudaStream_t s) {
  if (pass == kForward)
    norm_forward_wide_kernel<T><<<grid, kNormThreads, 0, s>>>(p);
  else
    norm_backward_wide_kernel<T><<<grid, kNormThreads, 0, s>>>(p);
  return cudaGetLastError();
}

muonh_status check_rows(int64_t rows, int64_t n, int32_t dtype) {
  if (rows < 0 || n < 1 || n > INT32_MAX - kNormThreads || bad_dtype(dtype))
    return norm_fail(MUONH_ERR_INVALID_ARG, "need rows >= 0, 1 <= n < 2^31 - 512 and a MUONH_DTYPE_* type");
  return MUONH_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The kernels move single elements where a row is not 16-byte aligned.
bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" muonh_status muonh_layer_norm(const void* x, int64_t ldx, void* y, int64_t ldy, const float* weight,
                                         const float* bias, float* mean, float* rstd, int64_t rows, int64_t n,
                                         int32_t dtype, float eps, void* stream) {
  set_error_message("");
  if (const muonh_status st = check_rows(rows, n, dtype)) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return norm_fail(MUONH_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (rows == 0) return MUONH_OK;   // pointers of empty buffers may be NULL
  if (!x || !y || !rstd) return norm_fail(MUONH_ERR_INVALID_ARG, "x, y or rstd is NULL");
  if (rows > 1 && (ldx < n || ldy < n)) return norm_fail(MUONH_ERR_INVALID_ARG, "row strides must be at least n");
  const int size = elem_size(dtype);
  if (misaligned(x, size) || misaligned(y, size) || misaligned(weight, 4) || misaligned(bias, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return norm_fail(MUONH_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  NormParams p{};
  p.x = x;
  p.out = y;
  p.weight = weight;
  p.bias = bias;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.ldx = ldx;
  p.ldo = ldy;
  p.n = static_cast<int32_t>(n);
  p.eps = eps;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n > kWide) {
    const int grid = static_cast<int>(std::min<int64_t>(rows, 4ll * sm_count()));
    e = dtype == MUONH_DTYPE_F32    ? launch_wide<float>(p, kForward, grid, s)
        : dtype == MUONH_DTYPE_BF16 ? launch_wide<__nv_bfloat16>(p, kForward, grid, s)
                                    : launch_wide<__half>(p, kForward, grid, s);
  } else {
    const bool vec = packed(x, ldx, n, size) && packed(y, ldy, n, size) && aligned16(weight) && aligned16(bias);
    // 8 elements per thread leave room for three blocks per SM
    p.group = group_for(n, n <= kNormThreads * 8 ? 8 : kMaxPack);
    const int elems = static_cast<int>((n + p.group - 1) / p.group);
    const int64_t blocks = (rows + kNormThreads / p.group - 1) / (kNormThreads / p.group);
    const int grid = static_cast<int>(std::min<int64_t>(blocks, (elems <= 8 ? 3ll : 1ll) * sm_count()));   // all at once
    e = launch(p, dtype, kForward, vec, elems, grid, 0, s);
  }
  if (e != cudaSuccess) return norm_fail(MUONH_ERR_CUDA, "launch of the layer norm kernel failed");
  return MUONH_OK;
}

extern "C" size_t muonh_layer_norm_workspace(int64_t rows, int64_t n) {
  if (rows < 1 || n < 1) return 0;
  return static_cast<size_t>(std::min<int64_t>(rows, kMaxParts)) * static_cast<size_t>(n) * 2 * sizeof(float);
}

extern "C" muonh_status muonh_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                                  const float* weight, const float* mean, const float* rstd, void* dx,
                                                  int64_t lddx, float* dweight, float* dbias, int64_t rows, int64_t n,
                                                  int32_t dtype, void* workspace, size_t workspace_bytes,
                                                  void* stream) {
  set_error_message("");
  if (const muonh_status st = check_rows(rows, n, dtype)) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (misaligned(dweight, 4) || misaligned(dbias, 4))
    return norm_fail(MUONH_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  if (rows == 0) {   // the sums over no rows
    if ((dweight && cudaMemsetAsync(dweight, 0, n * sizeof(float), s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, n * sizeof(float), s) != cudaSuccess))
      return norm_fail(MUONH_ERR_CUDA, "clearing the weight gradients failed");
    return MUONH_OK;
  }
  if (!dy || !x || !rstd || !dx) return norm_fail(MUONH_ERR_INVALID_ARG, "dy, x, rstd or dx is NULL");
  if (rows > 1 && (ldx < n || lddy < n || lddx < n))
    return norm_fail(MUONH_ERR_INVALID_ARG, "row strides must be at least n");
  const int size = elem_size(dtype);
  if (misaligned(x, size) || misaligned(dy, size) || misaligned(dx, size) || misaligned(weight, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return norm_fail(MUONH_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  const bool sums = dweight || dbias;
  if (sums && (!workspace || workspace_bytes < muonh_layer_norm_workspace(rows, n)))
    return norm_fail(MUONH_ERR_INVALID_ARG, "the workspace is smaller than muonh_layer_norm_workspace says");
  if (misaligned(workspace, 4)) return norm_fail(MUONH_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  NormParams p{};
  p.x = x;
  p.dy = dy;
  p.out = dx;
  p.weight = weight;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.rows = rows;
  p.ldx = ldx;
  p.lddy = lddy;
  p.ldo = lddx;
  p.n = static_cast<int32_t>(n);
  const int sms = sm_count();
  int parts;
  cudaError_t e;
  float* part = static_cast<float*>(workspace);
  const bool vec = packed(x, ldx, n, size) && packed(dy, lddy, n, size) && packed(dx, lddx, n, size) &&
                   aligned16(weight);
  // the column sums of 16 elements per thread fit next to a prefetched row
  // only where both rows are packed 16-bit; else they come from a kernel of
  // their own (x and dy are then read twice, the second time mostly from L2)
  const int most = vec && size == 2 ? kMaxPack : 8;
  const bool split = sums && n > static_cast<int64_t>(kNormThreads) * most;
  auto set_parts = [&](int count) {   // a single partial row is the result
    parts = count;
    if (dweight) p.part_w = parts == 1 ? dweight : part;
    if (dbias) p.part_b = parts == 1 ? dbias : part + static_cast<int64_t>(parts) * n;
  };
  parts = 0;
  if (n > kWide) {
    const int grid = static_cast<int>(std::min<int64_t>(rows, 4ll * sms));
    e = dtype == MUONH_DTYPE_F32    ? launch_wide<float>(p, kBackward, grid, s)
        : dtype == MUONH_DTYPE_BF16 ? launch_wide<__nv_bfloat16>(p, kBackward, grid, s)
                                    : launch_wide<__half>(p, kBackward, grid, s);
  } else {
    p.group = group_for(n, split || !sums ? kMaxPack : most);
    const int elems = static_cast<int>((n + p.group - 1) / p.group);
    const int per_block = kNormThreads / p.group;
    const int64_t blocks = (rows + per_block - 1) / per_block;
    if (split || !sums) {
      e = launch(p, dtype, kBackwardRows, vec, elems, static_cast<int>(std::min<int64_t>(blocks, 2ll * sms)), 0, s);
    } else {
      const int grid = static_cast<int>(std::min<int64_t>({blocks, sms, static_cast<int64_t>(kMaxParts)}));
      set_parts(grid);
      const size_t smem = per_block > 1 ? static_cast<size_t>(per_block) * n * sizeof(float) : 0;
      e = launch(p, dtype, kBackward, vec, elems, grid, smem, s);
    }
  }
  if (e == cudaSuccess && split) {
    set_parts(static_cast<int>(std::min<int64_t>(rows, 64)));
    e = launch_columns(p, dtype, parts, s);
  }
  if (e == cudaSuccess && sums && parts > 1) {
    norm_join_kernel<<<dim3((static_cast<unsigned>(n) + 31) / 32, dbias ? 2 : 1), 32 * kJoinSlices, 0, s>>>(
        p.part_w, p.part_b, dweight, dbias, parts, p.n);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return norm_fail(MUONH_ERR_CUDA, "launch of a layer norm backward kernel failed");
  return MUONH_OK;
}
