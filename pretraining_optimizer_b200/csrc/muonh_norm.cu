// Layer norm and RMS norm over rows, forward and backward (sm_100a).
//
//   forward    mu = <x>,  rstd = 1/sqrt(<(x - mu)^2> + eps),  y = (x - mu) rstd w + b
//   backward   xh = (x - mu) rstd,  g = dy w
//              dx = rstd (g - <g> - xh <g xh>)
//              dw = sum_rows dy xh,  db = sum_rows dy
// < > is the mean over the row; the RMS norm has mu = 0 and no <g> term.
//
// Everything is bound by HBM: the forward pass reads x and writes y once, the
// backward pass reads dy and x and writes dx once.  A group of G threads holds
// one row in registers, so a row is read once whatever the number of reductions
// over it, and its next rows are on their way meanwhile:
//   up to 32 lanes per row (n <= 256; backward, 16-bit rows in packs: 512)
//            the next row is loaded into registers
//   128 or 512 threads per row (n <= 8192) the next rows are copied to a ring in
//            shared memory (cp.async.bulk).  Prefetching such rows in registers
//            spilled, or left half of the threads: 1021 x 5003 fp32 backward took
//            57 us that way, and 35 us without any prefetch.  A row that does not
//            start on 16 bytes is copied from the 16-byte piece that it starts in.
//   wider    walked over in global memory; dw and db come from a kernel of their own.
// Backward, the dw/db sums of a thread's columns stay in registers over all rows
// of its group, the groups of a block join theirs in shared memory, each block
// writes one partial row, and a second small kernel adds the partial rows in a
// fixed order: no atomics, the same bits every time.
//
// All sums are fp32: per thread over at most 16 elements of a row (n / 512 of a wide
// one), then a tree; down the rows, over the rows that a group (of wide ones: one
// of 64 slices) takes in turn, then the join's tree.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "muonh_common.cuh"

namespace muonh {
namespace {

constexpr int kNormThreads = 512;
constexpr int kMaxPack = 16;                        // elements of a row per thread
constexpr int kWide = kNormThreads * kMaxPack;      // widest row held in registers: 8192
constexpr int kMaxParts = 512;                      // partial rows of dw/db
constexpr int kMaxRing = 4;                         // rows in flight per group
constexpr int kMaxShared = 227 * 1024;

__device__ int g_norm_timeout;                      // a wait gave up in some call since the flag was read

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
  int32_t ring, slot;        // rows in flight per group, and the bytes of one operand's row
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

// Two 16-bit values of a word as fp32, and back.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// V elements in 32-bit words, as they are in memory.
template <typename T, int V>
struct Words {
  static constexpr int kWords = V * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {   // aligned to all of them
    if constexpr (kWords == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 4)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void to(float* v) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void from(const float* v) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(v[i]);
      else
        w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
  }
};
template <typename T>
struct Words<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = w; }
  __device__ __forceinline__ void zero() { w = from_f<T>(0.f); }
  __device__ __forceinline__ void to(float* v) const { v[0] = to_f(w); }
  __device__ __forceinline__ void from(const float* v) { w = from_f<T>(v[0]); }
};
template <typename T, int V>
__device__ __forceinline__ void read_row(const T* p, float* v) {
  Words<T, V> w;
  w.load(p);
  w.to(v);
}
template <typename T, int V>
__device__ __forceinline__ void write_row(T* p, const float* v) {
  Words<T, V> w;
  w.from(v);
  w.store(p);
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

// Sums over the `group` lanes (up to 32) of a row, in each of them.
__device__ __forceinline__ float lane_sum(float a, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}
__device__ __forceinline__ void lane_sum(float& a, float& b, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
}

// Sums over the G threads (whole warps) of a row, in every thread of it: within
// the warps by shuffles, then over the warps in shared memory behind a barrier
// of the group's own.  Two slots alternate, so that one barrier per call is enough.
template <int G>
struct GroupSum {
  static constexpr int kWarps = G / 32;
  float2* slots;             // [2][kWarps] of this group
  int flip, warp, bar;
  __device__ __forceinline__ explicit GroupSum(float2* shared)   // [2 * kNormThreads / 32] of the block
      : slots(shared + threadIdx.x / G * 2 * kWarps), flip(0), warp(threadIdx.x % G / 32), bar(1 + threadIdx.x / G) {}
  template <bool kTwo>
  __device__ __forceinline__ void sum(float& a, float& b) {
    static_assert(G % 64 == 0, "two warps at least");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      if (kTwo) b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    float2* s = slots + flip;
    flip ^= kWarps;
    if ((threadIdx.x & 31) == 0) s[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(G) : "memory");
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; i += 2) {
      const float4 t = *reinterpret_cast<const float4*>(s + i);
      a += t.x;
      a += t.z;
      if (kTwo) b += t.y, b += t.w;
    }
  }
  __device__ __forceinline__ void operator()(float& a) {
    float unused = 0.f;
    sum<false>(a, unused);
  }
  __device__ __forceinline__ void operator()(float& a, float& b) { sum<true>(a, b); }
};
constexpr int kSumSlots = 2 * kNormThreads / 32;

template <typename T, int V, int P>
__global__ void __launch_bounds__(kNormThreads, 2) norm_forward_kernel(const __grid_constant__ NormParams p) {
  wait_for_stream();
  const int G = p.group, t = threadIdx.x % G, n = p.n;
  const int per_block = kNormThreads / G;
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
  Words<T, V> next[P];
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
    float mu = 0.f;
    if (p.mean) {
#pragma unroll
      for (int i = 0; i < P * V; ++i) mu += v[i];
      mu = lane_sum(mu, G) * inv_n;
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
    q = lane_sum(q, G);
    const float rstd = rsqrtf(fmaf(q, inv_n, p.eps));
    if (row >= p.rows) continue;
    T* y = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(v[k * V + i] * rstd, w[k * V + i], b[k * V + i]);
        write_row<T, V>(y + j, o);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
  }
}

// One partial row of dw and of db per block; `joined` is room for the columns
// of its groups, [kNormThreads / G][n], where it has several.
template <int V, int P>
__device__ __forceinline__ void write_parts(const NormParams& p, int G, float* joined, int t, const float (&dw)[P * V],
                                            const float (&db)[P * V]) {
  const int n = p.n, per_block = kNormThreads / G;
  for (int which = 0; which < 2; ++which) {
    float* part = which ? p.part_b : p.part_w;
    if (!part) continue;
    part += static_cast<int64_t>(blockIdx.x) * n;
    float* mine = part;
    if (per_block > 1) {
      __syncthreads();
      mine = joined + static_cast<int64_t>(threadIdx.x / G) * n;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) mine[j + i] = which ? db[k * V + i] : dw[k * V + i];
      }
    }
    if (per_block == 1) continue;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kNormThreads) {
      // in fours: one chain over up to 64 groups rounds more often where the sums cancel
      float s = 0.f;
      for (int g = 0; g < per_block; g += 4) {      // 4 groups at least
        const float* c = joined + static_cast<int64_t>(g) * n + j;
        s += (c[0] + c[n]) + (c[2 * n] + c[3 * n]);
      }
      part[j] = s;
    }
  }
}

// SUMS: also the partial rows of dw and db.
template <typename T, int V, int P, bool SUMS>
__global__ void __launch_bounds__(kNormThreads, 1) norm_backward_kernel(const __grid_constant__ NormParams p) {
  wait_for_stream();
  extern __shared__ float joined[];   // [kNormThreads / G][n]: at most kWide floats, 32 KB
  const int G = p.group, t = threadIdx.x % G, n = p.n;
  const int per_block = kNormThreads / G;
  float dw[P * V], db[P * V];
#pragma unroll
  for (int i = 0; i < P * V; ++i) dw[i] = db[i] = 0.f;
  const float inv_n = 1.f / n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  Words<T, V> next_x[P], next_dy[P];
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
    lane_sum(sg, sgx, G);
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
        write_row<T, V>(dx + j, o);
      }
    }
  }
  if constexpr (SUMS) write_parts<V, P>(p, G, joined, t, dw, db);
}

// ---- 128 or 512 threads per row: rows arrive in a ring in shared memory

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The ring of one group: `ring` slots of `kOperands` rows each.  Thread 0 of the
// group fills slot i % ring with the group's i-th row, from the 16-byte piece
// that the row starts in to the one that it ends in; a slot is filled again
// once the group has passed a barrier after reading it.
template <typename T, int kOperands, int G>
struct RowRing {
  uint8_t* base;
  uint64_t* full;            // [ring]
  int* err;
  const T* src[kOperands];
  int64_t ld[kOperands];
  int ring, slot_bytes, n;
  __device__ __forceinline__ void fill(int slot, int64_t row) {
    uint32_t total = 0;
    uintptr_t from[kOperands];
    uint32_t bytes[kOperands];
#pragma unroll
    for (int o = 0; o < kOperands; ++o) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(src[o] + row * ld[o]);
      from[o] = p & ~uintptr_t(15);
      bytes[o] = static_cast<uint32_t>(((p + n * sizeof(T) + 15) & ~uintptr_t(15)) - from[o]);
      total += bytes[o];
    }
    mbar_expect_tx(&full[slot], total);
#pragma unroll
    for (int o = 0; o < kOperands; ++o)
      bulk_load(base + (slot * kOperands + o) * slot_bytes, reinterpret_cast<const void*>(from[o]), bytes[o], &full[slot]);
  }
  // A wait that gives up records that and goes on: the group's barriers need all of its threads.
  __device__ __forceinline__ void wait(int slot, uint32_t phase) { mbar_wait(&full[slot], phase, err); }
  // After a wait that gave up, thread 0 of the group lets the copies of its last fills land (`next`: the row
  // after the group's last one).
  __device__ __forceinline__ void finish(int64_t next, int64_t first, int64_t step) {
    if (*reinterpret_cast<volatile int*>(err) == 0) return;
    const int64_t fills = (next - first) / step;
    for (int64_t i = fills > ring ? fills - ring : 0; i < fills; ++i) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&full[i % ring], static_cast<uint32_t>(i / ring) & 1) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
    atomicOr(&g_norm_timeout, 1);
  }
  // the row in the slot, once it is there
  __device__ __forceinline__ const T* at(int slot, int o, int64_t row) const {
    const uintptr_t p = reinterpret_cast<uintptr_t>(src[o] + row * ld[o]);
    return reinterpret_cast<const T*>(base + (slot * kOperands + o) * slot_bytes + (p & 15));
  }
};

// Per-block control words of the ring kernels, before the rows.
struct RingShared {
  alignas(16) float2 sums[kSumSlots];
  uint64_t full[kNormThreads / 64 * kMaxRing];
  int err;
};
constexpr int kRingOffset = (sizeof(RingShared) + 127) / 128 * 128;

template <typename T, int kOperands, int G>
__device__ __forceinline__ RowRing<T, kOperands, G> start_ring(const NormParams& p, uint8_t* smem, int64_t row, int64_t step) {
  RingShared* sh = reinterpret_cast<RingShared*>(smem);
  const int group = threadIdx.x / G;
  RowRing<T, kOperands, G> r;
  r.base = smem + kRingOffset + static_cast<size_t>(group) * p.ring * kOperands * p.slot;
  r.full = sh->full + group * kMaxRing;
  r.err = &sh->err;
  r.src[0] = static_cast<const T*>(p.x);
  r.ld[0] = p.ldx;
  if constexpr (kOperands == 2) {
    r.src[1] = static_cast<const T*>(p.dy);
    r.ld[1] = p.lddy;
  }
  r.ring = p.ring;
  r.slot_bytes = p.slot;
  r.n = p.n;
  if (threadIdx.x == 0) sh->err = 0;
  if (threadIdx.x % G == 0) {
    for (int s = 0; s < p.ring; ++s) mbar_init(&r.full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x % G == 0)
    for (int s = 0; s < p.ring && row + s * step < p.rows; ++s) r.fill(s, row + s * step);
  return r;
}

template <typename T, int V, int P, int G>
__global__ void __launch_bounds__(kNormThreads, 2) norm_forward_ring_kernel(const __grid_constant__ NormParams p) {
  wait_for_stream();
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int per_block = kNormThreads / G;
  const int t = threadIdx.x % G, n = p.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / G;
  int64_t row = first;
  GroupSum<G> total(reinterpret_cast<RingShared*>(smem)->sums);
  RowRing<T, 1, G> ring = start_ring<T, 1, G>(p, smem, row, step);
  const float inv_n = 1.f / n;
  int slot = 0;
  uint32_t phase = 0;
  for (; row < p.rows; row += step) {
    ring.wait(slot, phase);
    const T* x = ring.at(slot, 0, row);
    float v[P * V];
    float mu = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) v[k * V + i] = 0.f;
      if (j < n) read_row<T, V>(x + j, v + k * V);
    }
    if (p.mean) {
#pragma unroll
      for (int i = 0; i < P * V; ++i) mu += v[i];
      total(mu);
      mu *= inv_n;
    }
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
    total(q);
    // every thread has read the slot before that barrier
    if (t == 0 && row + ring.ring * step < p.rows) ring.fill(slot, row + ring.ring * step);
    const float rstd = rsqrtf(fmaf(q, inv_n, p.eps));
    T* y = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
        float w[V], b[V], o[V];
        load_f32<V>(p.weight, j, 1.f, w);
        load_f32<V>(p.bias, j, 0.f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(v[k * V + i] * rstd, w[i], b[i]);
        write_row<T, V>(y + j, o);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
    if (++slot == ring.ring) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (t == 0) ring.finish(row, first, step);
}

template <typename T, int V, int P, int G, bool SUMS>
__global__ void __launch_bounds__(kNormThreads, 1) norm_backward_ring_kernel(const __grid_constant__ NormParams p) {
  wait_for_stream();
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int per_block = kNormThreads / G;
  const int t = threadIdx.x % G, n = p.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / G;
  int64_t row = first;
  GroupSum<G> total(reinterpret_cast<RingShared*>(smem)->sums);
  RowRing<T, 2, G> ring = start_ring<T, 2, G>(p, smem, row, step);
  float dw[P * V], db[P * V];
#pragma unroll
  for (int i = 0; i < P * V; ++i) dw[i] = db[i] = 0.f;
  const float inv_n = 1.f / n;
  int slot = 0;
  uint32_t phase = 0;
  float next_rstd = row < p.rows ? p.rstd[row] : 0.f;
  float next_mean = row < p.rows && p.mean ? p.mean[row] : 0.f;
  for (; row < p.rows; row += step) {
    const float rstd = next_rstd, mu = next_mean;
    if (row + step < p.rows) {
      next_rstd = p.rstd[row + step];
      if (p.mean) next_mean = p.mean[row + step];
    }
    ring.wait(slot, phase);
    const T* x = ring.at(slot, 0, row);
    const T* dy = ring.at(slot, 1, row);
    float v[P * V], g[P * V];
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
#pragma unroll
      for (int i = k * V; i < (k + 1) * V; ++i) v[i] = g[i] = 0.f;
      if (j < n) {
        float w[V];
        read_row<T, V>(x + j, v + k * V);
        read_row<T, V>(dy + j, g + k * V);
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
    if (t == 0 && row + ring.ring * step < p.rows) ring.fill(slot, row + ring.ring * step);
    const float mg = p.mean ? sg * inv_n : 0.f, mgx = sgx * inv_n;
    T* dx = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int j = (k * G + t) * V;
      if (j < n) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = rstd * (g[k * V + i] - mg - v[k * V + i] * mgx);
        write_row<T, V>(dx + j, o);
      }
    }
    if (++slot == ring.ring) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (t == 0) ring.finish(row, first, step);
  __syncthreads();
  // the ring's space is free: every copy has been waited for
  if constexpr (SUMS) write_parts<V, P>(p, G, reinterpret_cast<float*>(smem + kRingOffset), t, dw, db);
}

// Rows wider than kWide: one block per row, three (two) walks over it.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_wide_kernel(const __grid_constant__ NormParams p) {
  wait_for_stream();
  __shared__ __align__(16) float2 sums[kSumSlots];
  GroupSum<kNormThreads> total(sums);
  const float inv_n = 1.f / p.n;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    T* y = static_cast<T*>(p.out) + row * p.ldo;
    float mu = 0.f, s = 0.f, q = 0.f;
    if (p.mean) {
      for (int j = threadIdx.x; j < p.n; j += kNormThreads) s += to_f(x[j]);
      total(s);
      mu = s * inv_n;
    }
    for (int j = threadIdx.x; j < p.n; j += kNormThreads) {
      const float d = to_f(x[j]) - mu;
      q = fmaf(d, d, q);
    }
    total(q);
    const float rstd = rsqrtf(fmaf(q, inv_n, p.eps));
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
  wait_for_stream();
  __shared__ __align__(16) float2 sums[kSumSlots];
  GroupSum<kNormThreads> total(sums);
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
  wait_for_stream();
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

// out[j] = sum over the partial rows: four sums within each of 16 slices, then a
// tree.  blockIdx.y: dw or db.
constexpr int kJoinSlices = 16;
__global__ void __launch_bounds__(32 * kJoinSlices)
    norm_join_kernel(const float* part_w, const float* part_b, float* dw, float* db, int parts, int n) {
  __shared__ float s[kJoinSlices][33];
  // launched while the kernel that writes the partial rows still runs
  wait_for_stream();
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  if (j < n) {
    for (int i = slice; i < parts; i += 4 * kJoinSlices)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * kJoinSlices < parts) a[k] += part[static_cast<int64_t>(i + k * kJoinSlices) * n + j];
  }
  s[slice][lane] = (a[0] + a[1]) + (a[2] + a[3]);
  __syncthreads();
  if (slice == 0 && j < n) {
    float sum[kJoinSlices];
#pragma unroll
    for (int i = 0; i < kJoinSlices; ++i) sum[i] = s[i][lane];
#pragma unroll
    for (int w = kJoinSlices / 2; w > 0; w /= 2)
#pragma unroll
      for (int i = 0; i < w; ++i) sum[i] += sum[i + w];
    out[j] = sum[0];
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

// Packs of 4 elements: the same for 4 elements' alignment.
bool fours(const void* p, int64_t ld, int64_t n, int size) {
  return (reinterpret_cast<uintptr_t>(p) & (4 * size - 1)) == 0 && ld % 4 == 0 && n % 4 == 0;
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
  if (pass == kForward) {
    if constexpr (V * P <= 8)   // the forward pass has at most 8 elements per thread here
      return launch_programmatic(norm_forward_kernel<T, V, P>, dim3(grid), kNormThreads, 0, s, p);
    return cudaErrorInvalidValue;
  }
  return pass == kBackward
             ? launch_programmatic(norm_backward_kernel<T, V, P, true>, dim3(grid), kNormThreads, smem, s, p)
             : launch_programmatic(norm_backward_kernel<T, V, P, false>, dim3(grid), kNormThreads, 0, s, p);
}

template <typename T, int V, int P, int G>
cudaError_t launch_ring(const NormParams& p, Pass pass, int grid, size_t smem, cudaStream_t s) {
  void (*kernel)(NormParams) = pass == kForward    ? norm_forward_ring_kernel<T, V, P, G>
                               : pass == kBackward ? norm_backward_ring_kernel<T, V, P, G, true>
                                                   : norm_backward_ring_kernel<T, V, P, G, false>;
  static std::atomic<uint64_t> done[3];
  const cudaError_t e = allow_shared(kernel, done[pass], kMaxShared);
  if (e != cudaSuccess) return e;
  return launch_programmatic(kernel, dim3(grid), kNormThreads, smem, s, p);
}

// 128 or 512 threads per row, with 8 or 16 elements each.  The group's size is
// a constant of the kernel: with addresses computed from a size at run time, the
// kernels were bound by their instructions (37 per element).  Half the threads
// with 32 elements each were no faster forward (24.9 against 22.6 us for 8192 x
// 2048 bf16) and slower for one row.
int ring_group(int64_t n) { return n <= 128 * kMaxPack ? 128 : 512; }
template <typename T, int V>
cudaError_t launch_rings(const NormParams& p, Pass pass, int grid, size_t smem, cudaStream_t s) {
  if (p.group == 128)
    return p.n <= 128 * 8 ? launch_ring<T, V, 8 / V, 128>(p, pass, grid, smem, s)
                          : launch_ring<T, V, 16 / V, 128>(p, pass, grid, smem, s);
  return p.n <= 512 * 8 ? launch_ring<T, V, 8 / V, 512>(p, pass, grid, smem, s)
                        : launch_ring<T, V, 16 / V, 512>(p, pass, grid, smem, s);
}

// vec: packs of 16 bytes (rows of up to 32 lanes) or of 4 elements (the ring).
template <typename T>
cudaError_t launch_typed(const NormParams& p, Pass pass, bool vec, int elems, int grid, size_t smem, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (p.group > 32) return vec ? launch_rings<T, 4>(p, pass, grid, smem, s) : launch_rings<T, 1>(p, pass, grid, smem, s);
  if (vec) {
    if (elems <= V) return launch_row<T, V, 1>(p, pass, grid, smem, s);
    if (elems <= 8) return launch_row<T, V, 8 / V>(p, pass, grid, smem, s);
    if constexpr (V == 8) return launch_row<T, 8, 2>(p, pass, grid, smem, s);
  }
  return launch_row<T, 1, 8>(p, pass, grid, smem, s);
}

cudaError_t launch(const NormParams& p, int32_t dtype, Pass pass, bool vec, int elems, int grid, size_t smem,
                   cudaStream_t s) {
  if (dtype == MUONH_DTYPE_F32) return launch_typed<float>(p, pass, vec, elems, grid, smem, s);
  if (dtype == MUONH_DTYPE_BF16) return launch_typed<__nv_bfloat16>(p, pass, vec, elems, grid, smem, s);
  return launch_typed<__half>(p, pass, vec, elems, grid, smem, s);
}

// Sizes p's ring; returns the dynamic shared memory.  `budget` bytes per block;
// two rows at least.
size_t size_ring(NormParams* p, int operands, int size, size_t budget) {
  const size_t groups = kNormThreads / p->group;
  p->slot = static_cast<int32_t>((static_cast<size_t>(p->n) * size + 15) / 16 * 16 + 16);
  p->ring = static_cast<int32_t>(std::max<size_t>(2, std::min<size_t>(kMaxRing, budget / (groups * operands * p->slot))));
  const size_t rows = groups * p->ring * operands * p->slot;
  const size_t joined = groups > 1 && operands == 2 ? groups * p->n * sizeof(float) : 0;
  return kRingOffset + std::max(rows, joined);
}

// Partial rows of dw and db from x and dy: a thread per column, `slices` shares of the rows.
cudaError_t launch_columns(const NormParams& p, int32_t dtype, int slices, cudaStream_t s) {
  const dim3 grid((p.n + 255) / 256, slices);
  void (*kernel)(NormParams) = dtype == MUONH_DTYPE_F32    ? norm_columns_kernel<float>
                               : dtype == MUONH_DTYPE_BF16 ? norm_columns_kernel<__nv_bfloat16>
                                                           : norm_columns_kernel<__half>;
  return launch_programmatic(kernel, grid, 256, 0, s, p);
}

template <typename T>
cudaError_t launch_wide(const NormParams& p, Pass pass, int grid, cudaStream_t s) {
  return launch_programmatic(pass == kForward ? norm_forward_wide_kernel<T> : norm_backward_wide_kernel<T>, dim3(grid),
                             kNormThreads, 0, s, p);
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
    // 8 elements per thread of rows within a warp, 16 beyond: both leave room for two blocks per SM
    p.group = group_for(n, 8);
    size_t smem = 0;
    bool vec;
    if (p.group > 32) {
      p.group = ring_group(n);
      vec = fours(x, ldx, n, size) && fours(y, ldy, n, size) && aligned16(weight) && aligned16(bias);
      smem = size_ring(&p, 1, size, 100 * 1024);
    } else {
      vec = packed(x, ldx, n, size) && packed(y, ldy, n, size) && aligned16(weight) && aligned16(bias);
    }
    const int elems = static_cast<int>((n + p.group - 1) / p.group);
    const int64_t blocks = (rows + kNormThreads / p.group - 1) / (kNormThreads / p.group);
    const int grid = static_cast<int>(std::min<int64_t>(blocks, 2ll * sm_count()));   // all at once
    e = launch(p, dtype, kForward, vec, elems, grid, smem, s);
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
    if (e == cudaSuccess && sums) {
      set_parts(static_cast<int>(std::min<int64_t>(rows, 64)));
      e = launch_columns(p, dtype, parts, s);
    }
  } else {
    // rows within a warp: 16 packed 16-bit elements per thread fit in the
    // registers next to the column sums and the next row, 8 of the others
    bool vec = packed(x, ldx, n, size) && packed(dy, lddy, n, size) && packed(dx, lddx, n, size) && aligned16(weight);
    p.group = group_for(n, vec && size == 2 ? kMaxPack : 8);
    size_t smem = 0;
    if (p.group > 32) {
      p.group = ring_group(n);
      vec = fours(x, ldx, n, size) && fours(dy, lddy, n, size) && fours(dx, lddx, n, size) && aligned16(weight);
      smem = size_ring(&p, 2, size, 200 * 1024);
    } else if (sums && p.group < kNormThreads) {
      smem = static_cast<size_t>(kNormThreads / p.group) * n * sizeof(float);
    }
    const int elems = static_cast<int>((n + p.group - 1) / p.group);
    const int per_block = kNormThreads / p.group;
    const int grid = static_cast<int>(
        std::min<int64_t>({(rows + per_block - 1) / per_block, sms, static_cast<int64_t>(kMaxParts)}));
    if (sums) set_parts(grid);
    e = launch(p, dtype, sums ? kBackward : kBackwardRows, vec, elems, grid, smem, s);
  }
  if (e == cudaSuccess && sums && parts > 1) {
    e = launch_programmatic(norm_join_kernel, dim3((static_cast<unsigned>(n) + 31) / 32, dbias ? 2 : 1),
                            32 * kJoinSlices, 0, s, p.part_w, p.part_b, dweight, dbias, parts, p.n);
  }
  if (e != cudaSuccess) return norm_fail(MUONH_ERR_CUDA, "launch of a layer norm backward kernel failed");
  return MUONH_OK;
}

cudaError_t muonh::take_norm_timeout(int* flag, cudaStream_t s) { return take_flag(g_norm_timeout, flag, s); }
