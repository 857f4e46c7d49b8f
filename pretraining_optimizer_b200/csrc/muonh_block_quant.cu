// Quantising to 8 bits with one power-of-two scale per block of 128 (sm_100a).
//
// The recipe's linear layers (Puro-2B report: blockwise e4m3, activations and
// gradients in 1 x 128 groups, weights in 128 x 128 blocks, E8M0 scales): for a
// block with the largest magnitude m
//   k = the smallest integer >= -127 with m <= 448 2^k   (0 for a block of zeros)
//   q = round(x 2^-k) to e4m3 (ties to even),  scale byte = k + 127.
// Both are exact functions of x: k comes from the bits of m, and the product
// with a power of two is exact.  A block that holds NaN or Inf gets scale byte
// 255 (NaN in E8M0) and NaN throughout.
//
// Bound by HBM: each element is read once and written once per orientation.
// Rows alone need no tile: 16 lanes take a group of 128, four groups per thread
// in flight.  For both orientations a block of 256 threads takes a 128 x 128
// tile, 8 x 8 elements per thread in registers; maxima along rows come from 16
// lanes' shuffles, maxima along columns go through shared memory, and so does
// the transposed copy, its 8-byte pieces swizzled so that neither its writes
// (down a column of pieces) nor its reads (along a row) meet in a bank.
#include "muonh_common.cuh"

#include <cuda_fp8.h>

#include <type_traits>

namespace muonh {
namespace {

constexpr int kTile = 128;
constexpr int kQuantThreads = 256;
constexpr int kRowsPerThread = 4;              // rows alone: groups in flight per thread

struct QuantParams {
  const void* x;
  int64_t ldx, rows, cols;
  uint8_t* q;                // rows x cols, or null
  uint8_t* qt;               // cols x rows, or null
  uint8_t* s;                // scales of q: one per row (or per 128 rows) and 128 columns
  uint8_t* st;
  int64_t ldq, ldqt, lds, ldst;
  int32_t whole;             // 1: one scale per 128 x 128 block
  int32_t vec;               // 16-byte loads of x
};

// Scale byte of a block whose largest magnitude has the bits m.
// m = 1.f x 2^e <= 448 2^k = 1.75 x 2^(8 + k): k = e - 8, plus one where 1.f > 1.75.
__device__ __forceinline__ int scale_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 255;
  if (m == 0u) return 127;
  const int b = static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0 : b;
}
__device__ __forceinline__ float inverse_scale(int byte) {   // 2^-(byte - 127); NaN for the NaN scale
  return byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The first `left` elements of 16 bytes, one by one, and zeros.  (Rare where speed
// counts: a function of its own, by value, keeps it out of the fast path.)
template <typename T>
__device__ __noinline__ uint4 load_tail(const T* p, int64_t left) {
  using Bits = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
  const Bits* b = reinterpret_cast<const Bits*>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < static_cast<int>(16 / sizeof(T)); ++j)
    if (j < left) w[j * sizeof(T) / 4] |= static_cast<uint32_t>(b[j]) << (sizeof(T) == 2 ? 16 * (j & 1) : 0);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// An 8-element piece of a row as it was loaded.
template <typename T>
struct Piece {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
  // `vec`: p is 16-byte aligned and all 8 elements exist; else the first `left`, the others zero
  __device__ __forceinline__ void load(const T* p, bool vec, int64_t left) {
    if (vec) {
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[k];
        w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) {
      const uint4 u = load_tail<T>(p + k * (16 / sizeof(T)), left - static_cast<int64_t>(k * (16 / sizeof(T))));
      w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0u;
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    const uint32_t u = w[j >> 1];
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
    const __half2 h = *reinterpret_cast<const __half2*>(&u);
    return (j & 1) ? __high2float(h) : __low2float(h);
  }
};

// Magnitudes in the type's own bits, ordered (NaN above Inf above numbers): one
// 32-bit word per fp32 element, two 16-bit halves otherwise.
template <typename T>
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
  return w & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  return sizeof(T) == 4 ? max(a, b) : __vmaxs2(a, b);
}
// Those bits of one element as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
}

// The first `left` (below 8) bytes of one output piece; what is behind the row's
// end is left as it was.  A function of its own: it is rare, and its code would
// crowd the others out of the instruction cache.
__device__ __noinline__ void store_tail(uint8_t* p, uint2 v, int left) {
  const uint64_t u = (static_cast<uint64_t>(v.y) << 32) | v.x;
  for (int i = 0; i < left; ++i) p[i] = static_cast<uint8_t>(u >> (8 * i));
}
__device__ __forceinline__ void store8(uint8_t* p, uint2 v, int64_t left) {
  if (left >= 8)
    *reinterpret_cast<uint2*>(p) = v;
  else if (left > 0)
    store_tail(p, v, static_cast<int>(left));
}

template <typename T>
__device__ __forceinline__ uint2 quantize_row(const Piece<T>& v, float f) {
  return make_uint2(to_e4m3x4(v.at(0) * f, v.at(1) * f, v.at(2) * f, v.at(3) * f),
                    to_e4m3x4(v.at(4) * f, v.at(5) * f, v.at(6) * f, v.at(7) * f));
}

// Groups of 128 along the rows alone; groups are numbered row by row.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) block_quantize_rows_kernel(const __grid_constant__ QuantParams p) {
  wait_for_stream();
  const uint32_t per_row = static_cast<uint32_t>((p.cols + kTile - 1) / kTile);
  const uint32_t total = static_cast<uint32_t>(p.rows) * per_row;   // below 2^31
  const uint32_t first = blockIdx.x * (kRowsPerThread * kQuantThreads / 16) + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  Piece<T> v[kRowsPerThread];
  int64_t row[kRowsPerThread], col[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const uint32_t u = first + i * (kQuantThreads / 16);
    const uint32_t r = u / per_row;
    row[i] = u < total ? r : p.rows;
    col[i] = static_cast<int64_t>(u - r * per_row) * kTile + lane * 8;
    if (row[i] < p.rows)
      v[i].load(static_cast<const T*>(p.x) + row[i] * p.ldx + col[i], p.vec && col[i] < p.cols, p.cols - col[i]);
    else
      v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < Piece<T>::kWords; ++k) m = larger<T>(m, magnitudes<T>(v[i].w[k]));
    if (sizeof(T) == 2) m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int b = scale_byte(as_f32_bits<T>(m));
    if (row[i] >= p.rows) continue;
    if (lane == 0) p.s[row[i] * p.lds + col[i] / kTile] = static_cast<uint8_t>(b);
    store8(p.q + row[i] * p.ldq + col[i], quantize_row(v[i], inverse_scale(b)), p.cols - col[i]);
  }
}

__device__ __forceinline__ uint32_t turned_piece(int row, int piece) {
  return static_cast<uint32_t>(row * kTile + ((piece ^ ((row >> 3) & 15)) << 3));
}

// Maxima along the rows of eight values per lane over 16 lanes: lane l ends
// with that of row (l >> 1) & 7 (8 shuffles, each halving what is left, in place of 32).
__device__ __forceinline__ uint32_t row_maxima(const uint32_t (&m)[8]) {
  const int lane = threadIdx.x & 15;
  uint32_t a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t keep = (lane & 8) ? m[i + 4] : m[i], give = (lane & 8) ? m[i] : m[i + 4];
    a[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, 8));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t keep = (lane & 4) ? a[i + 2] : a[i], give = (lane & 4) ? a[i] : a[i + 2];
    b[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, 4));
  }
  const uint32_t keep = (lane & 2) ? b[1] : b[0], give = (lane & 2) ? b[0] : b[1];
  const uint32_t c = max(keep, __shfl_xor_sync(0xffffffffu, give, 2));
  return max(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 3 : 2)
    block_quantize_kernel(const __grid_constant__ QuantParams p) {
  wait_for_stream();
  constexpr int kWords = Piece<T>::kWords;
  constexpr int kColumnWords = kTile / 8 * kWords;   // a row of the tile
  __shared__ uint32_t column_max[kQuantThreads / 32][kColumnWords];
  __shared__ __align__(16) float column_factor[kTile];
  __shared__ __align__(16) uint8_t turned[kTile * kTile];
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;   // this thread's 8 columns and 8 rows
  const int64_t col = c0 + tc * 8, row0 = r0 + tr * 8;

  Piece<T> v[8];
  {
    const T* x = static_cast<const T*>(p.x) + row0 * p.ldx + col;
#pragma unroll
    for (int i = 0; i < 8; ++i, x += p.ldx) {
      if (row0 + i < p.rows)
        v[i].load(x, p.vec && col < p.cols, p.cols - col);
      else
        v[i].zero();
    }
  }

  uint32_t m_row[8], m_col[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) m_col[k] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m_row[i] = 0u;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t m = magnitudes<T>(v[i].w[k]);
      m_row[i] = larger<T>(m_row[i], m);
      m_col[k] = larger<T>(m_col[k], m);
    }
    if (sizeof(T) == 2) m_row[i] = max(m_row[i] & 0xffffu, m_row[i] >> 16);
  }

  float f_row[8], f_col[8];
  if (p.whole) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, m_row[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) column_max[threadIdx.x >> 5][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, column_max[w][0]);
    const int b = scale_byte(as_f32_bits<T>(m));
    const float f = inverse_scale(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) f_row[i] = f_col[i] = f;
    if (threadIdx.x == 0) {
      if (p.q) p.s[blockIdx.y * p.lds + blockIdx.x] = static_cast<uint8_t>(b);
      if (p.qt) p.st[blockIdx.x * p.ldst + blockIdx.y] = static_cast<uint8_t>(b);
    }
  } else {
    if (p.qt) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const uint32_t m = larger<T>(m_col[k], __shfl_xor_sync(0xffffffffu, m_col[k], 16));
        if ((threadIdx.x & 16) == 0) column_max[threadIdx.x >> 5][tc * kWords + k] = m;
      }
    }
    if (p.q) {
      const int mine = (tc >> 1) & 7;
      const int b = scale_byte(as_f32_bits<T>(row_maxima(m_row)));
      if ((tc & 1) == 0 && row0 + mine < p.rows) p.s[(row0 + mine) * p.lds + blockIdx.x] = static_cast<uint8_t>(b);
      const float f = inverse_scale(b);
      // row i's factor is in lane 2 i: bit 2 of i was split by xor 8, bit 1 by xor 4, bit 0 by xor 2
#pragma unroll
      for (int i = 0; i < 8; ++i) f_row[i] = __shfl_sync(0xffffffffu, f, (threadIdx.x & 16) + 2 * i);
    }
    if (p.qt) {
      // one thread per column (16-bit: its half of a word)
      __syncthreads();
      if (threadIdx.x < kTile) {
        const int j = threadIdx.x;
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < kQuantThreads / 32; ++w)
          m = larger<T>(m, column_max[w][sizeof(T) == 4 ? j : j >> 1]);
        if (sizeof(T) == 2) m = (j & 1) ? m >> 16 : m & 0xffffu;
        const int b = scale_byte(as_f32_bits<T>(m));
        column_factor[j] = inverse_scale(b);
        if (c0 + j < p.cols) p.st[(c0 + j) * p.ldst + blockIdx.y] = static_cast<uint8_t>(b);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(column_factor + tc * 8 + j);
        f_col[j] = f.x, f_col[j + 1] = f.y, f_col[j + 2] = f.z, f_col[j + 3] = f.w;
      }
    }
  }

  if (p.q) {
    uint8_t* q = p.q + row0 * p.ldq + col;
#pragma unroll
    for (int i = 0; i < 8; ++i, q += p.ldq)
      if (row0 + i < p.rows) store8(q, quantize_row(v[i], f_row[i]), p.cols - col);
  }
  if (p.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = f_col[j];
      const uint2 u = make_uint2(to_e4m3x4(v[0].at(j) * f, v[1].at(j) * f, v[2].at(j) * f, v[3].at(j) * f),
                                 to_e4m3x4(v[4].at(j) * f, v[5].at(j) * f, v[6].at(j) * f, v[7].at(j) * f));
      *reinterpret_cast<uint2*>(turned + turned_piece(tc * 8 + j, tr)) = u;
    }
    __syncthreads();
    // 128 rows of the transposed tile, 16 pieces of 8 bytes each
    uint8_t* qt = p.qt + (c0 + tr) * p.ldqt + r0 + tc * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i, qt += 16 * p.ldqt) {
      const int row = i * 16 + tr;
      if (c0 + row < p.cols)
        store8(qt, *reinterpret_cast<const uint2*>(turned + turned_piece(row, tc)), p.rows - r0 - tc * 8);
    }
  }
}

template <typename T>
cudaError_t launch_quantize(const QuantParams& p, int64_t row_groups, int64_t col_groups, cudaStream_t s) {
  if (!p.whole && !p.qt) {
    const int64_t groups = p.rows * col_groups, per_block = kRowsPerThread * kQuantThreads / 16;
    return launch_programmatic(block_quantize_rows_kernel<T>, dim3(static_cast<unsigned>((groups + per_block - 1) / per_block)),
                               kQuantThreads, 0, s, p);
  }
  return launch_programmatic(block_quantize_kernel<T>,
                             dim3(static_cast<unsigned>(col_groups), static_cast<unsigned>(row_groups)), kQuantThreads, 0,
                             s, p);
}

muonh_status quant_fail(muonh_status st, const char* msg) {
  set_error_message(msg);
  return st;
}

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" muonh_status muonh_block_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int32_t dtype,
                                             int32_t block_rows, void* q, int64_t ldq, uint8_t* scale,
                                             int64_t ld_scale, void* qt, int64_t ldqt, uint8_t* scale_t,
                                             int64_t ld_scale_t, void* stream) {
  set_error_message("");
  if (rows < 0 || cols < 0 || rows > 65535 * kTile || cols > INT32_MAX || rows * ((cols + kTile - 1) / kTile) > INT32_MAX)
    return quant_fail(MUONH_ERR_INVALID_ARG, "rows must be in [0, 128 * 65535], with fewer than 2^31 groups of 128 in them");
  if (dtype != MUONH_DTYPE_F32 && dtype != MUONH_DTYPE_BF16 && dtype != MUONH_DTYPE_F16)
    return quant_fail(MUONH_ERR_INVALID_ARG, "dtype must be a MUONH_DTYPE_* type");
  if (block_rows != 1 && block_rows != kTile) return quant_fail(MUONH_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (rows == 0 || cols == 0) return MUONH_OK;
  if (!x || (!q && !qt) || (q && !scale) || (qt && !scale_t))
    return quant_fail(MUONH_ERR_INVALID_ARG, "need x, q or qt, and the scales of each");
  const int64_t row_groups = (rows + kTile - 1) / kTile, col_groups = (cols + kTile - 1) / kTile;
  if ((rows > 1 && ldx < cols) || (q && rows > 1 && ldq < cols) || (qt && cols > 1 && ldqt < rows) ||
      (q && ld_scale < col_groups) || (qt && ld_scale_t < row_groups))
    return quant_fail(MUONH_ERR_INVALID_ARG, "a row stride is smaller than its rows");
  const int size = dtype == MUONH_DTYPE_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) & (size - 1)) ||
      (q && ((reinterpret_cast<uintptr_t>(q) & 15) || (rows > 1 && ldq % 16))) ||
      (qt && ((reinterpret_cast<uintptr_t>(qt) & 15) || (cols > 1 && ldqt % 16))))
    return quant_fail(MUONH_ERR_ALIGNMENT, "q and qt need 16-byte aligned rows, x its type's alignment");
  QuantParams p{};
  p.x = x;
  p.ldx = ldx;
  p.rows = rows;
  p.cols = cols;
  p.q = static_cast<uint8_t*>(q);
  p.qt = static_cast<uint8_t*>(qt);
  p.s = scale;
  p.st = scale_t;
  p.ldq = ldq;
  p.ldqt = ldqt;
  p.lds = ld_scale;
  p.ldst = ld_scale_t;
  p.whole = block_rows == kTile;
  p.vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (rows == 1 || ldx * size % 16 == 0) && cols % 8 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MUONH_DTYPE_F32    ? launch_quantize<float>(p, row_groups, col_groups, s)
                        : dtype == MUONH_DTYPE_BF16 ? launch_quantize<__nv_bfloat16>(p, row_groups, col_groups, s)
                                                    : launch_quantize<__half>(p, row_groups, col_groups, s);
  if (e != cudaSuccess) return quant_fail(MUONH_ERR_CUDA, "launch of block_quantize_kernel failed");
  return MUONH_OK;
}
