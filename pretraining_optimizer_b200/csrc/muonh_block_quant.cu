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
// Bound by HBM: each element is read once and written once per orientation.  A
// block of 256 threads takes a 128 x 128 tile, 8 x 8 elements per thread in
// registers; maxima along rows come from 16 lanes' shuffles, maxima along
// columns go through shared memory, and so does the transposed copy.
#include "muonh_common.cuh"

#include <cuda_fp8.h>

namespace muonh {
namespace {

constexpr int kTile = 128;
constexpr int kQuantThreads = 256;
constexpr int kTransposedPitch = kTile + 16;   // bytes per row of the transposed tile in shared memory

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

// |v| as ordered bits: NaN above Inf above every number.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

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

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float(float v) { return v; }
template <>
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// 8 bytes of one output row; bytes behind the row's end are left as they were.
__device__ __forceinline__ void store8(uint8_t* p, uint2 v, int64_t left) {
  if (left >= 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    const uint64_t u = (static_cast<uint64_t>(v.y) << 32) | v.x;
    for (int i = 0; i < left; ++i) p[i] = static_cast<uint8_t>(u >> (8 * i));
  }
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads) block_quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t column_max[kQuantThreads / 32][kTile];
  __shared__ __align__(16) uint8_t turned[kTile * kTransposedPitch];
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;   // this thread's 8 columns and 8 rows
  const int64_t col = c0 + tc * 8;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + tr * 8 + i;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx + col;
    if (row < p.rows && p.vec && col < p.cols) {            // vec: cols is a multiple of 8
      uint4 u[sizeof(T) / 2];
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) u[k] = reinterpret_cast<const uint4*>(x)[k];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = as_float(reinterpret_cast<const T*>(u)[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = (row < p.rows && col + j < p.cols) ? as_float(x[j]) : 0.f;
    }
  }

  uint32_t m_row[8], m_col[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m_row[i] = m_col[i] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = magnitude(v[i][j]);
      m_row[i] = max(m_row[i], m);
      m_col[j] = max(m_col[j], m);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m_row[i] = max(m_row[i], __shfl_xor_sync(0xffffffffu, m_row[i], o));

  int b_row[8], b_col[8];
  if (p.whole) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, m_row[i]);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if ((threadIdx.x & 31) == 0) column_max[threadIdx.x >> 5][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, column_max[w][0]);
    const int b = scale_byte(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) b_row[i] = b_col[i] = b;
    if (threadIdx.x == 0) {
      if (p.q) p.s[blockIdx.y * p.lds + blockIdx.x] = static_cast<uint8_t>(b);
      if (p.qt) p.st[blockIdx.x * p.ldst + blockIdx.y] = static_cast<uint8_t>(b);
    }
  } else {
    if (p.q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b_row[i] = scale_byte(m_row[i]);
        const int64_t row = r0 + tr * 8 + i;
        if (tc == 0 && row < p.rows) p.s[row * p.lds + blockIdx.x] = static_cast<uint8_t>(b_row[i]);
      }
    }
    if (p.qt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = max(m_col[j], __shfl_xor_sync(0xffffffffu, m_col[j], 16));
        if ((threadIdx.x & 16) == 0) column_max[threadIdx.x >> 5][tc * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, column_max[w][tc * 8 + j]);
        b_col[j] = scale_byte(m);
        if (tr == 0 && col + j < p.cols) p.st[(col + j) * p.ldst + blockIdx.y] = static_cast<uint8_t>(b_col[j]);
      }
    }
  }

  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + tr * 8 + i;
      const float f = inverse_scale(b_row[i]);
      const uint2 u = make_uint2(to_e4m3x4(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                                 to_e4m3x4(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f));
      if (row < p.rows && col < p.cols) store8(p.q + row * p.ldq + col, u, p.cols - col);
    }
  }
  if (p.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = inverse_scale(b_col[j]);
      const uint2 u = make_uint2(to_e4m3x4(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f),
                                 to_e4m3x4(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f));
      *reinterpret_cast<uint2*>(turned + (tc * 8 + j) * kTransposedPitch + tr * 8) = u;
    }
    __syncthreads();
    // 128 rows of the transposed tile, 16 pieces of 8 bytes each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = i * 16 + tr;
      const int64_t to = c0 + row, at = r0 + tc * 8;
      if (to < p.cols && at < p.rows)
        store8(p.qt + to * p.ldqt + at, *reinterpret_cast<const uint2*>(turned + row * kTransposedPitch + tc * 8),
               p.rows - at);
    }
  }
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
  if (rows < 0 || cols < 0 || rows > (1 << 23) || cols > INT32_MAX)
    return quant_fail(MUONH_ERR_INVALID_ARG, "rows must be in [0, 2^23], cols in [0, 2^31 - 1]");
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
  const dim3 grid(static_cast<unsigned>(col_groups), static_cast<unsigned>(row_groups));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == MUONH_DTYPE_F32)
    block_quantize_kernel<float><<<grid, kQuantThreads, 0, s>>>(p);
  else if (dtype == MUONH_DTYPE_BF16)
    block_quantize_kernel<__nv_bfloat16><<<grid, kQuantThreads, 0, s>>>(p);
  else
    block_quantize_kernel<__half><<<grid, kQuantThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return quant_fail(MUONH_ERR_CUDA, "launch of block_quantize_kernel failed");
  return MUONH_OK;
}
