// Orthogonalising stacks of matrices with a small side where fp16 pairs do not
// hold the r x r iteration (muonh_orth.cu; ns_chain_run says where): long runs
// and coefficients that grow.  The same formulas in fp64, in runs of at most the
// factors that pairs would hold:
//   Y = s X;  per run: A = Y Y^T;  P = a I + b A + c A^2,  T = A P,  A <- T P,  Q <- Q P;  Y <- Q Y.
// Without the restarts an asymmetry of A (1e-16) grows with the square of the
// product's growth: 16 default steps in one run were off by 2e-3 on a matrix of
// rank one, and are by 5e-8 in runs of five.  Y is kept in fp64 between runs.
//
// All of it is products with at most 128 rows: 64 x 64 tiles by four warps of 32 x 32
// (mma m8n8k4 in fp64), the next 16 of k on their way in registers meanwhile, the
// r x r matrices and Y in the caller's scratch.  Y and O are written in blocks of
// 32 positions of the long side that were read whole before, so Y is updated in
// place and O may replace X.  X is read element by element at whatever stride, so
// no stack is copied first.
// 896 x [128, 2048] bf16: 22 ms for 6 steps, 24 for 8 (300 GFLOP: 14 of the card's
// 36 TFLOPS; the fp32 operations of PyTorch take 21 and 27), one such matrix 0.32
// and 0.41 ms (0.49 and 0.6), a product of r x r matrices 12 us of it.  Five steps
// in pairs take 0.4 and 0.04 ms: this is for what they cannot hold.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "muonh_common.cuh"

namespace muonh {
namespace {

constexpr int kSideMax = 128;
constexpr int kTile64 = 64;                      // side of a tile
constexpr int kSlab = 16;                        // k per round
constexpr int kPitch = kTile64 + 8;              // so a fragment's four rows fall in the two halves of the banks in turn
constexpr int kTileThreads = 128;
constexpr int kEach = kTile64 * kSlab / kTileThreads;   // elements of an operand per thread and round
constexpr int kPositions = 32;                   // of the long side per block of long_apply_kernel
constexpr int kApplyThreads = 256;
constexpr int kPitchX = kPositions + 8, kPitchQ = kSideMax + 8;
constexpr int kApplySmem = (kSideMax * kPitchX + kSlab * kPitchQ) * 8;
constexpr int kJoinThreads = 256, kJoinBlocks = 8;
// Few matrices share the long side of the Gram products among blocks, up to
// kTargetBlocks of them, with 8 slabs each at least ([128, 2048] alone: 276 us
// without, 21 with).
constexpr int kMaxShares = 16, kTargetBlocks = 128;
// Scratch of a part of the stack (one matrix at least): 97 [128, 2048] matrices, 290 blocks of the Gram
// products.  With 64 MB, which L2 would hold, the SMs were half empty.
constexpr int64_t kScratchBytes = int64_t(256) << 20;
constexpr int kMatrices = 5;                     // A, P, T and two of Q

// One part of the stack: matrices first .. first + grid.y of it.
struct LongParams {
  const uint16_t* x;
  uint16_t* out;
  int64_t x_stride, ldx, out_stride, ldo;
  int64_t length;            // the long side
  // kMatrices stacks of r x r, `shares` more for the Gram products' shares, s of
  // each matrix, and Y, r x length, where there is a restart
  double* scratch;
  int64_t part;              // matrices in a stack of the scratch
  int32_t shares;            // of the long side
  int32_t r, tall, bf16;
  float a, b, c, eps;
};

__device__ __forceinline__ double* stack_at(const LongParams& p, int which) {
  return p.scratch + (static_cast<int64_t>(which) * p.part + blockIdx.y) * p.r * p.r;
}
__device__ __forceinline__ double* scale_at(const LongParams& p) {
  return p.scratch + static_cast<int64_t>(kMatrices + p.shares) * p.part * p.r * p.r + blockIdx.y;
}
__device__ __forceinline__ double* y_at(const LongParams& p) {
  return p.scratch + static_cast<int64_t>(kMatrices + p.shares) * p.part * p.r * p.r + p.part + blockIdx.y * p.length * p.r;
}
__device__ __forceinline__ float value(const LongParams& p, uint16_t u) {
  return p.bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}
// Element (i, j) of the wide orientation of Y, or the bits of X's.
template <bool kY>
__device__ __forceinline__ auto element(const LongParams& p, int i, int64_t j) {
  if constexpr (kY) {
    return y_at(p)[i * p.length + j];
  } else {
    const uint16_t* x = p.x + blockIdx.y * p.x_stride;
    return p.tall ? x[j * p.ldx + i] : x[i * p.ldx + j];
  }
}
__device__ __forceinline__ double number(const LongParams&, double v) { return v; }
__device__ __forceinline__ double number(const LongParams& p, uint16_t v) { return value(p, v); }

// D += A B for one 8 x 4 by 4 x 8 product: a = A[lane / 4][lane % 4], b = B[lane % 4][lane / 4],
// d = D[lane / 4][2 (lane % 4) + 0, 1].
__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(d[0]), "+d"(d[1])
               : "d"(a), "d"(b));
}

// A 64 x 64 tile of a product over k from `begin` to `depth`: left(k, row) and
// right(k, column) give the operands' elements as they lie in memory (0 outside;
// converted only once the round before is through, so that its MMAs do not wait for
// them), done(row, column, value) takes each result.  `across`: consecutive threads
// load along rows and columns rather than along k.
template <typename Raw, typename Left, typename Right, typename Done>
__device__ __forceinline__ void tile_product(const LongParams& p, int64_t begin, int64_t depth, bool left_across,
                                             bool right_across, Left left, Right right, Done done) {
  __shared__ double l[kSlab][kPitch], r[kSlab][kPitch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = (warp >> 1) * 32, j0 = (warp & 1) * 32;
  auto place = [&](bool across, int n, int& k, int& i) {
    const int e = n * kTileThreads + threadIdx.x;
    k = across ? e / kTile64 : e % kSlab;
    i = across ? e % kTile64 : e / kSlab;
  };
  Raw nl[kEach], nr[kEach];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      int k, i;
      place(left_across, n, k, i);
      nl[n] = k0 + k < depth ? left(k0 + k, i) : Raw(0);
      place(right_across, n, k, i);
      nr[n] = k0 + k < depth ? right(k0 + k, i) : Raw(0);
    }
  };
  double v[4][4][2] = {};
  fetch(begin);
  for (int64_t k0 = begin; k0 < depth; k0 += kSlab) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      int k, i;
      place(left_across, n, k, i);
      l[k][i] = number(p, nl[n]);
      place(right_across, n, k, i);
      r[k][i] = number(p, nr[n]);
    }
    __syncthreads();
    fetch(k0 + kSlab);
#pragma unroll
    for (int k = 0; k < kSlab; k += 4) {
      double a[4], b[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        a[n] = l[k + (lane & 3)][i0 + 8 * n + (lane >> 2)];
        b[n] = r[k + (lane & 3)][j0 + 8 * n + (lane >> 2)];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f64(v[i][j], a[i], b[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) done(i0 + 8 * i + (lane >> 2), j0 + 8 * j + 2 * (lane & 3) + h, v[i][j][h]);
}

// The shares (blockIdx.z) of A = X X^T or Y Y^T: the tiles (0, 0), (0, 1) and (1, 1), each with its mirror.
template <bool kY>
__global__ void __launch_bounds__(kTileThreads) long_gram_kernel(const __grid_constant__ LongParams p) {
  wait_for_stream();
  const int i0 = blockIdx.x == 2 ? kTile64 : 0, j0 = blockIdx.x == 0 ? 0 : kTile64;
  const bool across = !kY && p.tall;
  double* out = stack_at(p, kMatrices + blockIdx.z);
  const int64_t slabs = (p.length + kSlab - 1) / kSlab;
  const int64_t begin = slabs * blockIdx.z / p.shares * kSlab;
  const int64_t end = min(slabs * (blockIdx.z + 1) / p.shares * kSlab, p.length);
  using Raw = typename std::conditional<kY, double, uint16_t>::type;
  tile_product<Raw>(
      p, begin, end, across, across,
      [&](int64_t k, int i) { return i0 + i < p.r ? element<kY>(p, i0 + i, k) : Raw(0); },
      [&](int64_t k, int j) { return j0 + j < p.r ? element<kY>(p, j0 + j, k) : Raw(0); },
      [&](int i, int j, double v) {
        if (i0 + i >= p.r || j0 + j >= p.r) return;
        out[(i0 + i) * p.r + j0 + j] = v;
        if (i0 != j0) out[(j0 + j) * p.r + i0 + i] = v;
      });
}

// A, the sum of its shares.  kFirst: and s = 1 / (||X|| + eps) from the trace (0 for zeros without eps, NaN where
// X has NaN or Inf), and A s^2.
template <bool kFirst>
__global__ void __launch_bounds__(kJoinThreads) long_join_kernel(const __grid_constant__ LongParams p) {
  wait_for_stream();
  __shared__ double diagonal[kSideMax];
  const int64_t stride = p.part * p.r * p.r;
  const double* share = stack_at(p, kMatrices);
  auto sum = [&](int i) {
    double v = 0.0;
    for (int n = 0; n < p.shares; ++n) v += share[n * stride + i];
    return v;
  };
  double s = 1.0;
  if (kFirst) {
    for (int i = threadIdx.x; i < kSideMax; i += kJoinThreads) diagonal[i] = i < p.r ? sum(i * p.r + i) : 0.0;
    for (int w = kSideMax / 2; w > 0; w /= 2) {
      __syncthreads();
      if (threadIdx.x < w) diagonal[threadIdx.x] += diagonal[threadIdx.x + w];
    }
    __syncthreads();
    const double norm = sqrt(diagonal[0]) + static_cast<double>(p.eps);
    s = !isfinite(norm) ? nan("") : norm > 0.0 ? 1.0 / norm : 0.0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *scale_at(p) = s;
  }
  double* a = stack_at(p, 0);
  for (int i = blockIdx.x * kJoinThreads + threadIdx.x; i < p.r * p.r; i += kJoinBlocks * kJoinThreads) a[i] = sum(i) * s * s;
}

// Stack `out` = L R of the stacks `left` and `right`, or, with kFactor, a I + b L + c L L.
template <bool kFactor>
__global__ void __launch_bounds__(kTileThreads)
    long_product_kernel(const __grid_constant__ LongParams p, int left, int right, int out) {
  wait_for_stream();
  const int side = (p.r + kTile64 - 1) / kTile64;
  const int i0 = blockIdx.x / side * kTile64, j0 = blockIdx.x % side * kTile64;
  const double *lm = stack_at(p, left), *rm = stack_at(p, right);
  double* to = stack_at(p, out);
  tile_product<double>(
      p, 0, p.r, false, true,
      [&](int64_t k, int i) { return i0 + i < p.r ? lm[(i0 + i) * p.r + k] : 0.0; },
      [&](int64_t k, int j) { return j0 + j < p.r ? rm[k * p.r + j0 + j] : 0.0; },
      [&](int i, int j, double v) {
        const int row = i0 + i, col = j0 + j;
        if (row >= p.r || col >= p.r) return;
        if (kFactor) v = (row == col ? static_cast<double>(p.a) : 0.0) + p.b * lm[row * p.r + col] + p.c * v;
        to[row * p.r + col] = v;
      });
}

// Q times X (kFirst: and s) or Y, to O (kLast) or Y, for kPositions of the long side: all of their inputs first.
// Eight warps: 32 rows by 16 positions each.
template <bool kFirst, bool kLast>
__global__ void __launch_bounds__(kApplyThreads) long_apply_kernel(const __grid_constant__ LongParams p, int q) {
  wait_for_stream();
  extern __shared__ double apply_smem[];
  double(*x)[kPitchX] = reinterpret_cast<double(*)[kPitchX]>(apply_smem);                          // [kSideMax]
  double(*qs)[kPitchQ] = reinterpret_cast<double(*)[kPitchQ]>(apply_smem + kSideMax * kPitchX);    // [kSlab]
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kPositions;
  const int depth = (p.r + kSlab - 1) / kSlab * kSlab;
  const bool tall_in = kFirst && p.tall, tall_out = kLast && p.tall;
#pragma unroll 4
  for (int n = 0; n < kSideMax * kPositions / kApplyThreads; ++n) {
    const int e = n * kApplyThreads + threadIdx.x;
    const int i = tall_in ? e % kSideMax : e / kPositions, j = tall_in ? e / kSideMax : e % kPositions;
    if (i < depth) x[i][j] = i < p.r && j0 + j < p.length ? number(p, element<!kFirst>(p, i, j0 + j)) : 0.0;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = (warp >> 1) * 32, col0 = (warp & 1) * 16;
  const double* qm = stack_at(p, q);
  double v[4][2][2] = {};
  for (int k0 = 0; k0 < depth; k0 += kSlab) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kSlab * kSideMax / kApplyThreads; ++n) {
      const int e = n * kApplyThreads + threadIdx.x, k = e % kSlab, i = e / kSlab;
      qs[k][i] = i < p.r && k0 + k < p.r ? qm[i * p.r + k0 + k] : 0.0;
    }
    __syncthreads();
    if (row0 >= p.r) continue;
#pragma unroll
    for (int k = 0; k < kSlab; k += 4) {
      double a[4], b[2];
#pragma unroll
      for (int n = 0; n < 4; ++n) a[n] = qs[k + (lane & 3)][row0 + 8 * n + (lane >> 2)];
#pragma unroll
      for (int n = 0; n < 2; ++n) b[n] = x[k0 + k + (lane & 3)][col0 + 8 * n + (lane >> 2)];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_f64(v[i][j], a[i], b[j]);
    }
  }
  const double s = kFirst ? *scale_at(p) : 1.0;
  uint16_t* out = p.out + blockIdx.y * p.out_stride;
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    const int i = row0 + 8 * (n >> 2) + (lane >> 2), j = col0 + 8 * ((n >> 1) & 1) + 2 * (lane & 3) + (n & 1);
    if (i >= p.r || j0 + j >= p.length) continue;
    const double d = v[n >> 2][(n >> 1) & 1][n & 1] * s;
    if (!kLast) {
      y_at(p)[i * p.length + j0 + j] = d;
      continue;
    }
    const float f = static_cast<float>(d);
    const uint16_t u = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
    out[tall_out ? (j0 + j) * p.ldo + i : i * p.ldo + j0 + j] = u;
  }
}

template <bool kFirst, bool kLast>
cudaError_t launch_apply(const LongParams& p, int q, dim3 grid, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  const cudaError_t e = allow_shared(long_apply_kernel<kFirst, kLast>, done, kApplySmem);
  return e != cudaSuccess ? e : launch_programmatic(long_apply_kernel<kFirst, kLast>, grid, kApplyThreads, kApplySmem, s, p, q);
}

// Factors per run, shares of the long side, and doubles of scratch per matrix.
int run_of(const muonh_orthogonalize_desc& d) {
  return std::max(1, ns_chain_run(d.ns_a, d.ns_b, d.ns_c, d.ns_steps));
}
int shares_of(const muonh_orthogonalize_desc& d) {
  const int64_t tiles = std::min(d.rows, d.cols) > kTile64 ? 3 : 1, slabs = (std::max(d.rows, d.cols) + kSlab - 1) / kSlab;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kMaxShares, kTargetBlocks / (d.batch * tiles), slabs / 8})));
}
int64_t doubles_of(const muonh_orthogonalize_desc& d) {
  const int64_t r = std::min(d.rows, d.cols), length = std::max(d.rows, d.cols);
  return r * r * (kMatrices + shares_of(d)) + 1 + (run_of(d) < d.ns_steps ? r * length : 0);
}
int64_t part_of(const muonh_orthogonalize_desc& d) {
  return std::min<int64_t>({d.batch, 65535, std::max<int64_t>(1, kScratchBytes / (doubles_of(d) * 8))});
}

}  // namespace
}  // namespace muonh

using namespace muonh;

size_t muonh::orthogonalize_fp64_workspace(const muonh_orthogonalize_desc& d) {
  return static_cast<size_t>(part_of(d) * doubles_of(d)) * sizeof(double);
}

cudaError_t muonh::orthogonalize_fp64(const muonh_orthogonalize_desc& d, void* workspace, cudaStream_t s) {
  LongParams p{};
  p.x_stride = d.x_stride;
  p.ldx = d.ldx;
  p.out_stride = d.out_stride;
  p.ldo = d.ldo;
  p.tall = d.rows > d.cols;
  p.r = static_cast<int32_t>(std::min(d.rows, d.cols));
  p.length = std::max(d.rows, d.cols);
  p.scratch = static_cast<double*>(workspace);
  p.part = part_of(d);
  p.shares = shares_of(d);
  p.bf16 = d.dtype == MUONH_DTYPE_BF16;
  p.a = d.ns_a;
  p.b = d.ns_b;
  p.c = d.ns_c;
  p.eps = d.eps;
  const unsigned side = static_cast<unsigned>((p.r + kTile64 - 1) / kTile64);   // 1 or 2
  const unsigned blocks = static_cast<unsigned>((p.length + kPositions - 1) / kPositions);
  const int run = run_of(d);
  enum { kA, kP, kT, kQ };   // kQ and kQ + 1 in turn
  for (int64_t first = 0; first < d.batch; first += p.part) {
    const unsigned count = static_cast<unsigned>(std::min(p.part, d.batch - first));
    p.x = static_cast<const uint16_t*>(d.x) + first * d.x_stride;
    p.out = static_cast<uint16_t*>(d.out) + first * d.out_stride;
    cudaError_t e = cudaSuccess;
    auto product = [&](bool factor, int left, int right, int out) {
      if (e == cudaSuccess)
        e = launch_programmatic(factor ? long_product_kernel<true> : long_product_kernel<false>, dim3(side * side, count),
                                kTileThreads, 0, s, p, left, right, out);
    };
    for (int k0 = 0; k0 < d.ns_steps && e == cudaSuccess; k0 += run) {
      const bool from_x = k0 == 0, to_out = k0 + run >= d.ns_steps;
      const int steps = std::min(run, d.ns_steps - k0);
      e = launch_programmatic(from_x ? long_gram_kernel<false> : long_gram_kernel<true>,
                              dim3(side * (side + 1) / 2, count, static_cast<unsigned>(p.shares)), kTileThreads, 0, s, p);
      if (e == cudaSuccess)
        e = launch_programmatic(from_x ? long_join_kernel<true> : long_join_kernel<false>, dim3(kJoinBlocks, count),
                                kJoinThreads, 0, s, p);
      int q = kQ;
      for (int k = 0; k < steps; ++k) {
        const int factor = k == 0 ? kQ : kP;       // the first factor is Q
        product(true, kA, kA, factor);
        if (k > 0) {
          const int next = kQ + kQ + 1 - q;
          product(false, q, factor, next);
          q = next;
        }
        if (k == steps - 1) break;
        product(false, kA, factor, kT);
        product(false, kT, factor, kA);
      }
      const dim3 grid(blocks, count);
      if (e == cudaSuccess)
        e = from_x ? (to_out ? launch_apply<true, true>(p, q, grid, s) : launch_apply<true, false>(p, q, grid, s))
                   : (to_out ? launch_apply<false, true>(p, q, grid, s) : launch_apply<false, false>(p, q, grid, s));
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
