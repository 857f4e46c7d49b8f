// Orthogonalising stacks of matrices with a small side (at most 128): one
// Newton-Schulz update per attention head (sm_100a).
//
// For each matrix X (r x c on its wide orientation, r <= 128)
//   Y = s X,  s = 1/(||X||_F + eps);   n times: A = Y Y^T, Y <- p(A) Y,
//   p(A) = a I + b A + c A^2
// Every iterate is a polynomial in A_0 = Y Y^T times Y, so the whole iteration
// runs on r x r matrices (they commute, and stay symmetric):
//   P_k = p(A_k),  A_{k+1} = (A_k P_k) P_k,  Q_{k+1} = Q_k P_k,   O = s Q_n X.
// X is read once for the Gram matrix X X^T, whose trace is ||X||_F^2 (so the
// scale needs no pass of its own), and once more, out of L2, for Q X; O is
// written once.  Nothing r x c is kept in between.
//
// One cluster of 1 to 8 CTAs computes one matrix; a CTA walks over its share
// of the 128-wide slices of the long side.  A slice of X is 128 x 128 in
// shared memory, loaded by TMA as two boxes of 64 columns (128-byte swizzle),
// and serves every product without being moved:
//             wide X (r x c)                     tall X (c x r)
//   Gram      both operands K-major              both operands MN-major
//   Q X, X Q  Q K-major, slice MN-major          slice K-major, Q MN-major
// The clusters' Gram shares are added through distributed shared memory, in
// rank order, and every CTA then runs the same r x r iteration: with few
// matrices the SMs would otherwise be idle, with many the cluster is one CTA.
//
// What bounds it, for one [128, 2048] bf16 matrix on each of 148 SMs (119k
// cycles, 76 us): X X^T 28k cycles, reading 78 MB from HBM; the r x r iteration
// 50k, a chain of 14 dependent products of 24 MMAs (128 x 128 x 16, 2k cycles
// each with their hand-over, 1.5k without) and as many passes of the epilogue
// (1.0 to 1.4k: TMEM reads, the split into pairs, two barriers; without its
// stores it would be 5% of the chain shorter); Q X 29k, 1.5k per slice: its
// operands' reads, the slice's arrival and its result's way out share the 128
// bytes per cycle of shared memory.  The chain is what a single matrix costs
// whatever its long side.
//
// Precision.  The products are 16-bit with fp32 accumulation.  X X^T is exact
// up to the accumulation: X is used as it is.  The r x r operands are kept as
// fp16 pairs (hi + lo, 22 bits) and each product is lo hi + hi lo + hi hi:
// with single fp16 operands the Gram-space form loses the small singular
// directions (errors of 0.1 and more on ill-conditioned updates, by emulation,
// against 2e-4 with pairs).  Q enters the last product as a pair of X's type.
// Pairs hold five steps of the default coefficients; where ns_chain_run finds that
// they do not hold all of a run, it is muonh_orth_fp64.cu's.
// The tensor cores' accumulation truncates: the slices take kGramAccs accumulators
// in turn (the r x r products' columns are idle then), which are added in IEEE fp32
// registers after at most kGramChunk slices, and each pair product adds up its
// small parts first.  An X next to rank one with few rows and a long side was off
// by 3e-2 of ||out|| with 16 slices in one accumulator and the small parts last,
// and is by 7e-3 at most, in the same time (896 x [128, 2048]: 446 to 451 us under
// the power cap with 8, 16 or 32 slices and with the old sums).
// The result is rounded once to X's type.
#include <algorithm>
#include <cmath>

#include "muonh_common.cuh"

namespace muonh {
namespace {

constexpr int kSide = 128;                        // padded small side; also the slice width
constexpr int kChunkBytes = kSide * 64 * 2;       // 128 rows x 64 columns, 16-bit: 16 KB
constexpr int kSliceBytes = 2 * kChunkBytes;      // one slice of X, or one r x r 16-bit matrix
constexpr int kPairBytes = 2 * kSliceBytes;       // an r x r operand as hi and lo
constexpr int kRing = 4;                          // slices in flight
constexpr int kQOffset = kRing * kSliceBytes;     // the ring's space doubles as the operands A and P
constexpr int kBarsOffset = kQOffset + kPairBytes;
constexpr int kOrthSmem = kBarsOffset + 1024 + 1024;   // barriers, scalars; alignment slack
static_assert(kRing * kSliceBytes == 2 * kPairBytes, "A and P share the ring's space");
static_assert(kOrthSmem <= 227 * 1024, "shared memory of the orthogonalize kernel exceeds 227 KB");
constexpr int kEpiThreads = 512;                  // 16 epilogue warps: 32 rows x 32 columns each
constexpr int kOrthThreads = 64 + kEpiThreads;    // warp 0 TMA, warp 1 MMA
constexpr int kGramAccs = 4;                      // accumulators that slices take in turn
constexpr int kGramChunk = 8;                     // slices (1024 columns) before they are read
constexpr int kMaxSteps = kMaxChainSteps;
// With several matrices per SM all SMs read X, iterate and write at the same
// time, and HBM idles during the r x r iterations.  Half of the SMs start later by
// about what one walk over X takes.  Against none, at 600 to 1500 matrices of 16,
// 64 and 128 rows and 0 to 5 steps: 2 to 9% faster with 64 and 128 rows of 1024 and
// more, even with 16; shorter ones read too little to be apart.  (15 us whatever the
// length, as for 2048, cost up to 17% where a matrix takes less than that.)
constexpr int kLateSliceNs = 940;                 // of a walk: 28k cycles for 16 slices
constexpr int kLateMostNs = 30000;
constexpr int kLateSlices = 4;
constexpr int kLateWaves = 4;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxBatch = 1 << 24, kMaxLong = 1 << 30;

__device__ int g_orth_timeout;                    // a wait gave up in some call since the flag was read

struct OrthParams {
  int32_t slices;            // 128-wide slices of the long side
  int32_t tall;              // X is c x r
  int32_t steps;
  float a, b, c, eps;
  // power-of-two scales of the stored fp16 operands: A and A P; P; Q after
  // step k; and the final Q
  int32_t ea, eb, eq[kMaxSteps], eq_last;
  int32_t rows, cols;        // of X, for skipping stores outside
  int32_t late_below;        // odd CTAs below this number start late_ns late
  int32_t late_ns;
  int32_t used;              // small side rounded up to 64 or 128: columns and k of the r x r products
};

__device__ __forceinline__ uint32_t row_piece(int row, int piece) {
  return static_cast<uint32_t>(row * 128 + ((piece ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi) {
  if (!BF16) return pack_f16(lo, hi);
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack_16(uint32_t u) {
  if (!BF16) return __half22float2(*reinterpret_cast<__half2*>(&u));
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u));
}

// TMA with an L2 eviction priority: X is read a second time and is to stay until
// then, what is read last or written goes first.
__device__ __forceinline__ uint64_t policy_keep() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_drop() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// 32 values of one row as a 16-bit pair hi + lo: pieces piece0 .. piece0 + 3
// of the row in the 64-column chunk at `hi`, and the same in the lo matrix.
template <bool BF16>
__device__ __forceinline__ void store_split(uint8_t* hi, int row, int piece0, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[8 * q + 2 * i], y = v[8 * q + 2 * i + 1];
      h[i] = pack_16<BF16>(x, y);
      const float2 back = unpack_16<BF16>(h[i]);
      l[i] = pack_16<BF16>(x - back.x, y - back.y);
    }
    const uint32_t at = row_piece(row, piece0 + q);
    *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(hi + kSliceBytes + at) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Descriptors of a 128 x 128 slice or operand (two chunks of 128 rows x 64
// columns), and their advance over k steps of 16 along k.
__device__ __forceinline__ uint64_t k_major(uint32_t at) { return sdesc_sw128(at, 16, 1024); }
__device__ __forceinline__ uint64_t mn_major(uint32_t at) { return sdesc_sw128(at, kChunkBytes, 1024); }
__device__ constexpr uint32_t k_major_step(int k) { return ((k >> 2) * kChunkBytes + (k & 3) * 32) >> 4; }
__device__ constexpr uint32_t mn_major_step(int k) { return (k * 16 * 128) >> 4; }

// D (+)= L R over K steps: L K-major, R MN-major, both as their rows are
// stored.  Inlined straight-line code, so that the descriptors stay in uniform
// registers: in a function of its own, in a loop, or with a branch around each
// MMA, one took 135 cycles to issue, against the 64 that it takes to run.  The
// small side is rounded up to 64 or 128 for that (kHalf, kFull).
constexpr int kHalf = 4, kFull = 8;
template <int K>
__device__ __forceinline__ void products(uint32_t d, uint64_t left, uint64_t right, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < K; ++k)
    umma_f16(d, left + k_major_step(k), right + mn_major_step(k), idesc, k == 0 ? accumulate : 1u);
}

// D = L R for the 128 x 128 pairs at l and r: lo hi + hi lo + hi hi, the small
// products first, so that 8 accumulations truncate the full sum and not 24.  R is
// symmetric up to rounding, but reading it as its transpose (K-major) compounds
// that asymmetry from product to product: the last A_k was off by 1e-4 instead
// of 1e-6.
template <int K>
__device__ __forceinline__ void pair_product(uint32_t d, uint32_t l, uint32_t r, uint32_t idesc) {
#pragma unroll 1
  for (int prod = 0; prod < 3; ++prod)
    products<K>(d, k_major(l + (prod == 0 ? kSliceBytes : 0)), mn_major(r + (prod == 1 ? kSliceBytes : 0)), idesc, prod);
}

// The sum over the cluster's R CTAs of the 32 values of each epilogue thread,
// which every CTA has left at smem as 8 vectors per thread.  Each CTA adds
// 8/R of the vectors, in rank order, and then all fetch each other's: 2 x 64
// KB per CTA instead of R x 64 KB, and the same sums everywhere.  Loads start
// at the next CTA, so that no CTA's shared memory is read by all at once.
// All threads call it, between two cluster barriers.
template <int R>
__device__ __forceinline__ void add_shares(uint8_t* smem, uint32_t rank, float (&acc)[32]) {
  constexpr int kEach = 8 / R;
  const bool mine = threadIdx.x >= 64;
  const uint32_t at = (threadIdx.x - 64) * 16;
  float4* const own = reinterpret_cast<float4*>(smem) + (threadIdx.x - 64);
  if (mine) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t from = map_shared_rank(smem, (rank + 1 + i) % R) + at;
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[i * kEach + j] = load_cluster_f4(from + (rank * kEach + j) * kEpiThreads * 16);
    }
    // v[i] came from CTA (rank + 1 + i) % R: rotated back, so that the sum is in rank order
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (uint32_t r = 0; r < R; ++r) {
        float4 w = v[j];
#pragma unroll
        for (int i = 1; i < R; ++i)
          if ((rank + 1 + i) % R == r) w = v[i * kEach + j];
        sum.x += w.x;
        sum.y += w.y;
        sum.z += w.z;
        sum.w += w.w;
      }
      own[(rank * kEach + j) * kEpiThreads] = sum;
    }
  }
  cluster_sync();
  if (mine) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t r = (rank + 1 + i) % R;
      const uint32_t from = map_shared_rank(smem, r) + at;
      // the vectors of CTA r are numbers r kEach and on; acc is indexed statically
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float4 v = load_cluster_f4(from + (r * kEach + j) * kEpiThreads * 16);
#pragma unroll
        for (int s = 0; s < R; ++s)
          if (static_cast<uint32_t>(s) == r) {
            acc[4 * (s * kEach + j)] = v.x;
            acc[4 * (s * kEach + j) + 1] = v.y;
            acc[4 * (s * kEach + j) + 2] = v.z;
            acc[4 * (s * kEach + j) + 3] = v.w;
          }
      }
    }
  }
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

template <bool BF16>
__global__ void __launch_bounds__(kOrthThreads, 1)
    orthogonalize_kernel(const __grid_constant__ OrthParams p, const __grid_constant__ CUtensorMap xmap,
                         const __grid_constant__ CUtensorMap omap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sm_a = smem;                     // A, then A P
  uint8_t* const sm_p = smem + kPairBytes;
  uint8_t* const sm_q = smem + kQOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarsOffset);   // [pass][slot]
  uint64_t* empty = full + 2 * kRing;             // [pass][slot]; pass 0: products done, pass 1: output stored
  uint64_t* tfull = empty + 2 * kRing;            // [pass][accumulator]; pass 0: one for all of them
  uint64_t* tempty = tfull + 4;
  uint64_t* ready = tempty + 4;                   // the epilogue wrote the next r x r operand
  uint64_t* q_ready = ready + 1;                  // ... the final Q; the ring's space is free again
  uint64_t* done = q_ready + 1;                   // a product of the A chain
  uint64_t* done_q = done + 1;                    // a product of the Q chain
  uint64_t* drain = done_q + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);
  float* trace = reinterpret_cast<float*>(err + 1);   // [4]: shares of the diagonal

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const uint32_t rank = cluster_ctarank();
  const int matrix = blockIdx.x / ranks;
  const int first = static_cast<int>(static_cast<int64_t>(p.slices) * rank / ranks);
  const int count = static_cast<int>(static_cast<int64_t>(p.slices) * (rank + 1) / ranks) - first;
  const int chunks = (count + kGramChunk - 1) / kGramChunk;

  if (static_cast<int>(blockIdx.x) < p.late_below && (blockIdx.x & 1)) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < static_cast<uint64_t>(p.late_ns)) __nanosleep(500);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&full[kRing + s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&empty[kRing + s], kEpiThreads / 64);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiThreads);
    }
    mbar_init(ready, kEpiThreads);
    mbar_init(q_ready, kEpiThreads);
    mbar_init(done, 1);
    mbar_init(done_q, 1);
    mbar_init(drain, 1);
    *err = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_stream();
  if (p.late_below == 0) let_next_set_up();        // 1 us of the 21 to 45 of a small call; the norms lost by it
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_d = tmem + 256, tm_q = tmem + 384;   // r x r products; X X^T uses all columns, Q X 0 .. 255

  // One walk of the producer over this CTA's slices.  A copy in flight lands
  // before the CTA may exit: the MMA issuer or, after a wait that gave up,
  // the producer itself waits for it.
  auto produce = [&](int pass) {
    uint64_t* f = full + pass * kRing;
    uint64_t* e = empty + pass * kRing;
    const uint64_t policy = pass == 0 ? policy_keep() : policy_drop();
    int i = 0;
    for (; i < count; ++i) {
      const int slot = i % kRing;
      if (i >= kRing && !mbar_wait(&e[slot], (i / kRing - 1) & 1, err)) break;
      mbar_expect_tx(&f[slot], kSliceBytes);
      uint8_t* dst = smem + slot * kSliceBytes;
      // the second walk runs backwards: the last slices read are the likeliest to be in L2 still
      const int at = (first + (pass == 0 ? i : count - 1 - i)) * kSide;
      for (int h = 0; h < 2; ++h)
        load_box(dst + h * kChunkBytes, &xmap, &f[slot], p.tall ? 64 * h : at + 64 * h, p.tall ? at : 0, matrix,
                 policy);
    }
    for (int j = i > kRing ? i - kRing : 0; j < i; ++j) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&f[j % kRing], (j / kRing) & 1) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
  };

  // epilogue threads: one row and 32 of its columns each (a warp reaches the
  // TMEM lanes of its number mod 4)
  const int quarter = warp & 3, col0 = ((warp - 2) >> 2) * 32;
  const int row = quarter * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const int ch = (col0 >> 6) * kChunkBytes;        // the 64-column chunk of these columns
  const int piece0 = (col0 & 32) >> 3;             // and their first 16-byte piece in its rows
  const bool inside = col0 < p.used;               // columns behind the small side are not computed (per warp)
  float acc[32];                                   // its part of X X^T, then of A_k

  // ------------------------------------------------------------ X X^T
  if (warp == 0) {
    if (lane == 0) produce(0);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16(kSide, p.used, BF16, p.tall) | (static_cast<uint32_t>(p.tall) << 15);
    const bool leader = elect_lane();
    bool ok = true;
    for (int i = 0; i < count && ok; ++i) {
      const int slot = i % kRing, chunk = i / kGramChunk;
      if (i % kGramChunk == 0 && chunk >= 1) ok = mbar_wait(&tempty[0], (chunk - 1) & 1, err);
      ok = ok && mbar_wait(&full[slot], (i / kRing) & 1, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t x = smem_u32(smem + slot * kSliceBytes);
      const uint64_t d = p.tall ? mn_major(x) : k_major(x);
      if (leader) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t dk = d + (p.tall ? mn_major_step(k) : k_major_step(k));
          umma_f16(tmem + (i % kGramAccs) * kSide, dk, dk, idesc, (i % kGramChunk) >= kGramAccs || k != 0);
        }
        umma_commit(&empty[slot]);
        if (i % kGramChunk == kGramChunk - 1 || i == count - 1) umma_commit(&tfull[0]);
      }
      __syncwarp();
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0.f;
    for (int c = 0; c < chunks; ++c) {
      if (!mbar_wait(&tfull[0], c & 1, err)) break;
      tc_fence_after();
      const int accs = min(kGramAccs, count - c * kGramChunk);
      for (int a = 0; a < accs && inside; ++a) {
        float v[32];
        tmem_ld32(tmem + lanes + a * kSide + col0, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] += v[j];
      }
      tc_fence_before();
      mbar_arrive(&tempty[0]);
    }
    if (ranks > 1) {   // this CTA's share, for the others to add
      float4* mine = reinterpret_cast<float4*>(smem) + (threadIdx.x - 64);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        mine[j * kEpiThreads] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
    }
  }
  if (ranks > 1) {
    cluster_sync();
    if (ranks == 2)
      add_shares<2>(smem, rank, acc);
    else if (ranks == 4)
      add_shares<4>(smem, rank, acc);
    else
      add_shares<8>(smem, rank, acc);
    cluster_sync();
  }

  // ------------------------------------------------- the r x r iteration
  float scale = 0.f;                                // 1 / (||X|| + eps)
  if (warp == 1) {
    const uint32_t idesc = idesc_f16(kSide, p.used, 0, 1);
    const uint32_t a = smem_u32(sm_a), q = smem_u32(sm_q);
    const bool leader = elect_lane();
    // per step: A_k^2 once A_k is there, A_k P_k once P_k is, (A_k P_k) P_k once A_k P_k is, and then
    // Q_k P_k, which runs while the epilogue works on A_{k+1}.  The last step has the first and the Q
    // product only, the first step no Q product (P_0 is Q_1).
    int waits = 0;
    bool ok = true;
    for (int n = 0; n < 4 * p.steps && ok; ++n) {
      const int k = n >> 2, phase = n & 3;
      const bool last = k == p.steps - 1;
      if (phase < 2 || (phase == 2 && !last)) {      // the last P_k has to be there for its Q product, too
        ok = mbar_wait(ready, waits++ & 1, err);
        tc_fence_after();
      }
      if (!ok || (last && (phase == 1 || phase == 2)) || (k == 0 && phase == 3)) continue;
      const uint32_t pk = k == 0 ? q : smem_u32(sm_p);
      const uint32_t d = phase == 3 ? tm_q : tm_d, l = phase == 3 ? q : a, r = phase == 0 ? a : pk;
      if (leader) {
        if (p.used == 64)
          pair_product<kHalf>(d, l, r, idesc);
        else
          pair_product<kFull>(d, l, r, idesc);
        umma_commit(phase == 3 ? done_q : done);
      }
      __syncwarp();
    }
  } else if (warp >= 2) {
    // ||X||^2 is the trace; summed over a warp's rows, then over the warps
    const bool diagonal = col0 == quarter * 32;     // this warp's block holds diagonal elements, one per lane
    float d = 0.f;
    if (diagonal) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == lane) d = acc[j];
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) trace[quarter] = d;
    }
    epilogue_sync();
    d = (trace[0] + trace[1]) + (trace[2] + trace[3]);
    const float norm = sqrtf(d) + p.eps;
    // zeros stay zeros; a norm that is not finite makes the matrix NaN (1 / Inf would leave finite elements at 0)
    scale = norm > 0.f ? (isinf(norm) ? __int_as_float(0x7fffffff) : 1.f / norm) : (norm == 0.f ? 0.f : norm);
    // from here on acc is 2^ea A_k
    const float start = scale * exp2i(p.ea);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = acc[j] * scale * start;

    auto publish = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar);
    };
    int n_done = 0, n_done_q = 0;
    auto wait_done = [&] {
      const bool ok = mbar_wait(done, n_done++ & 1, err);
      tc_fence_after();
      return ok;
    };
    const float f_last = exp2i(p.eq_last);
    float v[32];
    auto read_scaled = [&](uint32_t from, float f) {
      tmem_ld32(from + lanes + col0, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= f;
    };
    auto add_diagonal = [&](float x) {
      if (!diagonal) return;
      const uint32_t mine = 1u << lane;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (mine & (1u << j)) v[j] += x;
    };
    bool ok = true;
    if (p.steps == 0 && inside) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.f;
      add_diagonal(f_last);
      store_split<BF16>(sm_q + ch, row, piece0, v);
    }
    for (int k = 0; k < p.steps; ++k) {
      const bool last = k == p.steps - 1;
      const int ep = k == 0 ? p.eq[0] : p.eb;       // P_0 is Q_1 and is stored as such
      if (inside) store_split<false>(sm_a + ch, row, piece0, acc);
      publish(ready);
      if (k > 1) {
        // Q_{k-1} P_{k-1} from the step before, while A_k^2 runs
        ok = mbar_wait(done_q, n_done_q++ & 1, err);
        tc_fence_after();
        if (!ok) break;
        if (inside) {
          read_scaled(tm_q, exp2i(p.eq[k - 1] - p.eq[k - 2] - p.eb));
          store_split<false>(sm_q + ch, row, piece0, v);
        }
      }
      // P = a I + b A + c A^2
      if (!(ok = wait_done())) break;
      if (inside) {
        const float f = (last && k == 0) ? f_last : exp2i(ep);
        const float fc = p.c * f * exp2i(-2 * p.ea), fb = p.b * f * exp2i(-p.ea);
        tmem_ld32(tm_d + lanes + col0, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = fmaf(fc, v[j], fb * acc[j]);
        add_diagonal(p.a * f);
        if (last && k == 0)
          store_split<BF16>(sm_q + ch, row, piece0, v);
        else
          store_split<false>((k == 0 ? sm_q : sm_p) + ch, row, piece0, v);
      }
      publish(ready);
      if (last) break;
      // A P replaces A
      if (!(ok = wait_done())) break;
      if (inside) {
        read_scaled(tm_d, exp2i(-ep));
        store_split<false>(sm_a + ch, row, piece0, v);
      }
      publish(ready);
      if (!(ok = wait_done())) break;
      if (inside) {
        tmem_ld32(tm_d + lanes + col0, acc);
        const float fn = exp2i(-ep);
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] *= fn;
      }
    }
    if (ok && p.steps > 1) {                        // the final Q, in X's type
      ok = mbar_wait(done_q, n_done_q++ & 1, err);
      tc_fence_after();
      if (inside) {
        read_scaled(tm_q, exp2i(p.eq_last - p.eq[p.steps - 2] - p.eb));
        store_split<BF16>(sm_q + ch, row, piece0, v);
      }
    }
    publish(q_ready);
    scale *= exp2i(-p.eq_last);
  }

  // ------------------------------------------------------------ O = s Q X
  if (warp == 0) {
    if (lane == 0 && mbar_wait(q_ready, 0, err)) produce(1);
    __syncwarp();
  } else if (warp == 1) {
    // wide: N is the slice's width and k the small side; tall: N and k are the small side
    const uint32_t idesc = idesc_f16(kSide, p.tall ? p.used : kSide, BF16, 1);
    const uint32_t q = smem_u32(sm_q);
    const bool leader = elect_lane();
    bool ok = mbar_wait(q_ready, 0, err);
    tc_fence_after();
    for (int i = 0; i < count && ok; ++i) {
      const int slot = i % kRing;
      ok = (i < 2 || mbar_wait(&tempty[2 + (i & 1)], ((i >> 1) - 1) & 1, err)) &&
           mbar_wait(&full[kRing + slot], (i / kRing) & 1, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t x = smem_u32(smem + slot * kSliceBytes);
      if (leader) {
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {      // Q's lo, then its hi: the small products first
          const uint32_t qp = q + (1 - part) * kSliceBytes, left = p.tall ? x : qp, right = p.tall ? qp : x;
          if (p.used == 64)
            products<kHalf>(tmem + (i & 1) * kSide, k_major(left), mn_major(right), idesc, part);
          else
            products<kFull>(tmem + (i & 1) * kSide, k_major(left), mn_major(right), idesc, part);
        }
        umma_commit(&tfull[2 + (i & 1)]);
      }
      __syncwarp();
    }
    // no MMA may still write TMEM when the CTA frees it
    if (leader) umma_commit(drain);
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  } else {
    // two warps write their 32 rows x 64 columns over the slice that they came
    // from (whose products are done), and the first stores that box.  A wait
    // that gives up records that and goes on: the pair's barrier needs both.
    const uint64_t policy = policy_drop();
    const int pair = 2 + quarter + 4 * (col0 >> 6);   // named barrier of the two
    const bool store = (col0 & 32) == 0 && lane == 0;
    for (int i = 0; i < count; ++i) {
      mbar_wait(&tfull[2 + (i & 1)], (i >> 1) & 1, err);
      tc_fence_after();
      uint8_t* box = smem + (i % kRing) * kSliceBytes + ch;
      float v[32];
      tmem_ld32(tmem + lanes + (i & 1) * kSide + col0, v);
      tc_fence_before();
      mbar_arrive(&tempty[2 + (i & 1)]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = pack_16<BF16>(v[8 * q + 2 * j] * scale, v[8 * q + 2 * j + 1] * scale);
        *reinterpret_cast<uint4*>(box + row_piece(row, piece0 + q)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      if (store) {
        const int at = (first + count - 1 - i) * kSide;
        const int x0 = p.tall ? col0 : at + col0, y0 = p.tall ? at + quarter * 32 : quarter * 32;
        if (x0 < p.cols && y0 < p.rows) store_box(&omap, box + quarter * 4096, x0, y0, matrix, policy);
        bulk_commit();
        if (i > 0) {                                // the previous slice's box has been read
          bulk_wait_read<1>();
          mbar_arrive(&empty[kRing + (i - 1) % kRing]);
        }
      }
    }
    if (store) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && *err) atomicOr(&g_orth_timeout, 1);
}

// Copies a stack whose rows TMA cannot address to one whose rows it can, or
// back: `lanes` lanes of a warp per row, element by element.
__global__ void __launch_bounds__(256)
    copy_stack_kernel(const uint16_t* from, int64_t from_stride, int64_t from_ld, uint16_t* to, int64_t to_stride,
                      int64_t to_ld, int64_t batch, int64_t rows, int cols, int lanes) {
  wait_for_stream();
  const int per_block = 256 / lanes, lane = threadIdx.x % lanes;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / lanes; r < batch * rows;
       r += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t b = r / rows, y = r - b * rows;
    const uint16_t* src = from + b * from_stride + y * from_ld;
    uint16_t* dst = to + b * to_stride + y * to_ld;
#pragma unroll 8
    for (int c = lane; c < cols; c += lanes) dst[c] = src[c];
  }
}

cudaError_t copy_stack(const void* from, int64_t from_stride, int64_t from_ld, void* to, int64_t to_stride, int64_t to_ld,
                       const muonh_orthogonalize_desc& d, int sms, cudaStream_t s) {
  int lanes = 4;
  while (lanes < 32 && lanes < d.cols) lanes *= 2;
  const int64_t blocks = (d.batch * d.rows + 256 / lanes - 1) / (256 / lanes);
  return launch_programmatic(copy_stack_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 16ll * sms))), 256, 0,
                             s, static_cast<const uint16_t*>(from), from_stride, from_ld, static_cast<uint16_t*>(to),
                             to_stride, to_ld, d.batch, d.rows, static_cast<int>(d.cols), lanes);
}

muonh_status orth_fail(muonh_status st, const char* msg) {
  set_error_message(msg);
  return st;
}

// Rows of a 16-bit stack that TMA can address: 16-byte aligned base and strides.
bool tma_stack(const void* p, int64_t stride, int64_t ld, int64_t batch, int64_t rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows == 1 || (ld % 8 == 0 && ld > 0)) &&
         (batch == 1 || (stride % 8 == 0 && stride > 0));
}

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

struct Stack {
  void* p;
  int64_t stride, ld;
};

bool encode_stack(CUtensorMap* map, const Stack& s, const muonh_orthogonalize_desc& d, int box_rows) {
  // strides that no coordinate uses still have to be valid ones
  const int64_t ld = d.rows == 1 ? up8(d.cols) : s.ld, stride = d.batch == 1 ? up8(ld * d.rows) : s.stride;
  return encode_tiled_stack(map, s.p, d.dtype == MUONH_DTYPE_BF16, d.cols, d.rows, d.batch, ld, stride, box_rows);
}

muonh_status check_orth(const muonh_orthogonalize_desc* d) {
  if (!d) return orth_fail(MUONH_ERR_INVALID_ARG, "desc is NULL");
  if (d->batch < 0 || d->rows < 0 || d->cols < 0 || d->batch > kMaxBatch || d->rows > kMaxLong || d->cols > kMaxLong)
    return orth_fail(MUONH_ERR_INVALID_ARG, "batch must be in [0, 2^24], rows and cols in [0, 2^30]");
  if (d->dtype != MUONH_DTYPE_BF16 && d->dtype != MUONH_DTYPE_F16)
    return orth_fail(MUONH_ERR_INVALID_ARG, "dtype must be MUONH_DTYPE_BF16 or MUONH_DTYPE_F16");
  if (d->ns_steps < 0 || d->ns_steps > kMaxSteps) return orth_fail(MUONH_ERR_INVALID_ARG, "ns_steps must be in [0, 16]");
  if (!std::isfinite(d->ns_a) || !std::isfinite(d->ns_b) || !std::isfinite(d->ns_c) || !std::isfinite(d->eps) ||
      d->eps < 0.f)
    return orth_fail(MUONH_ERR_INVALID_ARG, "the coefficients must be finite and eps finite and >= 0");
  if (std::min(d->rows, d->cols) > kSide)
    return orth_fail(MUONH_ERR_UNSUPPORTED, "the smaller side of a matrix must be at most 128");
  if (d->batch == 0 || d->rows == 0 || d->cols == 0) return MUONH_OK;
  if (!d->x || !d->out) return orth_fail(MUONH_ERR_INVALID_ARG, "x or out is NULL");
  if ((d->rows > 1 && (d->ldx < d->cols || d->ldo < d->cols)) || d->x_stride < 0 || d->out_stride < 0)
    return orth_fail(MUONH_ERR_INVALID_ARG, "row strides must be at least cols, matrix strides at least 0");
  if ((reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->out)) & 1)
    return orth_fail(MUONH_ERR_ALIGNMENT, "x and out must be 2-byte aligned");
  return MUONH_OK;
}

// Clusters of `ranks` CTAs that the device holds at once.  A cluster has to fit
// in one GPC, so fewer of the large ones fit than the SMs alone would say: 16
// clusters of 8 took two waves and 100 us where 16 of 4 took 57.
int clusters_at_once(bool bf16, int ranks, int dev) {
  static std::atomic<int> known[64][4];          // per device and log2(ranks), plus one
  int log = 0;
  while ((1 << log) < ranks) ++log;
  std::atomic<int>* memo = dev >= 0 && dev < 64 ? &known[dev][log] : nullptr;
  if (memo && memo->load()) return memo->load() - 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kOrthThreads);
  cfg.dynamicSmemBytes = kOrthSmem;
  cudaLaunchAttribute attr = cluster_launch(static_cast<unsigned>(ranks));
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  const cudaError_t e = bf16 ? cudaOccupancyMaxActiveClusters(&n, orthogonalize_kernel<true>, &cfg)
                             : cudaOccupancyMaxActiveClusters(&n, orthogonalize_kernel<false>, &cfg);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (memo) memo->store(n + 1);
  return n;
}

// More CTAs per matrix while all clusters still run at once and each CTA has
// two slices at least.
int pick_cluster(bool bf16, int64_t batch, int slices, int dev) {
  int ranks = 1;
  while (ranks < kMaxCluster && slices >= 4 * ranks && batch <= clusters_at_once(bf16, 2 * ranks, dev)) ranks *= 2;
  return ranks;
}

// Whether the r x r iterates can be kept as pairs; else the run is muonh_orth_fp64.cu's.
bool pairs_hold(const muonh_orthogonalize_desc& d) {
  return ns_chain_run(d.ns_a, d.ns_b, d.ns_c, d.ns_steps) >= d.ns_steps;
}

size_t copy_bytes(const muonh_orthogonalize_desc& d) {
  return static_cast<size_t>(d.batch) * d.rows * up8(d.cols) * 2;
}

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" size_t muonh_orthogonalize_workspace(const muonh_orthogonalize_desc* d) {
  if (!d || d->batch < 1 || d->rows < 1 || d->cols < 1) return 0;
  // refused (and sizes whose products might not fit in 64 bits)
  if (std::min(d->rows, d->cols) > kSide || d->ns_steps < 0 || d->ns_steps > kMaxSteps || d->batch > kMaxBatch ||
      d->rows > kMaxLong || d->cols > kMaxLong)
    return 0;
  if (!pairs_hold(*d)) return orthogonalize_fp64_workspace(*d);
  size_t n = 0;
  if (!tma_stack(d->x, d->x_stride, d->ldx, d->batch, d->rows)) n += copy_bytes(*d);
  if (!tma_stack(d->out, d->out_stride, d->ldo, d->batch, d->rows)) n += copy_bytes(*d);
  return n;
}

extern "C" muonh_status muonh_orthogonalize(const muonh_orthogonalize_desc* d, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  set_error_message("");
  if (const muonh_status st = check_orth(d)) return st;
  if (d->batch == 0 || d->rows == 0 || d->cols == 0) return MUONH_OK;
  const size_t scratch = muonh_orthogonalize_workspace(d);
  if (workspace_bytes < scratch || (scratch && !workspace))
    return orth_fail(MUONH_ERR_INVALID_ARG, "the workspace is smaller than muonh_orthogonalize_workspace says");
  if (reinterpret_cast<uintptr_t>(workspace) & 15)
    return orth_fail(MUONH_ERR_ALIGNMENT, "the workspace must be 16-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!pairs_hold(*d))
    return orthogonalize_fp64(*d, workspace, s) == cudaSuccess
               ? MUONH_OK
               : orth_fail(MUONH_ERR_CUDA, "launch of a kernel of the fp64 orthogonalize run failed");
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);

  const int64_t ld = up8(d->cols);
  Stack in{const_cast<void*>(d->x), d->x_stride, d->ldx}, out{d->out, d->out_stride, d->ldo};
  uint8_t* work = static_cast<uint8_t*>(workspace);
  if (!tma_stack(in.p, in.stride, in.ld, d->batch, d->rows)) {
    if (copy_stack(in.p, in.stride, in.ld, work, ld * d->rows, ld, *d, sms, s) != cudaSuccess)
      return orth_fail(MUONH_ERR_CUDA, "launch of copy_stack_kernel failed");
    in = Stack{work, ld * d->rows, ld};
    work += copy_bytes(*d);
  }
  const bool copy_back = !tma_stack(out.p, out.stride, out.ld, d->batch, d->rows);
  if (copy_back) out = Stack{work, ld * d->rows, ld};

  OrthParams p{};
  p.tall = d->rows > d->cols;
  p.rows = static_cast<int32_t>(d->rows);
  p.cols = static_cast<int32_t>(d->cols);
  p.used = std::min(d->rows, d->cols) <= 64 ? 64 : kSide;
  p.slices = static_cast<int32_t>((std::max(d->rows, d->cols) + kSide - 1) / kSide);
  p.steps = d->ns_steps;
  p.a = d->ns_a;
  p.b = d->ns_b;
  p.c = d->ns_c;
  p.eps = d->eps;
  ns_chain_scales(p.a, p.b, p.c, p.steps, &p.ea, &p.eb, p.eq);
  p.eq_last = (d->dtype == MUONH_DTYPE_BF16 || p.steps == 0) ? 0 : p.eq[p.steps - 1];
  CUtensorMap xmap, omap;
  if (!encode_stack(&xmap, in, *d, kSide) || !encode_stack(&omap, out, *d, 32))
    return orth_fail(MUONH_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  const bool bf16 = d->dtype == MUONH_DTYPE_BF16;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = bf16 ? allow_shared(orthogonalize_kernel<true>, done[1], kOrthSmem)
                       : allow_shared(orthogonalize_kernel<false>, done[0], kOrthSmem);
  if (e != cudaSuccess) return orth_fail(MUONH_ERR_CUDA, "the kernel's shared memory was refused");
  const int ranks = pick_cluster(bf16, d->batch, p.slices, dev);
  p.late_below = d->batch >= static_cast<int64_t>(kLateWaves) * sms && p.slices >= kLateSlices ? sms : 0;
  p.late_ns = static_cast<int32_t>(std::min<int64_t>(int64_t(kLateSliceNs) * p.slices, kLateMostNs));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(d->batch * ranks));
  cfg.blockDim = dim3(kOrthThreads);
  cfg.dynamicSmemBytes = kOrthSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {cluster_launch(static_cast<unsigned>(ranks)), programmatic_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = bf16 ? cudaLaunchKernelEx(&cfg, orthogonalize_kernel<true>, p, xmap, omap)
           : cudaLaunchKernelEx(&cfg, orthogonalize_kernel<false>, p, xmap, omap);
  if (e == cudaSuccess && copy_back) e = copy_stack(out.p, out.stride, out.ld, d->out, d->out_stride, d->ldo, *d, sms, s);
  if (e != cudaSuccess) return orth_fail(MUONH_ERR_CUDA, "launch of the orthogonalize kernel failed");
  return MUONH_OK;
}

cudaError_t muonh::take_orth_timeout(int* flag, cudaStream_t s) { return take_flag(g_orth_timeout, flag, s); }
