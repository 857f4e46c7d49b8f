// Products of 8-bit matrices with a power-of-two scale per block of 128
// (sm_100a): D = A B^T, the forward, activation-gradient and weight-gradient
// products of the recipe's linear layers (Puro-2B report: blockwise e4m3).
//
//   D[m, n] (+)= sum over k-blocks b of 2^(sa[m, b] + sb[n, b] - 254)
//                                       sum_{k in b} qa[m, k] qb[n, k]
// The tensor cores take the scales themselves: tcgen05.mma kind::mxf8f6f4
// multiplies blocks of 32 along k by a pair of E8M0 scales, so a block of 128 is
// four MMAs that use the same scale byte.  A 32-bit TMEM word per row holds the
// bytes of four k-blocks (512 of k); the instruction descriptor picks the byte.
//
// Three shapes of the same kernel, with one CTA per SM:
//   pair    a cluster of two CTAs computes 256 x 256 tiles with cta_group::2, each
//           CTA loading its 128 rows of A and half of the 256 rows of B.  A CTA
//           then fetches 32 KB per 128 of k for 128 x 256 results, against 48 KB
//           for a 128 x 256 tile of its own: L2 bandwidth is what bounds that one.
//   single  128 x 128 or 128 x 64 tiles, where the pair's would leave SMs idle.
//   split   a cluster of up to 8 CTAs shares the k of one 128 x 64 tile, where even
//           those are few and k is long (a narrow layer's weight gradient): the
//           partial sums are added through distributed shared memory, in rank order.
// Warps 0 and 3 load A and B by TMA (one k-block of 128 bytes is one 128-byte
// swizzled row; a TMA instruction holds its thread for hundreds of cycles, so one
// warp for both could not keep up).  Warp 2 gathers the scale words of both
// operands into shared memory; warp 1 copies them to TMEM (tcgen05.cp) and issues
// the MMAs; warps 4 to 11 take the accumulator into registers, hand it back, round
// once and store.
//
// 8192 x 6144 x 2048 to bf16: 94 us in a burst, 111 us (1.85 PFLOP/s) under the power
// cap at some 1.7 GHz; 256 x 192 tiles with two accumulators took 108 against 98 side
// by side (more operand traffic per product).
//
// The tensor cores' fp32 accumulation truncates, with an error that grows with
// the number of products added up (5e-7 of the result's norm at k = 8192, for
// random operands).  fp32 results are therefore accumulated over at most
// kChunkBlocks k-blocks in TMEM, and the chunks are added in IEEE fp32 in the
// result itself, by the thread that wrote it: 2e-7.
#include <algorithm>

#include "muonh_common.cuh"

namespace muonh {
namespace {

constexpr int kTm = 128;                         // tile rows
constexpr int kKBlock = 128;                     // k per stage: one scale block
constexpr int kThreads = 384;
constexpr int kEpi = 256;                        // epilogue threads
constexpr int kScaleRing = 4;                    // scale words in flight: 512 of k each
constexpr int kChunkBlocks = 32;                 // fp32 results: k-blocks per TMEM accumulation

// PAIR: BN is 256, shared by the two CTAs.  SPLIT: one tile per cluster.
template <int BN, bool PAIR>
struct BlockCfg {
  static_assert(!PAIR || BN == 256, "a pair computes 256 x 256 tiles");
  static constexpr int kTileRows = PAIR ? 2 * kTm : kTm;
  static constexpr int kBRows = PAIR ? BN / 2 : BN;    // rows of B that this CTA loads
  static constexpr int kABytes = kTm * kKBlock;
  static constexpr int kBBytes = kBRows * kKBlock;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 6;
  static constexpr int kAccs = BN == 256 ? 1 : 2;      // accumulators in TMEM, next to the scales
  static constexpr int kScaleBlocks = 1 + (BN + 127) / 128;   // 512-byte blocks of scale words: A, and B per 128 rows
  static constexpr int kScaleBytes = kScaleBlocks * 512;
  static constexpr int kScaleOffset = kStages * kStageBytes;
  static constexpr int kBarOffset = kScaleOffset + kScaleRing * kScaleBytes;
  static constexpr int kSmem = kBarOffset + 512 + 1024;
  static constexpr uint32_t kScaleCol = 256;           // first TMEM column of the scale words
  static_assert(kSmem <= 227 * 1024, "shared memory of the block-scaled kernel exceeds 227 KB");
};

__device__ int g_block_timeout;                  // a wait gave up in some call since the flag was read

struct BlockParams {
  const uint8_t* sa;
  const uint8_t* sb;
  int64_t ld_sa, ld_sb;
  int32_t sa_shift, sb_shift;                    // 7: one scale per 128 rows, 0: one per row
  int32_t sa_words, sb_words;                    // scales can be read four at a time
  void* d;
  int64_t ldd;
  int32_t m, n, k_blocks;
  int32_t dtype, accumulate, wide_store;
  int32_t tiles_m, tiles_n, band;
  int32_t shares;                                // SPLIT: CTAs per tile
};

// D[tmem] (+)= (A 2^sa) (B 2^sb)^T over 32 of k, e4m3 operands with E8M0 scales.
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                          uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

// The same over a CTA pair: 256 rows of A, half in each CTA.
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                               uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes from shared memory to 4 TMEM columns of lanes 0..31, repeated for the other three lane groups.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// ... in both CTAs of a pair, each from its own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}

// Descriptor of that 512-byte block: no swizzle, 8 rows of 16 bytes per 128 bytes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Instruction descriptor, kind::mxf8f6f4: both operands e4m3 and K-major, E8M0
// scales, byte `id` of the scale words.
__device__ __forceinline__ uint32_t idesc_mxf8(int m, int n, int id) {
  return (static_cast<uint32_t>(id) << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(id) << 29);
}

// Tile t of the walk: bands of `band` tile rows, column by column within a
// band, so that the tiles in flight share operands in L2.
__device__ __forceinline__ void tile_at(const BlockParams& p, int64_t t, int& tm, int& tn) {
  const int64_t per_band = static_cast<int64_t>(p.band) * p.tiles_n;
  const int b = static_cast<int>(t / per_band);
  const int rows = min(p.band, p.tiles_m - b * p.band);
  const int r = static_cast<int>(t - b * per_band);
  tm = b * p.band + r % rows;
  tn = r / rows;
}

// Scale bytes of k-blocks 4 g .. 4 g + 3 of one operand row (null: behind the
// last one), as one word; 2^0 where there is no row or no such block (what they
// scale is zero).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int words, int g, int k_blocks) {
  if (!row) return 0x7f7f7f7fu;
  const uint8_t* p = row + 4 * g;
  if (words && 4 * g + 4 <= k_blocks) return __ldg(reinterpret_cast<const uint32_t*>(p));
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(4 * g + i < k_blocks ? __ldg(p + i) : 127) << (8 * i);
  return w;
}

struct alignas(32) Vec32 {
  uint32_t u[8];
};
__device__ __forceinline__ void store32(void* p, const Vec32& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.u[0]), "r"(v.u[1]),
               "r"(v.u[2]), "r"(v.u[3]), "r"(v.u[4]), "r"(v.u[5]), "r"(v.u[6]), "r"(v.u[7])
               : "memory");
}

// 32 results of one row.  `add`: fp32 results are added to what is there.
__device__ __forceinline__ void store_row(const BlockParams& p, int row, int col, float* v, bool add) {
  if (row >= p.m || col >= p.n) return;
  if (p.dtype == MUONH_DTYPE_F32) {
    float* d = static_cast<float*>(p.d) + static_cast<int64_t>(row) * p.ldd + col;
    if (p.wide_store && col + 32 <= p.n) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        Vec32 o;
        if (add) {
          const float4 x = reinterpret_cast<const float4*>(d)[2 * q], y = reinterpret_cast<const float4*>(d)[2 * q + 1];
          v[8 * q] += x.x, v[8 * q + 1] += x.y, v[8 * q + 2] += x.z, v[8 * q + 3] += x.w;
          v[8 * q + 4] += y.x, v[8 * q + 5] += y.y, v[8 * q + 6] += y.z, v[8 * q + 7] += y.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o.u[j] = __float_as_uint(v[8 * q + j]);
        store32(d + 8 * q, o);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j < p.n) d[j] = add ? d[j] + v[j] : v[j];
    }
    return;
  }
  const bool bf16 = p.dtype == MUONH_DTYPE_BF16;
  uint32_t u[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (bf16) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<uint32_t*>(&h);
    } else {
      __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<uint32_t*>(&h);
    }
  }
  uint16_t* d = static_cast<uint16_t*>(p.d) + static_cast<int64_t>(row) * p.ldd + col;
  if (p.wide_store && col + 32 <= p.n) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      Vec32 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.u[j] = u[8 * q + j];
      store32(d + 16 * q, o);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col + j < p.n) d[j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
  }
}

// One result.
__device__ __forceinline__ void store_one(const BlockParams& p, int row, int col, float v) {
  if (row >= p.m || col >= p.n) return;
  const int64_t at = static_cast<int64_t>(row) * p.ldd + col;
  if (p.dtype == MUONH_DTYPE_F32) {
    float* d = static_cast<float*>(p.d) + at;
    *d = p.accumulate ? *d + v : v;
  } else if (p.dtype == MUONH_DTYPE_BF16) {
    static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
  } else {
    static_cast<__half*>(p.d)[at] = __float2half_rn(v);
  }
}

template <int BN, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    block_matmul_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ CUtensorMap amap,
                        const __grid_constant__ CUtensorMap bmap) {
  using C = BlockCfg<BN, PAIR>;
  constexpr int kCtas = PAIR ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + C::kStages;
  uint64_t* sfull = empty + C::kStages;
  uint64_t* sempty = sfull + kScaleRing;
  uint64_t* tfull = sempty + kScaleRing;
  uint64_t* tempty = tfull + C::kAccs;
  uint64_t* drain = tempty + C::kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  static_assert(!SPLIT || (!PAIR && BN == 64), "k is shared over 128 x 64 tiles");
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;   // 0 = leader: issues the MMAs, holds full, sfull and tempty
  // SPLIT: this CTA's k-blocks, in whole scale words; the cluster's tile is its worker number
  const uint32_t share = SPLIT ? cluster_ctarank() : 0, shares = SPLIT ? p.shares : 1;
  const int words = (p.k_blocks + 3) / 4;
  const int k_first = SPLIT ? 4 * static_cast<int>(words * share / shares) : 0;
  const int k_last = SPLIT ? min(p.k_blocks, 4 * static_cast<int>(words * (share + 1) / shares)) : p.k_blocks;
  const int worker = SPLIT ? blockIdx.x / shares : blockIdx.x / kCtas;
  const int workers = SPLIT ? gridDim.x / shares : gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) {
      mbar_init(&sfull[s], kCtas);
      mbar_init(&sempty[s], 1);
    }
    for (int a = 0; a < C::kAccs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpi * kCtas);
    }
    mbar_init(drain, 1);
    *err = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR)
      tmem_alloc_pair(tmem_slot, 512);
    else
      tmem_alloc(tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                      // barriers initialised in both CTAs
  tc_fence_after();
  wait_for_stream();
  const uint32_t tmem = *tmem_slot;
  auto arrive_leader = [&](uint64_t* bar) {
    if (PAIR)
      mbar_arrive_cluster(map_shared_rank(bar, 0));
    else
      mbar_arrive(bar);
  };
  auto commit = [&](uint64_t* bar) {             // in both CTAs of a pair
    if (PAIR)
      umma_commit_pair(bar);
    else
      umma_commit(bar);
  };

  // every role walks over the same (tile, chunk of k) sequence
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const int chunk = p.dtype == MUONH_DTYPE_F32 ? kChunkBlocks : p.k_blocks;
  float sum[SPLIT ? 32 : 1] = {};                // SPLIT: an epilogue thread's part of the tile

  if (warp == 0 || warp == 3) {
    if (lane == 0) {
      // ---------------------------------------------------------- TMA producers
      const bool role_a = warp == 0;             // also announces the stage's bytes
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;                            // up to kStages
      bool ok = true;
      for (int64_t t = worker; t < tiles && ok; t += workers) {
        int tm, tn;
        tile_at(p, t, tm, tn);
        const int row = role_a ? tm * C::kTileRows + static_cast<int>(rank) * kTm
                               : tn * BN + static_cast<int>(rank) * C::kBRows;
        for (int kb = k_first; kb < k_last; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, err)) {
            ok = false;
            break;
          }
          if (rank == 0 && role_a) mbar_expect_tx(&full[stage], kCtas * C::kStageBytes);
          uint8_t* dst = smem + stage * C::kStageBytes + (role_a ? 0 : C::kABytes);
          if (PAIR)
            tma_load_2d_pair(dst, role_a ? &amap : &bmap, map_shared_rank(&full[stage], 0), kb * kKBlock, row);
          else
            tma_load_2d(dst, role_a ? &amap : &bmap, &full[stage], kb * kKBlock, row);
          if (issued < C::kStages) ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // copies in flight land before a CTA may exit
      for (int j = 0; j < issued && rank == 0; ++j) {
        if (--stage < 0) {
          stage = C::kStages - 1;
          phase ^= 1u;
        }
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&full[stage], phase) && globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      const bool leader = elect_lane();
      int stage = 0, ring = 0, acc = 0;
      uint32_t phase = 0, ring_phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = worker; t < tiles && ok; t += workers) {
        int left = 0;                            // k-blocks until the accumulator is complete
        for (int kb = k_first; kb < k_last; ++kb) {
          const bool fresh = left == 0;
          if (fresh) {
            left = min(chunk, k_last - kb);
            if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, err)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          const uint32_t sc = tmem + C::kScaleCol + ring * 16;
          if ((kb & 3) == 0) {
            // copies and MMAs of one thread run in the order that they are
            // issued in, so the words are in place for the MMAs below and the
            // ones that they replace have been used
            if (!mbar_wait(&sfull[ring], ring_phase, err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t from = smem_u32(smem + C::kScaleOffset + ring * C::kScaleBytes);
            if (leader) {
#pragma unroll
              for (int b = 0; b < C::kScaleBlocks; ++b) {
                if (PAIR)
                  copy_scales_pair(sc + 4 * b, scale_desc(from + 512 * b));
                else
                  copy_scales(sc + 4 * b, scale_desc(from + 512 * b));
              }
              commit(&sempty[ring]);
            }
            __syncwarp();
          }
          if (!mbar_wait(&full[stage], phase, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + stage * C::kStageBytes), b = a + C::kABytes;
          const uint32_t idesc = idesc_mxf8(C::kTileRows, BN, kb & 3);
          const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
          if (leader) {
#pragma unroll
            for (int k = 0; k < kKBlock / 32; ++k) {   // 32 bytes of a row each
              if (PAIR)
                umma_mxf8_pair(tmem + acc * 128, ad + 2 * k, bd + 2 * k, idesc, sc, sc + 4, !fresh || k != 0);
              else
                umma_mxf8(tmem + acc * 128, ad + 2 * k, bd + 2 * k, idesc, sc, sc + 4, !fresh || k != 0);
            }
            commit(&empty[stage]);
            if (left == 1) commit(&tfull[acc]);
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (((kb & 3) == 3 || kb == k_last - 1) && ++ring == kScaleRing) {
            ring = 0;
            ring_phase ^= 1u;
          }
          if (--left == 0 && ++acc == C::kAccs) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (leader) commit(drain);
    }
    __syncwarp();
  } else if (warp == 2) {
    // --------------------------------------------------------- scale words
    // row r of a block of 128 is word r / 32 of the 16 bytes of TMEM lane r % 32;
    // a pair's CTAs each need the words of their own rows of A and of all of B
    int ring = 0;
    uint32_t ring_phase = 0;
    bool ok = true;
    for (int64_t t = worker; t < tiles && ok; t += workers) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int arow = tm * C::kTileRows + static_cast<int>(rank) * kTm;
      const uint8_t* rows[C::kScaleBlocks][4];
#pragma unroll
      for (int b = 0; b < C::kScaleBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int in_b = 128 * (b - 1) + 32 * j;     // of B's rows
          const int row = b == 0 ? arow + 32 * j + lane : tn * BN + in_b + lane;
          rows[b][j] = b == 0 ? (row < p.m ? p.sa + static_cast<int64_t>(row >> p.sa_shift) * p.ld_sa : nullptr)
                              : (in_b < BN && row < p.n ? p.sb + static_cast<int64_t>(row >> p.sb_shift) * p.ld_sb : nullptr);
        }
      for (int w0 = k_first / 4; 4 * w0 < k_last && ok; w0 += kScaleRing) {
        // kScaleRing groups at once: their loads are in flight together (one
        // group at a time, the MMAs waited for scales a third of the time)
        uint32_t u[kScaleRing][C::kScaleBlocks][4];
#pragma unroll
        for (int g = 0; g < kScaleRing; ++g)
#pragma unroll
          for (int b = 0; b < C::kScaleBlocks; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              u[g][b][j] = 4 * (w0 + g) < k_last
                               ? scale_word(rows[b][j], b == 0 ? p.sa_words : p.sb_words, w0 + g, p.k_blocks)
                               : 0u;
#pragma unroll
        for (int g = 0; g < kScaleRing; ++g) {
          if (4 * (w0 + g) >= k_last) break;
          if (!mbar_wait(&sempty[ring], ring_phase ^ 1u, err)) ok = false;
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          uint8_t* to = smem + C::kScaleOffset + ring * C::kScaleBytes + lane * 16;
#pragma unroll
          for (int b = 0; b < C::kScaleBlocks; ++b)
            *reinterpret_cast<uint4*>(to + 512 * b) = make_uint4(u[g][b][0], u[g][b][1], u[g][b][2], u[g][b][3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_leader(&sfull[ring]);
          if (++ring == kScaleRing) {
            ring = 0;
            ring_phase ^= 1u;
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    constexpr int kCols = BN / 2;                // columns per thread
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t t = worker; t < tiles && ok; t += workers) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int row = tm * C::kTileRows + static_cast<int>(rank) * kTm + quarter * 32 + lane;
      const int col = tn * BN + half * kCols;
      for (int kb = k_first; kb < k_last; kb += chunk) {
        if (!mbar_wait(&tfull[acc], acc_phase, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // all of it into registers first: the next tile's MMAs wait for this
        float v[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tmem + lanes + acc * 128 + half * kCols + 32 * c, v[c]);
        tc_fence_before();
        arrive_leader(&tempty[acc]);
        if (++acc == C::kAccs) {
          acc = 0;
          acc_phase ^= 1u;
        }
        if constexpr (SPLIT) {
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[j] += v[0][j];
        } else {
          const bool add = kb > 0 || p.accumulate;
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) store_row(p, row, col + 32 * c, v[c], add);
        }
      }
    }
  }

  if constexpr (SPLIT) {
    // the operands' space is free (every product is done): each CTA leaves its
    // sums there, 8 vectors per epilogue thread, and adds up and stores the
    // vectors whose number modulo the CTAs is its own
    __syncthreads();
    float4* const mine = reinterpret_cast<float4*>(smem) + (threadIdx.x - (kThreads - kEpi));
    if (warp >= 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        mine[j * kEpi] = make_float4(sum[4 * j], sum[4 * j + 1], sum[4 * j + 2], sum[4 * j + 3]);
    }
    cluster_sync();
    if (warp >= 4) {
      int tm, tn;
      tile_at(p, worker, tm, tn);
      const int row = tm * kTm + (warp & 3) * 32 + lane, col = tn * BN + ((warp - 4) >> 2) * (BN / 2);
      for (int j = share; j < 8; j += shares) {
        float4 total = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t r = 0; r < shares; ++r) {
          const float4 v = load_cluster_f4(map_shared_rank(mine + j * kEpi, r));
          total.x += v.x, total.y += v.y, total.z += v.z, total.w += v.w;
        }
        const float out[4] = {total.x, total.y, total.z, total.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) store_one(p, row, col + 4 * j + i, out[i]);
      }
    }
    cluster_sync();                              // no CTA leaves while another reads its sums
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    // no MMA may still write TMEM when a CTA frees it (the last commit arrives in both CTAs of a pair)
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
    }
  }
  if (PAIR) cluster_sync();                      // neither CTA's memory is in use by the other
  tc_fence_after();
  if (warp == 1) {
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *err) atomicOr(&g_block_timeout, 1);
}

// D = 0 where there is nothing to add up.
__global__ void __launch_bounds__(256) clear_rows_kernel(uint8_t* d, int64_t pitch, int64_t bytes, int64_t rows) {
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; j < bytes; j += static_cast<int64_t>(gridDim.x) * 256)
      d[r * pitch + j] = 0;
}

muonh_status block_fail(muonh_status st, const char* msg) {
  set_error_message(msg);
  return st;
}

template <int BN, bool PAIR, bool SPLIT>
cudaError_t launch_block(const BlockParams& p, const CUtensorMap& a, const CUtensorMap& b, int workers, cudaStream_t s) {
  const auto kernel = block_matmul_kernel<BN, PAIR, SPLIT>;
  static std::atomic<uint64_t> done;
  const cudaError_t e = allow_shared(kernel, done, BlockCfg<BN, PAIR>::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned cluster = PAIR ? 2u : SPLIT ? static_cast<unsigned>(p.shares) : 1u;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cluster * static_cast<unsigned>(workers));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = BlockCfg<BN, PAIR>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {programmatic_launch(), cluster_launch(cluster)};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, a, b);
}

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" muonh_status muonh_block_matmul(const muonh_block_operand* a, const muonh_block_operand* b, int64_t k,
                                           void* d, int64_t ldd, int32_t dtype, int32_t accumulate, void* stream) {
  set_error_message("");
  if (!a || !b) return block_fail(MUONH_ERR_INVALID_ARG, "an operand is NULL");
  if (a->rows < 0 || b->rows < 0 || k < 0 || a->rows > (1 << 30) || b->rows > (1 << 30) || k > (1 << 30))
    return block_fail(MUONH_ERR_INVALID_ARG, "rows and k must be in [0, 2^30]");
  if (dtype != MUONH_DTYPE_F32 && dtype != MUONH_DTYPE_BF16 && dtype != MUONH_DTYPE_F16)
    return block_fail(MUONH_ERR_INVALID_ARG, "dtype must be a MUONH_DTYPE_* type");
  if (accumulate && dtype != MUONH_DTYPE_F32)
    return block_fail(MUONH_ERR_INVALID_ARG, "only fp32 results can be accumulated");
  for (const muonh_block_operand* o : {a, b})
    if (o->block_rows != 1 && o->block_rows != 128)
      return block_fail(MUONH_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (a->rows == 0 || b->rows == 0) return MUONH_OK;
  if (!d || (a->rows > 1 && ldd < b->rows)) return block_fail(MUONH_ERR_INVALID_ARG, "d is NULL or its stride too small");
  const int size = dtype == MUONH_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(d) & (size - 1)) return block_fail(MUONH_ERR_ALIGNMENT, "d is not aligned to its type");
  const int64_t k_blocks = (k + kKBlock - 1) / kKBlock;
  for (const muonh_block_operand* o : {a, b}) {
    if (k == 0) break;
    if (!o->q || !o->scale || (o->rows > 1 && o->ld < k) || (o->rows > o->block_rows && o->ld_scale < k_blocks))
      return block_fail(MUONH_ERR_INVALID_ARG, "an operand's pointers are NULL or its strides too small");
    if ((reinterpret_cast<uintptr_t>(o->q) & 15) || (o->rows > 1 && o->ld % 16))
      return block_fail(MUONH_ERR_ALIGNMENT, "operands need 16-byte aligned rows");
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k == 0) {
    if (accumulate) return MUONH_OK;
    clear_rows_kernel<<<dim3(static_cast<unsigned>(std::min<int64_t>((b->rows * size + 255) / 256, 64)),
                             static_cast<unsigned>(std::min<int64_t>(a->rows, 4096))),
                        256, 0, s>>>(static_cast<uint8_t*>(d), ldd * size, b->rows * size, a->rows);
    return cudaGetLastError() == cudaSuccess ? MUONH_OK : block_fail(MUONH_ERR_CUDA, "launch of clear_rows_kernel failed");
  }
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  BlockParams p{};
  p.sa = a->scale;
  p.sb = b->scale;
  p.ld_sa = a->ld_scale;
  p.ld_sb = b->ld_scale;
  p.sa_shift = a->block_rows == 128 ? 7 : 0;
  p.sb_shift = b->block_rows == 128 ? 7 : 0;
  auto words = [](const muonh_block_operand* o) {
    return (reinterpret_cast<uintptr_t>(o->scale) & 3) == 0 && (o->rows <= o->block_rows || o->ld_scale % 4 == 0);
  };
  p.sa_words = words(a);
  p.sb_words = words(b);
  p.d = d;
  p.ldd = ldd;
  p.m = static_cast<int32_t>(a->rows);
  p.n = static_cast<int32_t>(b->rows);
  p.k_blocks = static_cast<int32_t>(k_blocks);
  p.dtype = dtype;
  p.accumulate = accumulate != 0;
  p.wide_store = (reinterpret_cast<uintptr_t>(d) & 31) == 0 && (a->rows == 1 || ldd * size % 32 == 0);
  // the pair's tiles where they fill the SMs, else narrower ones
  auto tiles = [&](int rows, int cols) {
    return static_cast<int64_t>((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols);
  };
  const bool pair = tiles(256, 256) >= sms / 2;
  const int bn = pair ? 256 : tiles(128, 128) >= sms ? 128 : 64, rows = pair ? 256 : kTm;
  p.tiles_m = (p.m + rows - 1) / rows;
  p.tiles_n = (p.n + bn - 1) / bn;
  p.band = pair ? 8 : 16;
  CUtensorMap amap, bmap;
  auto map = [&](CUtensorMap* out, const muonh_block_operand* o, int box_rows) {
    return encode_bytes(out, const_cast<void*>(o->q), k, o->rows, o->rows == 1 ? (k + 15) / 16 * 16 : o->ld, box_rows);
  };
  if (!map(&amap, a, kTm) || !map(&bmap, b, pair ? 128 : bn))
    return block_fail(MUONH_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  const int workers = static_cast<int>(std::min<int64_t>(tiles(rows, bn), pair ? sms / 2 : sms));
  // few tiles and a long k: up to 8 CTAs per tile, with 512 of k each at least
  p.shares = 1;
  // (clusters of 8 have to find 8 free SMs in one GPC: two thirds of the SMs at most)
  while (bn == 64 && p.shares < 8 && tiles(kTm, 64) * p.shares * 2 <= (p.shares == 4 ? sms * 2 / 3 : sms) &&
         k_blocks >= 8 * p.shares)
    p.shares *= 2;
  const cudaError_t e = pair           ? launch_block<256, true, false>(p, amap, bmap, workers, s)
                        : bn == 128    ? launch_block<128, false, false>(p, amap, bmap, workers, s)
                        : p.shares > 1 ? launch_block<64, false, true>(p, amap, bmap, workers, s)
                                       : launch_block<64, false, false>(p, amap, bmap, workers, s);
  if (e != cudaSuccess) return block_fail(MUONH_ERR_CUDA, "launch of block_matmul_kernel failed");
  return MUONH_OK;
}

cudaError_t muonh::take_block_timeout(int* flag, cudaStream_t s) { return take_flag(g_block_timeout, flag, s); }
