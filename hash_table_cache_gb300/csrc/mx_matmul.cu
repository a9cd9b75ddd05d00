// mx_matmul.cu -- hkv_mx_matmul: the product of two 4-bit microscaled matrices
// on the block-scaled 4-bit tensor cores.
//
// y[i][j] = sum_k A[i][k] B[j][k].  The rows of B are the rows of the tensor
// core's tile (128 of them, one TMEM lane each) and the rows of A its columns
// (16 to 192 of them), so one token still fills a tile with 128 useful rows,
// and a store of one TMEM column is contiguous along y's rows whatever y's
// alignment.  A step of k is 256 columns: 128 bytes of codes per row, brought
// by TMA in the 128-byte swizzle the tensor core reads, and two 512-byte
// groups of scales per 128 rows, which the format stores as they are copied
// to TMEM.  One warp loads, one issues the copies of scales and the products,
// four read the accumulators out; accumulators and scales are held twice, so
// a tile's output leaves while the next one is computed.
#include <cuda.h>

#include "mx.cuh"

namespace hkv {
namespace {

__device__ unsigned long long g_wait_timeouts;

constexpr int kRows = 128;       // rows of B per block
constexpr int kStepBytes = 128;  // bytes of codes per row and step: 256 columns
constexpr int kStep = 256;
constexpr int kStoreWarps = 8;   // two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kStoreWarps;  // warp 0 loads, warp 1 multiplies, the others store
constexpr int kMaxSplits = 8;
constexpr unsigned kSmemLimit = 232448 - 1024;  // 227 KB less the alignment of the stages

struct Problem {
  uint64_t m, n, k;
  uint64_t tiles_m, tiles_n;
  void* y;
  uint64_t stride;
  int type;
  bool pairs;   // two neighbours of a row of a 16-bit y may be stored at once
  bool staged;  // y is stored by TMA: its rows start on 16-byte boundaries
  bool whole;   // and end on them
  int splits;  // thread blocks of a cluster that share a tile's k
};

struct Maps {  // the codes and the scales of A and B, and y
  CUtensorMap a, b, a_scales, b_scales, y;
};

// Rows of y that leave through shared memory at once, 128 columns of them: 8 KB.
constexpr int kStageOut = 8192;
__host__ __device__ inline int rows_out(int type) { return type == HKV_F32 ? 16 : 32; }

// A tile of kBlocks * 128 rows of B by kCols rows of A, computed by one block
// or by the two of a pair.  Either block of a pair holds its own 128 rows of
// B, half of the rows of A, and the scales of its rows of B and of all of A's.
template <int kCols, int kBlocks>
struct Shape {
  static constexpr int kScaleRows = kCols > 128 ? 2 : 1;  // groups of 128 rows of A that a tile spans
  static constexpr int kACols = kCols / kBlocks;          // rows of A that a block loads
  static constexpr int kBBytes = kRows * kStepBytes, kABytes = kACols * kStepBytes;
  static constexpr int kStageBytes = kBBytes + kABytes + 1024 + 1024 * kScaleRows;
  static constexpr int kFit = (kSmemLimit - 1024 - 4 * kStageOut) / kStageBytes;
  static constexpr int kStages = kFit > 10 ? 10 : kFit;
  static constexpr int kOutAt = kStages * kStageBytes;  // four buffers for rows of y
  static constexpr int kSmem = kOutAt + 4 * kStageOut + 1024;
  // TMEM columns: two buffers of 256, each an accumulator and a step's scales
  static constexpr int kScaleCol = 192;
  static_assert(kCols <= kScaleCol && kScaleCol + 8 + 8 * kScaleRows <= 256, "TMEM columns");
  static_assert(kABytes % 1024 == 0, "swizzle");
};

// Bounded wait for a phase of a barrier: false after kWaitNs, with the
// device's count of timeouts raised.
constexpr uint64_t kWaitNs = 4000000000ull;
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t begin = now_ns();
  while (!mbar_try_wait(bar, parity))
    if (now_ns() - begin > kWaitNs) {
      atomicAdd(&g_wait_timeouts, 1ull);
      return false;
    }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || slow_wait(bar, parity);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
  uint32_t far;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(smem_u32(p)), "r"(rank));
  return far;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// A box into this block's shared memory, counted on a barrier given by its
// cluster address; a pair's loads are counted on its first block's barrier.
template <int kBlocks>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if constexpr (kBlocks == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared-memory descriptors: version 1, K-major.  Codes: rows of 128 bytes in
// the 128-byte swizzle, 1024 bytes from one group of 8 rows to the next.
// Scales: 32 rows of 16 bytes without a swizzle, 128 bytes per 8 rows.
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | 1ull << 16 | (1024ull >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (128ull >> 4) << 32 | 1ull << 46;
}
// Instruction descriptor of the block-scaled e2m1 product: both types e2m1,
// ue8m0 scales, `cols` columns, 128 or 256 rows, the pair of a scale word's
// bytes that a product of 64 columns takes (0 or 2).
__host__ __device__ constexpr uint32_t product_desc(int blocks, int cols, int pair) {
  return (uint32_t)pair << 4 | 1u << 7 | 1u << 10 | (uint32_t)(cols >> 3) << 17 | 1u << 23 |
         (uint32_t)(blocks * kRows >> 4) << 24 | (uint32_t)pair << 29;
}

// For a pair, the first block's thread issues these for both blocks: each
// copies its own scales and multiplies its own rows of B by both halves of A.
template <int kBlocks>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (kBlocks == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}
template <int kBlocks>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sa, uint32_t sb, bool add) {
  if constexpr (kBlocks == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::
            "r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::
            "r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
}
// The barrier (in both blocks of a pair) is reached when the products issued
// so far by this thread are done.
template <int kBlocks>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kBlocks == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
            "r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(smem_u32(bar))
                 : "memory");
}
// All of an SM's TMEM, by one warp of each block.
template <int kBlocks>
__device__ __forceinline__ void take_tmem(uint32_t* base) {
  if constexpr (kBlocks == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int kBlocks>
__device__ __forceinline__ void give_tmem(uint32_t tmem) {
  if constexpr (kBlocks == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}
__device__ __forceinline__ void read_columns(uint32_t tmem, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(tmem));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_one(const Problem& p, uint64_t i, uint64_t j, float v) {
  const uint64_t at = i * p.stride + j;
  if (p.type == HKV_F32) static_cast<float*>(p.y)[at] = v;
  else if (p.type == HKV_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p.y)[at] = __float2half_rn(v);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Sixteen accumulator columns (rows i .. i + 15 of y, all of them in y) of
// this lane's column j of a 16-bit y: neighbouring lanes trade values, so
// that an even lane stores both lanes' columns of one row and the odd lane
// those of the next, 4 bytes at a time.
template <bool kBf16>
__device__ __forceinline__ void store_pairs(const Problem& p, uint64_t i, uint64_t j,
                                            const float (&v)[16]) {
  const uint32_t odd = j & 1, pick = odd ? 0x3276 : 0x5410;
  const uint64_t step = 4 * p.stride;
  char* y = static_cast<char*>(p.y) + ((i + odd) * p.stride + (j & ~1ull)) * 2;
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    const uint32_t own = pack2<kBf16>(v[c], v[c + 1]);
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
    *reinterpret_cast<uint32_t*>(y) = __byte_perm(own, other, pick);
    y += step;
  }
}

// Sixteen accumulator columns of this lane's column j.
__device__ __forceinline__ void store_columns(const Problem& p, uint64_t i, uint64_t j,
                                              const float (&v)[16]) {
  // a whole warp's columns lie in y, and all sixteen rows
  const bool inside = i + 16 <= p.m && (j | 31) < p.n;
  if (inside && p.pairs) {
    if (p.type == HKV_BF16) store_pairs<true>(p, i, j, v);
    else store_pairs<false>(p, i, j, v);
  } else if (inside && p.type == HKV_F32) {
    char* y = reinterpret_cast<char*>(static_cast<float*>(p.y) + i * p.stride + j);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      *reinterpret_cast<float*>(y) = v[c];
      y += 4 * p.stride;
    }
  } else if (j < p.n) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (i + c < p.m) store_one(p, i + c, j, v[c]);
  }
}

// One lane of a converged warp.  What only that lane does is then known to be
// the work of one thread: a branch on the lane's number leaves the operands
// of the tensor core's instructions in per-lane registers, and issuing them
// took longer than the products.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}

// The four storing warps that share a set of columns: a barrier, and whether
// something holds for all of them.
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool group_all(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(group + 1)
      : "memory");
  return r != 0;
}

// Sixteen accumulator columns of column `j` of the tile into sixteen rows of a
// buffer of 128 columns.
__device__ __forceinline__ void stage_columns(uint8_t* buffer, int j, int type,
                                              const float (&v)[16]) {
  if (type == HKV_F32) {
    float* to = reinterpret_cast<float*>(buffer) + j;
#pragma unroll
    for (int c = 0; c < 16; ++c) to[c * kRows] = v[c];
  } else {
    uint16_t* to = reinterpret_cast<uint16_t*>(buffer) + j;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const uint32_t two = type == HKV_BF16 ? pack2<true>(v[c], v[c + 1]) : pack2<false>(v[c], v[c + 1]);
      to[c * kRows] = static_cast<uint16_t>(two);
      to[(c + 1) * kRows] = static_cast<uint16_t>(two >> 16);
    }
  }
}
// A buffer's rows to y; rows and 16-byte pieces past y are left out.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* from) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                   "l"(map), "r"(x), "r"(y), "r"(smem_u32(from))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The tiles of a block: every `step`-th from `first`, along y's rows first.
struct Tiles {
  uint64_t row, col, step_row, step_col, left;  // in tiles; left: tiles still to come
  __device__ __forceinline__ Tiles(const Problem& p, uint64_t first, uint64_t step) {
    const uint64_t all = p.tiles_m * p.tiles_n;
    row = first / p.tiles_n;
    col = first % p.tiles_n;
    step_row = step / p.tiles_n;
    step_col = step % p.tiles_n;
    left = first < all ? (all - first + step - 1) / step : 0;
  }
  __device__ __forceinline__ void next(const Problem& p) {
    row += step_row;
    col += step_col;
    if (col >= p.tiles_n) {
      col -= p.tiles_n;
      ++row;
    }
    --left;
  }
};

template <int kCols, int kBlocks>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Problem p) {
  using S = Shape<kCols, kBlocks>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ uint64_t full[S::kStages], empty[S::kStages], ready[2], drained[2];
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The blocks of a cluster: a pair (kBlocks 2), or the `splits` that share a
  // tile's k (kBlocks 1).
  const uint32_t splits = kBlocks == 2 ? 1 : p.splits;
  const uint32_t rank = blockIdx.x % (splits * kBlocks);
  const uint32_t half_of = kBlocks == 2 ? rank : 0, part = kBlocks == 2 ? 0 : rank;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ready[b], 1);
      mbar_init(&drained[b], kStoreWarps * kBlocks);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) take_tmem<kBlocks>(&tmem_base);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (kBlocks == 2) cluster_sync();  // the other block's barriers are ready
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  pdl_trigger();
  pdl_wait();  // every role: the bounded waits below start when the inputs are there

  Tiles t(p, blockIdx.x / (splits * kBlocks), gridDim.x / (splits * kBlocks));
  const uint64_t all = (p.k + kStep - 1) / kStep;
  const uint64_t k0 = all * part / splits, k1 = all * (part + 1) / splits;

  if (warp == 0 && elect()) {
    uint32_t it = 0;
    bool ok = true;
    for (; t.left && ok; t.next(p)) {
      const int n0 = static_cast<int>((t.col * kBlocks + half_of) * kRows);
      const uint64_t m0 = t.row * kCols;
      for (uint64_t k = k0; k < k1; ++k, ++it) {
        const uint32_t s = it % S::kStages;
        if (it >= S::kStages && !wait(&empty[s], (it / S::kStages + 1) & 1)) {
          ok = false;
          break;
        }
        uint8_t* stage = smem + s * S::kStageBytes;
        uint8_t* scales = stage + S::kBBytes + S::kABytes;
        const int x = static_cast<int>(k * kStepBytes), xs = static_cast<int>(k * 256);
        uint32_t bar = smem_u32(&full[s]);
        if (kBlocks == 2) bar = cluster_address(&full[s], 0);
        if (half_of == 0) mbar_arrive_expect_tx(&full[s], kBlocks * S::kStageBytes);
        tma_load<kBlocks>(stage, &maps.b, x, n0, bar);
        tma_load<kBlocks>(stage + S::kBBytes, &maps.a, x,
                          static_cast<int>(m0 + half_of * S::kACols), bar);
        tma_load<kBlocks>(scales, &maps.b_scales, xs, n0 / 128, bar);
        tma_load<kBlocks>(scales + 1024, &maps.a_scales, xs, static_cast<int>(m0 / 128), bar);
      }
    }
    // Before the block ends: the loads still in flight where a wait ran out,
    // and in a pair the products' arrivals on this block's barriers.
    if (!ok || kBlocks == 2)
      for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i)
        if (!wait(ok ? &empty[i % S::kStages] : &full[i % S::kStages], (i / S::kStages) & 1)) break;
  } else if (warp == 1 && half_of == 0 && elect()) {
    uint32_t it = 0, n_tile = 0;
    bool ok = true;
    for (; t.left && ok; t.next(p), ++n_tile) {
      const uint32_t b = n_tile & 1;
      const uint32_t d = tmem + b * 256;
      // the scales of a tile that starts in the middle of a group of 128 rows
      // (192 columns: at 0 or 64, so that the shift is even, as it has to be)
      const uint32_t shift = kCols > 128 ? t.row * kCols % 128 / 32 : 0;
      if (n_tile >= 2 && !wait(&drained[b], (n_tile / 2 + 1) & 1)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (uint64_t k = k0; k < k1; ++k, ++it) {
        const uint32_t s = it % S::kStages;
        if (!wait(&full[s], (it / S::kStages) & 1)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t stage = smem_u32(smem) + s * S::kStageBytes;
        const uint32_t sc = stage + S::kBBytes + S::kABytes;
        const uint64_t db = codes_desc(stage), da = codes_desc(stage + S::kBBytes);
        // two sets of scale columns, used by turns: a step's copies do not
        // wait for the products of the step before
        const uint32_t sb = tmem + (it & 1) * 256 + S::kScaleCol, sa = sb + 8;
        const int products = p.k - k * kStep >= kStep ? 4 : static_cast<int>((p.k - k * kStep + 63) / 64);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          copy_scales<kBlocks>(sb + 4 * g, scales_desc(sc + 512 * g));
#pragma unroll
          for (int r = 0; r < S::kScaleRows; ++r)
            copy_scales<kBlocks>(sa + 4 * (S::kScaleRows * g + r),
                                 scales_desc(sc + 1024 + 1024 * r + 512 * g));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= products) break;
          product<kBlocks>(d, db + 2 * q, da + 2 * q, product_desc(kBlocks, kCols, 2 * (q & 1)),
                           sb + 4 * (q / 2), sa + 4 * S::kScaleRows * (q / 2) + shift,
                           k > k0 || q > 0);
        }
        commit<kBlocks>(&empty[s]);
      }
      if (ok) commit<kBlocks>(&ready[b]);
    }
    if (!ok) {  // products in flight end before TMEM is given back
      commit<kBlocks>(&ready[0]);
      commit<kBlocks>(&ready[1]);
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;  // the TMEM lanes this warp can read
    const int row = quarter * 32 + lane;
    const bool issues = quarter == 0 && lane == 0;  // this group's stores by TMA
    uint8_t* out = smem + S::kOutAt + half * 2 * kStageOut;
    uint32_t n_tile = 0, n_out = 0;
    for (Tiles u = t; u.left; u.next(p), ++n_tile) {
      const uint32_t b = n_tile & 1;
      // all four warps of a group go on, or none
      if (!group_all(half, wait(&ready[b], (n_tile / 2) & 1))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint64_t n0 = (u.col * kBlocks + half_of) * kRows, m0 = u.row * kCols;
      const int cols = n0 >= p.n          ? 0
                       : p.m - m0 < kCols ? static_cast<int>(p.m - m0)
                                          : kCols;
      const uint32_t d = tmem + b * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
      // TMA writes whole 16 bytes: a ragged end of y's rows is not its work
      const bool staged = p.staged && (p.whole || n0 + kRows <= p.n);
      const int at_once = staged ? rows_out(p.type) : 16;
      for (int c = at_once * half; c < cols; c += 2 * at_once) {
        float v[16];
        if (staged) {
          uint8_t* buffer = out + (n_out++ & 1) * kStageOut;
          if (issues)  // the buffer's rows of two rounds ago have left it
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          group_sync(half);
          for (int q = 0; q < at_once && c + q < cols; q += 16) {
            read_columns(d + c + q, v);
            stage_columns(buffer + q * kRows * (p.type == HKV_F32 ? 4 : 2), row, p.type, v);
          }
          fence_proxy_async_smem();
          group_sync(half);
          if (issues)
            tma_store(&maps.y, static_cast<int>(n0), static_cast<int>(m0 + c), buffer);
          continue;
        }
        read_columns(d + c, v);
        if (splits == 1) {
          store_columns(p, m0 + c, n0 + row, v);
        } else {  // this block's part of the sum, for the cluster to add up
          float* mine = reinterpret_cast<float*>(smem) + row;
#pragma unroll
          for (int q = 0; q < 16; ++q) mine[(c + q) * kRows] = v[q];
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (kBlocks == 2) mbar_arrive_at(cluster_address(&drained[b], 0));
        else mbar_arrive(&drained[b]);
      }
    }
    if (issues) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  if (splits > 1) {
    cluster_sync();
    if (warp >= 2) {
      const int row = (warp & 3) * 32 + lane, half = (warp - 2) >> 2;
      const uint64_t j = t.col * kRows + row, m0 = t.row * kCols;
      const int cols = p.m - m0 < kCols ? static_cast<int>(p.m - m0) : kCols;
      const uint32_t parts = smem_u32(smem) + row * 4;
      for (int c = 2 * part + half; c < cols; c += 2 * splits) {
        float v = 0.f;
        for (uint32_t r = 0; r < splits; ++r) v += remote_f32(parts + c * kRows * 4, r);
        if (j < p.n) store_one(p, m0 + c, j, v);
      }
    }
    __syncwarp();
    cluster_sync();  // the others may still read this block's part
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // in a pair the other block may still use this one's barriers and TMEM
  if (kBlocks == 2) cluster_sync();
  if (warp == 1) give_tmem<kBlocks>(tmem);
}

__global__ void zero_kernel(const __grid_constant__ Problem p) {
  pdl_wait();
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.m * p.n; i += step)
    store_one(p, i / p.n, i % p.n, 0.f);
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) !=
            cudaSuccess || r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A matrix's codes as boxes of 128 bytes by `box` rows, swizzled, and its
// scales as boxes of two 512-byte groups by `groups`; what lies past the
// matrix reads as zeros.
bool make_maps(CUtensorMap* codes_map, CUtensorMap* scales_map, const uint8_t* codes,
               const uint8_t* scales, uint64_t rows, uint64_t k, int box, int groups) {
  EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint32_t steps[2] = {1, 1};
  const uint64_t bytes = (k + kMxBlock - 1) / kMxBlock * 16;
  const cuuint64_t dims[2] = {bytes, rows}, strides[1] = {bytes};
  const cuuint32_t boxes[2] = {kStepBytes, static_cast<cuuint32_t>(box)};
  const uint64_t words = (k + 127) / 128 * 128;  // of 4 bytes
  const cuuint64_t sdims[2] = {words, (rows + 127) / 128}, sstrides[1] = {words * 4};
  const cuuint32_t sboxes[2] = {256, static_cast<cuuint32_t>(groups)};
  return f(codes_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides,
           boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         f(scales_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(scales), sdims,
           sstrides, sboxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y as boxes of 128 columns.
bool make_y_map(CUtensorMap* map, const Problem& p) {
  const CUtensorMapDataType type = p.type == HKV_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : p.type == HKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t steps[2] = {1, 1};
  const cuuint64_t dims[2] = {p.n, p.m}, strides[1] = {p.stride * type_size(p.type)};
  const cuuint32_t boxes[2] = {kRows, static_cast<cuuint32_t>(rows_out(p.type))};
  EncodeFn f = encode_fn();
  return f && f(map, type, 2, p.y, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operands {
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
};

template <int kCols, int kBlocks>
cudaError_t run(Problem p, const Operands& o, cudaStream_t st) {
  using S = Shape<kCols, kBlocks>;
  p.tiles_m = (p.m + kCols - 1) / kCols;
  p.tiles_n = (p.n + kRows * kBlocks - 1) / (kRows * kBlocks);
  const uint64_t tiles = p.tiles_m * p.tiles_n, steps = (p.k + kStep - 1) / kStep;
  const uint64_t sms = sm_count();
  // few tiles: a cluster shares a tile's k while SMs are idle and each block
  // keeps two steps at least
  p.splits = 1;
  while (kBlocks == 1 && p.splits < kMaxSplits && tiles * p.splits * 2 <= sms &&
         steps >= 4ull * p.splits)
    p.splits *= 2;
  Maps maps{};
  if (!make_maps(&maps.a, &maps.a_scales, o.a_codes, o.a_scales, p.m, p.k, S::kACols, S::kScaleRows) ||
      !make_maps(&maps.b, &maps.b_scales, o.b_codes, o.b_scales, p.n, p.k, kRows, 1))
    return cudaErrorUnknown;
  // TMA wants 16-byte boundaries and a stride below 2^40 bytes
  const uint64_t row_bytes = p.stride * type_size(p.type);
  p.staged = p.splits == 1 && aligned(p.y, 16) && row_bytes % 16 == 0 && row_bytes < 1ull << 40;
  p.whole = p.n * type_size(p.type) % 16 == 0;
  if (p.staged && !make_y_map(&maps.y, p)) return cudaErrorUnknown;
  auto* kernel = matmul_kernel<kCols, kBlocks>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const uint32_t cluster = p.splits * kBlocks;
  const uint64_t clusters = p.splits > 1 || tiles < sms / kBlocks ? tiles : sms / kBlocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

cudaError_t matmul(const Problem& p, const Operands& o, cudaStream_t st) {
  if (p.k == 0) return launch_chained(zero_kernel, sm_count() * 4, 256, 0, st, p);
  if (p.m <= 16) return run<16, 1>(p, o, st);
  if (p.m <= 32) return run<32, 1>(p, o, st);
  if (p.m <= 64) return run<64, 1>(p, o, st);
  if (p.m <= 128) return run<128, 1>(p, o, st);
  // pairs halve what a block loads of A; one block per tile has twice as many
  // tiles to spread over the SMs
  const uint64_t pairs = (p.m + 191) / 192 * ((p.n + 255) / 256);
  if (pairs * 2 > static_cast<uint64_t>(sm_count())) return run<192, 2>(p, o, st);
  return run<192, 1>(p, o, st);
}

}  // namespace
}  // namespace hkv

extern "C" {

hkv_status hkv_mx_matmul(uint64_t m, uint64_t n, uint64_t k, const uint8_t* a_codes,
                         const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                         void* y, int y_type, uint64_t y_stride, void* stream) {
  using namespace hkv;
  if (m > HKV_MAX_BATCH || n > HKV_MAX_BATCH || k > HKV_MAX_BATCH || y_stride < n ||
      !type_ok(y_type))
    return HKV_ERR_INVALID;
  if (m == 0 || n == 0) return HKV_OK;
  if (!y || !aligned(y, type_size(y_type))) return HKV_ERR_INVALID;
  if (k && (!a_codes || !a_scales || !b_codes || !b_scales)) return HKV_ERR_INVALID;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(b_codes, 16) ||
      !aligned(b_scales, 16))
    return HKV_ERR_INVALID;
  Problem p{};
  p.m = m;
  p.n = n;
  p.k = k;
  p.y = y;
  p.stride = y_stride;
  p.type = y_type;
  p.pairs = y_type != HKV_F32 && aligned(y, 4) && y_stride % 2 == 0;
  return op_status(matmul(p, {a_codes, a_scales, b_codes, b_scales}, static_cast<cudaStream_t>(stream)));
}

hkv_status hkv_get_wait_timeouts(uint64_t* timeouts_host) {
  if (!timeouts_host) return HKV_ERR_INVALID;
  unsigned long long v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, hkv::g_wait_timeouts, sizeof(v));
  if (e != cudaSuccess) return hkv::op_status(e);
  *timeouts_host = v;
  return v ? HKV_ERR_TIMEOUT : HKV_OK;
}

}  // extern "C"
