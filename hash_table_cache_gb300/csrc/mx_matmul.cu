// mx_matmul.cu -- hkv_mx_matmul: the product of two 4-bit microscaled matrices
// on the block-scaled 4-bit tensor cores.
//
// y[i][j] = sum_k A[i][k] B[j][k].  One of the two matrices lies along the
// lanes of the tensor core's tile (128 rows, one TMEM lane each, or 256 for a
// pair of blocks), the other along its columns (16 to 192).  A step of k is
// 256 columns: 128 bytes of codes per row, brought by TMA in the 128-byte
// swizzle the tensor core reads, and two 512-byte groups of scales per 128
// rows, which the format stores as they are copied to TMEM.  One warp loads,
// one issues the copies of scales and the products, and 4 (16 columns), 8, or 12
// (192 columns and short k) read the accumulators out; accumulators and scales
// are held twice, so a tile's output leaves while the next one is computed.
//
// TMEM hands a thread one lane: neighbouring columns of one row of the tile.
// With A in the lanes that is a piece of a row of y, and a warp turns its 32
// pieces around in shared memory so that a store covers whole 128-byte lines
// (a thread storing its own piece, a 32-byte sector of 32 rows at once,
// reached 4.4 TB/s of y where this reaches 5.7: 2048 x 131072 x 64).  With B
// in the lanes a warp's lanes are 32 neighbouring columns of one row of y:
// that is for the few rows of a token or a small batch, which would leave most
// lanes empty the other way.
//
// Bounds and times (GB300): 8192 x 8192 x 8192 into bfloat16 159 us, 6.9
// PFLOP/s, the tensor pipe active for 74% of the cycles (137 us without the
// loads, 142 without the products), into float32 178 us; 4096 x 4096 x 4096 27
// and 34 us; 2048 x 131072 x 64 95 and 173 us, bound by the writes of y; 16 x
// 8192 x 8192 9.9 us, 3.6 TB/s of codes and scales; one row by 4096 x 4096 4.5
// us, a launch and the latencies of one pass.
#include <cuda.h>
#include <type_traits>

#include "mx.cuh"

namespace hkv {
namespace {

__device__ unsigned long long g_wait_timeouts;

constexpr int kRows = 128;       // lanes per block
constexpr int kStepBytes = 128;  // bytes of codes per row and step: 256 columns
constexpr int kStep = 256;
constexpr int kMaxSplits = 8;
constexpr unsigned kSmemLimit = 232448 - 1024;  // 227 KB less the alignment of the stages

struct Problem {
  uint64_t lanes, cols, k;      // rows of the matrix in the lanes and of the one in the columns
  uint32_t along, down;         // tiles along y's rows and down its columns
  void* y;
  uint64_t stride;
  int type;
  bool wide;   // y's rows start on 16-byte boundaries
  int splits;  // thread blocks of a cluster that share a tile's k
};

// Where a warp turns 32 pieces of rows around: 128 bytes, and 16 before them
// for what precedes the piece in its row, which also keeps either side of the
// turn from meeting a bank twice.
constexpr int kTurnPitch = 144, kTurnWarp = 32 * kTurnPitch;

struct Maps {  // codes and scales of the two matrices
  CUtensorMap lanes, cols, lanes_scales, cols_scales;
};

// A tile of kBlocks * 128 lanes by kCols columns, computed by one block or by
// the two of a pair.  Either block of a pair holds its own 128 rows of the
// lanes' matrix, half of the columns' matrix's rows, and the scales of its
// lanes and of all columns.  Warp 0 loads, warp 1 multiplies; kGroups groups of
// four warps, one for each quarter of the lanes, share the columns.
template <int kCols, int kBlocks, int kGroups>
struct Shape {
  static constexpr int kScaleRows = kCols > 128 ? 2 : 1;  // groups of 128 rows that the columns span
  static constexpr int kOwnCols = kCols / kBlocks;        // columns' rows that a block loads
  static constexpr int kLaneBytes = kRows * kStepBytes, kColBytes = kOwnCols * kStepBytes;
  static constexpr int kStageBytes = kLaneBytes + kColBytes + 1024 + 1024 * kScaleRows;
  static constexpr int kGroupCols = kCols / kGroups;
  static constexpr int kStoreWarps = 4 * kGroups, kThreads = 64 + 32 * kStoreWarps;
  static constexpr int kTurnBytes = kCols == 192 ? kStoreWarps * kTurnWarp : 0;
  static constexpr int kFit = (kSmemLimit - 1024 - kTurnBytes) / kStageBytes;
  static constexpr int kStages = kFit > 10 ? 10 : kFit;
  static constexpr int kTurnAt = kStages * kStageBytes;
  static constexpr int kSmem = kTurnAt + kTurnBytes + 1024;
  // TMEM columns: two buffers of 256, each an accumulator and a step's scales
  static constexpr int kScaleCol = 192;
  static_assert(kCols <= kScaleCol && kScaleCol + 8 + 8 * kScaleRows <= 256, "TMEM columns");
  static_assert(kColBytes % 1024 == 0, "swizzle");
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
// The same by a whole warp, with one answer for all of its lanes: each lane has a
// limit of its own, and a warp that parted at it must not run instructions that
// its lanes have to run together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity));
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

// Shared-memory descriptors, version 1, K-major.  Codes: rows of 128 bytes in
// the 128-byte swizzle, 1024 bytes from one group of 8 rows to the next.
// Scales: 32 rows of 16 bytes without a swizzle, 128 bytes per 8 rows.  The
// upper halves are constants; the lower halves hold the address in 16-byte
// units, in which the issuing thread counts.
constexpr uint32_t kCodesDesc = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kScalesDesc = (128 >> 4) | 1u << 14;
__device__ __forceinline__ uint32_t desc_units(uint32_t addr) { return (addr & 0x3FFFF) >> 4; }

// Instruction descriptor of the block-scaled e2m1 product: both types e2m1,
// ue8m0 scales, `cols` columns, 128 or 256 rows, the pair of a scale word's
// bytes that a product of 64 columns takes (0 or 2).
__host__ __device__ constexpr uint32_t product_desc(int blocks, int cols, int pair) {
  return (uint32_t)pair << 4 | 1u << 7 | 1u << 10 | (uint32_t)(cols >> 3) << 17 | 1u << 23 |
         (uint32_t)(blocks * kRows >> 4) << 24 | (uint32_t)pair << 29;
}

// For a pair, the first block's thread issues these for both blocks: each
// copies its own scales and multiplies its own lanes by both blocks' columns.
template <int kBlocks>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t from) {
  if constexpr (kBlocks == 2)
    asm volatile(
        "{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n"
        " tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n}" ::"r"(tmem),
        "r"(from), "n"(kScalesDesc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n"
        " tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n}" ::"r"(tmem),
        "r"(from), "n"(kScalesDesc)
        : "memory");
}
template <int kBlocks>
__device__ __forceinline__ void product(uint32_t d, uint32_t lanes, uint32_t cols, uint32_t idesc,
                                        uint32_t s_lanes, uint32_t s_cols, uint32_t add) {
  if constexpr (kBlocks == 2)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n"
        " mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n}" ::
            "r"(d),
        "r"(lanes), "r"(cols), "r"(idesc), "r"(s_lanes), "r"(s_cols), "r"(add), "n"(kCodesDesc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n"
        " mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n}" ::
            "r"(d),
        "r"(lanes), "r"(cols), "r"(idesc), "r"(s_lanes), "r"(s_cols), "r"(add), "n"(kCodesDesc)
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

// kN accumulator columns of this warp's TMEM lanes into v from kFrom on, on
// their way until columns_read().
template <int kFrom, int kN, int N>
__device__ __forceinline__ void read_columns(uint32_t tmem, float (&v)[N]) {
  static_assert(kN % 16 == 0 && kFrom + kN <= N, "columns");
#pragma unroll
  for (int c = 0; c < kN; c += 16) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v) + kFrom + c;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(tmem + c));
  }
}
// Eight of them.
template <int kFrom, int N>
__device__ __forceinline__ void read_eight(uint32_t tmem, float (&v)[N]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v) + kFrom;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(tmem));
}
template <int N>
__device__ __forceinline__ void columns_read(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < N; ++c) asm volatile("" : "+f"(v[c]));  // used after the wait only
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

// Columns j .. j + 3 of row i of y, with B in the lanes.
__device__ __forceinline__ void store_four(const Problem& p, uint64_t i, uint64_t j, float4 v) {
  const uint64_t at = i * p.stride + j;
  if (p.wide && j + 4 <= p.lanes) {
    if (p.type == HKV_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
          p.type == HKV_BF16 ? make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w))
                             : make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
    return;
  }
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (j + k < p.lanes) store_one(p, i, j + k, e[k]);
}

// B in the lanes: N accumulator columns are rows of y from i on, of this
// lane's column j.
template <int N>
__device__ __forceinline__ void store_columns(const Problem& p, uint64_t i, uint64_t j,
                                              const float (&v)[N]) {
  if (j >= p.lanes) return;
  if (i + N <= p.cols && p.type != HKV_F32) {  // no test per row
    uint16_t* y = static_cast<uint16_t*>(p.y) + i * p.stride + j;
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint32_t two = p.type == HKV_BF16 ? pack2<true>(v[c], v[c + 1]) : pack2<false>(v[c], v[c + 1]);
      *y = static_cast<uint16_t>(two);
      y[p.stride] = static_cast<uint16_t>(two >> 16);
      y += 2 * p.stride;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (i + c < p.cols) store_one(p, i + c, j, v[c]);
}

// 16 bytes of a row of y from accumulator columns kFrom on.
template <int kType, int kFrom, int N>
__device__ __forceinline__ uint4 word_of(const float (&v)[N]) {
  if constexpr (kType == HKV_F32)
    return make_uint4(__float_as_uint(v[kFrom]), __float_as_uint(v[kFrom + 1]),
                      __float_as_uint(v[kFrom + 2]), __float_as_uint(v[kFrom + 3]));
  else
    return make_uint4(pack2<kType == HKV_BF16>(v[kFrom], v[kFrom + 1]),
                      pack2<kType == HKV_BF16>(v[kFrom + 2], v[kFrom + 3]),
                      pack2<kType == HKV_BF16>(v[kFrom + 4], v[kFrom + 5]),
                      pack2<kType == HKV_BF16>(v[kFrom + 6], v[kFrom + 7]));
}
template <int kType, int kFrom, int kN, int N>
__device__ __forceinline__ void stage_row(uint8_t* row, const float (&v)[N]) {
  constexpr int kPer = kType == HKV_F32 ? 4 : 8;
  *reinterpret_cast<uint4*>(row) = word_of<kType, kFrom>(v);
  if constexpr (kN > kPer) stage_row<kType, kFrom + kPer, kN - kPer>(row + 16, v);
}

// A in the lanes: columns kFrom .. kFrom + kN - 1 of v are columns j ..
// j + kN - 1 of y, a piece of each of the warp's rows, from i on.  kWide: y's
// rows start on 16-byte boundaries.  Otherwise every row is cut at the
// boundaries that it has in y.  A word that lies across the start of a piece
// is the work of that piece, for which `before` are the columns before it (the
// last of them in before[kBefore + 7]); the tile's first and last words, whose
// rest belongs to other tiles, are stored element by element (`starts`, `ends`).
template <int kType, bool kWide, int kFrom, int kN, int kBefore, int N, int M>
__device__ __forceinline__ void turn_and_store(uint8_t* room, const Problem& p, uint64_t i,
                                               uint64_t j, const float (&v)[N],
                                               const float (&before)[M], bool starts, bool ends) {
  constexpr int kSize = kType == HKV_F32 ? 4 : 2, kPer = 16 / kSize;
  constexpr int kLanes = kN * kSize / 16;  // threads that store a row's piece, 16 bytes each
  constexpr int kRowsAtOnce = 32 / kLanes;
  static_assert(kN * kSize <= 128 && 32 % kLanes == 0, "a piece of a row");
  using E = std::conditional_t<kSize == 4, uint32_t, uint16_t>;
  const int lane = threadIdx.x & 31;
  uint8_t* mine = room + lane * kTurnPitch;
  if constexpr (!kWide)
    *reinterpret_cast<uint4*>(mine) = word_of<kType, kBefore + 8 - kPer>(before);
  stage_row<kType, kFrom, kN>(mine + 16, v);
  __syncwarp();
  const int first = lane / kLanes, at = lane % kLanes;
  const uint8_t* from = room + first * kTurnPitch + 16;
  char* y = static_cast<char*>(p.y) + ((i + first) * p.stride + j) * kSize;
  const uint64_t step = kRowsAtOnce * p.stride * kSize;
  // what of the piece lies in y, and how many of this thread's rows
  const int cols = p.cols - j < kN ? static_cast<int>(p.cols - j) : kN;
  const int rows = p.lanes - i < 32 ? (static_cast<int>(p.lanes - i) - first + kRowsAtOnce - 1) / kRowsAtOnce
                                    : kLanes;
  // (__stcs, not the library's asm store, behind which no load would move up)
  if (cols == kN && rows == kLanes) {
    ends |= j + kN == p.cols;
#pragma unroll
    for (int r = 0; r < kLanes; ++r, y += step, from += kRowsAtOnce * kTurnPitch) {
      const uint4 word = *reinterpret_cast<const uint4*>(from + at * 16);
      if constexpr (kWide) {
        __stcs(reinterpret_cast<uint4*>(y) + at, word);
      } else {
        // the word from the boundary at or before the piece's start on
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(y) & 15);
        const uint4 left = *reinterpret_cast<const uint4*>(from + at * 16 - 16);
        uint32_t x[8] = {left.x, left.y, left.z, left.w, word.x, word.y, word.z, word.w};
        shift_bytes(x, (16 - off) & 15);
        const int head = static_cast<int>((16 - off) / kSize), tail = static_cast<int>(off / kSize);
        const uint4 cut = make_uint4(off ? x[0] : word.x, off ? x[1] : word.y, off ? x[2] : word.z,
                                     off ? x[3] : word.w);
        if (off == 0 || at > 0 || !starts) __stcs(reinterpret_cast<uint4*>(y - off) + at, cut);
        if (off && (starts || ends))
#pragma unroll
          for (int t = at; t < kPer; t += kLanes) {
            if (starts && t < head) reinterpret_cast<E*>(y)[t] = reinterpret_cast<const E*>(from)[t];
            if (ends && t < tail)
              reinterpret_cast<E*>(y)[kN - tail + t] = reinterpret_cast<const E*>(from)[kN - tail + t];
          }
      }
    }
  } else {  // the ends of y, element by element
    for (int r = 0; r < rows; ++r, y += step, from += kRowsAtOnce * kTurnPitch) {
      const int tail = kWide || starts ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(y) & 15) / kSize);
      for (int e = at - tail; e < cols; e += kLanes)
        reinterpret_cast<E*>(y)[e] = reinterpret_cast<const E*>(from)[e];
    }
  }
  __syncwarp();
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

// The tiles of a block: every `step`-th from `first`, in an order that goes down
// kDown tiles of y before it goes along its rows: the blocks that run side by
// side then share their lanes' matrix with few and their columns' with few,
// and no line of L2 is asked for by all of them at once.  Bands of 1, 4, 8, 16 and
// 64: 2048 x 131072 x 64 115, 101, 93, 93, 93 us; 8192 x 16384 x 1024 73, 71, 72,
// 74, 78; 8192^3 155 to 158 with all.
constexpr uint32_t kDown = 8;
struct Tiles {
  uint32_t row, col, at, step, all;
  __device__ __forceinline__ Tiles(const Problem& p, uint32_t first, uint32_t by)
      : at(first), step(by), all(p.down * p.along) {
    place(p);
  }
  __device__ __forceinline__ void place(const Problem& p) {
    const uint32_t band = at / (kDown * p.along), rest = at % (kDown * p.along);
    const uint32_t high = min(kDown, p.down - min(p.down, band * kDown));
    if (high == 0) return;  // past the last tile
    col = rest / high;
    row = band * kDown + rest % high;
  }
  __device__ __forceinline__ bool left() const { return at < all; }
  __device__ __forceinline__ void next(const Problem& p) {
    at += step;
    place(p);
  }
};

// kAInLanes: the rows of A in the lanes, else the rows of B.  The tile of 192
// columns leaves room in TMEM for two accumulators and two sets of scales, and
// in shared memory for six (a pair) or four stages, three with 3 groups.
template <int kCols, int kBlocks, bool kAInLanes, int kGroups>
__global__ void __launch_bounds__(Shape<kCols, kBlocks, kGroups>::kThreads, 1)
    matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Problem p) {
  using S = Shape<kCols, kBlocks, kGroups>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ uint64_t full[S::kStages], empty[S::kStages], ready[2], drained[2];
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The blocks of a cluster: a pair (kBlocks 2), or the `splits` that share a
  // tile's k (kBlocks 1).
  const uint32_t splits = kBlocks == 2 || kAInLanes ? 1 : p.splits;
  const uint32_t rank = blockIdx.x % (splits * kBlocks);
  const uint32_t half_of = kBlocks == 2 ? rank : 0, part = splits > 1 ? rank : 0;

  if (warp == 0 && lane == 0) {
    const CUtensorMap* map[4] = {&maps.lanes, &maps.cols, &maps.lanes_scales, &maps.cols_scales};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("prefetch.tensormap [%0];" ::"l"(map[i]) : "memory");
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ready[b], 1);
      mbar_init(&drained[b], S::kStoreWarps * kBlocks);
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
  const uint32_t all = static_cast<uint32_t>((p.k + kStep - 1) / kStep);
  const uint32_t k0 = static_cast<uint64_t>(all) * part / splits;
  const uint32_t k1 = static_cast<uint64_t>(all) * (part + 1) / splits;

  if (warp == 0 && elect()) {
    uint32_t s = 0, round = 0;  // the next stage, and how often the stages have been used up
    bool ok = true;
    const uint32_t bars = kBlocks == 2 ? cluster_address(&full[0], 0) : smem_u32(&full[0]);
    for (; t.left() && ok; t.next(p)) {
      const int lane0 =
          static_cast<int>((static_cast<uint64_t>(kAInLanes ? t.row : t.col) * kBlocks + half_of) * kRows);
      const int col0 = static_cast<int>(static_cast<uint64_t>(kAInLanes ? t.col : t.row) * kCols);
      for (uint32_t k = k0; k < k1; ++k) {
        if (round > 0 && !wait(&empty[s], (round + 1) & 1)) {
          ok = false;
          break;
        }
        uint8_t* stage = smem + s * S::kStageBytes;
        uint8_t* scales = stage + S::kLaneBytes + S::kColBytes;
        const int x = static_cast<int>(k * kStepBytes), xs = static_cast<int>(k * 256);
        const uint32_t bar = bars + 8 * s;
        if (half_of == 0) mbar_arrive_expect_tx(&full[s], kBlocks * S::kStageBytes);
        tma_load<kBlocks>(stage, &maps.lanes, x, lane0, bar);
        tma_load<kBlocks>(stage + S::kLaneBytes, &maps.cols, x, col0 + half_of * S::kOwnCols, bar);
        tma_load<kBlocks>(scales, &maps.lanes_scales, xs, lane0 / 128, bar);
        tma_load<kBlocks>(scales + 1024, &maps.cols_scales, xs, col0 / 128, bar);
        if (++s == S::kStages) {
          s = 0;
          ++round;
        }
      }
    }
    // Before the block ends: the loads still in flight where a wait ran out,
    // and in a pair the products' arrivals on this block's barriers.
    if (!ok || kBlocks == 2)
      for (uint32_t i = 0; i < S::kStages; ++i) {
        const uint32_t uses = round + (i < s);
        if (uses && !wait(ok ? &empty[i] : &full[i], (uses + 1) & 1)) break;
      }
  } else if (warp == 1 && half_of == 0 && elect()) {
    // This thread sets the pace: a step is 4 products of 92 cycles each (192
    // columns), so everything that does not change from step to step is outside.
    uint32_t s = 0, parity = 0, set = 0, n_tile = 0;
    bool ok = true;
    const uint32_t units = desc_units(smem_u32(smem));
    const uint32_t rest = static_cast<uint32_t>(p.k % kStep);
    const int last = rest == 0 ? 4 : static_cast<int>((rest + 63) / 64);  // products of the last step
    for (; t.left() && ok; t.next(p), ++n_tile) {
      const uint32_t b = n_tile & 1;
      const uint32_t d = tmem + b * 256;
      // the scales of a tile that starts in the middle of a group of 128 rows
      // (192 columns: at 0 or 64, so that the shift is even, as it has to be)
      const uint32_t shift = kCols > 128 ? (kAInLanes ? t.col : t.row) % 2 * 2 : 0;
      if (n_tile >= 2 && !wait(&drained[b], (n_tile / 2 + 1) & 1)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (uint32_t k = k0; k < k1; ++k) {
        if (!wait(&full[s], parity)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t lanes = units + s * (S::kStageBytes / 16), cols = lanes + S::kLaneBytes / 16;
        const uint32_t sc = cols + S::kColBytes / 16;
        // two sets of scale columns, used by turns: a step's copies do not
        // wait for the products of the step before
        const uint32_t s_lanes = tmem + S::kScaleCol + set, s_cols = s_lanes + 8;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          copy_scales<kBlocks>(s_lanes + 4 * g, sc + 32 * g);
#pragma unroll
          for (int r = 0; r < S::kScaleRows; ++r)
            copy_scales<kBlocks>(s_cols + 4 * (S::kScaleRows * g + r), sc + 64 + 64 * r + 32 * g);
        }
        const int products = k + 1 == all ? last : 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q > 0 && q >= products) break;
          product<kBlocks>(d, lanes + 2 * q, cols + 2 * q, product_desc(kBlocks, kCols, 2 * (q & 1)),
                           s_lanes + 4 * (q / 2), s_cols + shift + 4 * S::kScaleRows * (q / 2),
                           q > 0 ? 1 : k - k0);
        }
        commit<kBlocks>(&empty[s]);
        set ^= 256;
        if (++s == S::kStages) {
          s = 0;
          parity ^= 1;
        }
      }
      if (ok) commit<kBlocks>(&ready[b]);
    }
    if (!ok) {  // products in flight end before TMEM is given back
      commit<kBlocks>(&ready[0]);
      commit<kBlocks>(&ready[1]);
      // and loads before the block ends: the loading thread may have issued its
      // last one and be gone (stages without a load run out once more)
      for (int i = 0; i < S::kStages && wait(&full[s], parity); ++i)
        if (++s == S::kStages) {
          s = 0;
          parity ^= 1;
        }
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3, group = (warp - 2) >> 2;  // the TMEM lanes this warp can read
    // This group's columns of a tile: neighbours, or with A in the lanes 64
    // (a 128-byte line of a 16-bit y) and, of two groups, 32 more.
    constexpr bool kMore = kAInLanes && kGroups == 2;
    const int from = kAInLanes ? group * 64 : group * S::kGroupCols, more = 128 + group * 32;
    uint8_t* room = smem + S::kTurnAt + (warp - 2) * kTurnWarp;
    uint32_t n_tile = 0;
    for (Tiles u = t; u.left(); u.next(p), ++n_tile) {
      const uint32_t b = n_tile & 1;
      if (!wait_warp(&ready[b], (n_tile / 2) & 1)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint64_t l = (static_cast<uint64_t>(kAInLanes ? u.row : u.col) * kBlocks + half_of) * kRows + quarter * 32;
      const uint64_t c = static_cast<uint64_t>(kAInLanes ? u.col : u.row) * kCols;
      const bool any = l < p.lanes && c + from < p.cols;
      const uint32_t d = tmem + b * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
      // the accumulators are given back as soon as they are read: the stores
      // run beside the products of the tile after the next
      float v[S::kGroupCols], before[16];
      if (any) {
        if constexpr (kAInLanes) {
          read_columns<0, 64>(d + from, v);
          if constexpr (kMore) read_columns<64, 32>(d + more, v);
          if (!p.wide) {
            read_eight<0>(d + (from ? from - 8 : 0), before);
            if constexpr (kMore) read_eight<8>(d + more - 8, before);
          }
          columns_read(before);
        } else {
          read_columns<0, S::kGroupCols>(d + from, v);
        }
        columns_read(v);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (kBlocks == 2) mbar_arrive_at(cluster_address(&drained[b], 0));
        else mbar_arrive(&drained[b]);
      }
      if (!any) continue;
      if constexpr (kAInLanes) {
        auto store = [&](auto type, auto wide) {
          constexpr int kType = decltype(type)::value;
          constexpr bool kWide = decltype(wide)::value;
          const bool first = group == 0, ends = !kMore && group == kGroups - 1;  // of the tile
          if constexpr (kType == HKV_F32) {
            turn_and_store<kType, kWide, 0, 32, 0>(room, p, l, c + from, v, before, first, false);
            if (c + from + 32 < p.cols)
              turn_and_store<kType, kWide, 32, 32, 24>(room, p, l, c + from + 32, v, v, false, ends);
          } else {
            turn_and_store<kType, kWide, 0, 64, 0>(room, p, l, c + from, v, before, first, ends);
          }
          if constexpr (kMore)
            if (c + more < p.cols)
              turn_and_store<kType, kWide, 64, 32, 8>(room, p, l, c + more, v, before, false, !first);
        };
        auto with = [&](auto wide) {
          if (p.type == HKV_F32) store(std::integral_constant<int, HKV_F32>{}, wide);
          else if (p.type == HKV_BF16) store(std::integral_constant<int, HKV_BF16>{}, wide);
          else store(std::integral_constant<int, HKV_F16>{}, wide);
        };
        if (p.wide) with(std::true_type{});
        else with(std::false_type{});
      } else if (splits > 1) {  // this block's part of the sum, for the cluster to add up
        float* mine = reinterpret_cast<float*>(smem) + from * kRows + quarter * 32 + lane;
#pragma unroll
        for (int q = 0; q < S::kGroupCols; ++q) mine[q * kRows] = v[q];
      } else {
        store_columns(p, c + from, l + lane, v);
      }
    }
  }
  __syncwarp();
  if (splits > 1) {
    cluster_sync();
    if (warp >= 2) {
      // a warp takes a column, a thread four neighbouring lanes of it; all
      // blocks' parts are on their way together and added in their order
      const uint64_t l = static_cast<uint64_t>(t.col) * kRows + lane * 4;
      const uint64_t c0 = static_cast<uint64_t>(t.row) * kCols;
      const int cols = p.cols - c0 < kCols ? static_cast<int>(p.cols - c0) : kCols;
#pragma unroll 2
      for (int c = part + splits * (warp - 2); c < cols; c += S::kStoreWarps * splits) {
        const uint32_t at = smem_u32(smem) + (c * kRows + lane * 4) * 4;
        float4 v[kMaxSplits];
#pragma unroll
        for (uint32_t r = 0; r < kMaxSplits; ++r)
          if (r < splits) v[r] = remote_f32x4(at, r);
        float4 sum = v[0];
#pragma unroll
        for (uint32_t r = 1; r < kMaxSplits; ++r)
          if (r < splits) {
            sum.x += v[r].x;
            sum.y += v[r].y;
            sum.z += v[r].z;
            sum.w += v[r].w;
          }
        store_four(p, c0 + c, l, sum);
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
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < p.cols * p.lanes; i += step)
    store_one(p, i / p.lanes, i % p.lanes, 0.f);
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

struct Operand {
  const uint8_t *codes, *scales;
  uint64_t rows;
};

// A matrix's codes as boxes of 128 bytes by `box` rows, swizzled, and its
// scales as boxes of two 512-byte groups by `groups`; what lies past the
// matrix reads as zeros.
bool make_maps(CUtensorMap* codes_map, CUtensorMap* scales_map, const Operand& o, uint64_t k,
               int box, int groups) {
  EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint32_t steps[2] = {1, 1};
  const uint64_t bytes = (k + kMxBlock - 1) / kMxBlock * 16;
  const cuuint64_t dims[2] = {bytes, o.rows}, strides[1] = {bytes};
  const cuuint32_t boxes[2] = {kStepBytes, static_cast<cuuint32_t>(box)};
  const uint64_t words = (k + 127) / 128 * 128;  // of 4 bytes
  const cuuint64_t sdims[2] = {words, (o.rows + 127) / 128}, sstrides[1] = {words * 4};
  const cuuint32_t sboxes[2] = {256, static_cast<cuuint32_t>(groups)};
  return f(codes_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(o.codes), dims, strides,
           boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         f(scales_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(o.scales), sdims,
           sstrides, sboxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCols, int kBlocks, bool kAInLanes, int kGroups = (kCols > 16 ? 2 : 1)>
cudaError_t run(Problem p, const Operand& a, const Operand& b, int splits, cudaStream_t st) {
  using S = Shape<kCols, kBlocks, kGroups>;
  const Operand &lanes = kAInLanes ? a : b, &cols = kAInLanes ? b : a;
  p.lanes = lanes.rows;
  p.cols = cols.rows;
  const uint64_t along_lanes = (p.lanes + kRows * kBlocks - 1) / (kRows * kBlocks);
  const uint64_t along_cols = (p.cols + kCols - 1) / kCols;
  const uint64_t tiles = along_lanes * along_cols;
  if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;  // no y in memory has as many
  p.along = static_cast<uint32_t>(kAInLanes ? along_cols : along_lanes);
  p.down = static_cast<uint32_t>(kAInLanes ? along_lanes : along_cols);
  p.splits = splits;
  Maps maps{};
  if (!make_maps(&maps.lanes, &maps.lanes_scales, lanes, p.k, kRows, 1) ||
      !make_maps(&maps.cols, &maps.cols_scales, cols, p.k, S::kOwnCols, S::kScaleRows))
    return cudaErrorUnknown;
  auto* kernel = matmul_kernel<kCols, kBlocks, kAInLanes, kGroups>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const uint32_t cluster = splits * kBlocks;
  const uint64_t room = sm_count() / kBlocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((splits > 1 || tiles < room ? tiles : room) * cluster));
  cfg.blockDim = dim3(S::kThreads);
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

cudaError_t matmul(Problem p, const Operand& a, const Operand& b, cudaStream_t st) {
  p.lanes = b.rows;
  p.cols = a.rows;
  if (p.k == 0) return launch_chained(zero_kernel, sm_count() * 4, 256, 0, st, p);
  const uint64_t sms = sm_count(), m = a.rows, n = b.rows, steps = (p.k + kStep - 1) / kStep;
  const int cols = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : m <= 128 ? 128 : 192;
  const uint64_t tiles = (n + kRows - 1) / kRows * ((m + cols - 1) / cols);
  // few tiles: a cluster shares a tile's k while SMs are idle and each block
  // keeps two steps at least.  With and without: 1 x 4096 x 4096 4.5 and 6.2 us,
  // 300 x 300 x 5000 8.2 and 13.7, 16 x 4096 x 16384 9.9 and 16.1, 64 x 2048 x 2048
  // 4.7 and 4.6.  One step a block and two rounds of SMs instead: 1 x 4096 x 4096
  // 10.7, 64 x 2048 x 2048 9.3; four steps a block: 300 x 300 x 5000 8.7, 64 x 2048
  // x 2048 5.4.
  int splits = 1;
  while (splits < kMaxSplits && tiles * splits * 2 <= sms && steps >= 4ull * splits) splits *= 2;
  if (cols == 16) return run<16, 1, false>(p, a, b, splits, st);
  if (cols == 32) return run<32, 1, false>(p, a, b, splits, st);
  if (cols == 64) return run<64, 1, false>(p, a, b, splits, st);
  if (cols == 128) return run<128, 1, false>(p, a, b, splits, st);
  if (splits > 1) return run<192, 1, false>(p, a, b, splits, st);
  // A pair loads 31 KB per block and step where a single block loads 43, and
  // an SM takes in 54 bytes a cycle; but a tile's way from the products to the
  // stores and back crosses the cluster.  Measured at 8192 x 16384, single and
  // pair: k 512 52 and 75 us, 1024 72 and 86, 1280 85 and 91, 2048 119 and 101.
  // Where pairs leave SMs without a tile, single blocks have twice as many.
  const bool pair = steps > 5 && (m + 191) / 192 * ((n + 255) / 256) * 2 > sms;
  if (pair) return run<192, 2, true>(p, a, b, 1, st);
  // Short k is bound by the stores, the more so where rows of y have to be cut:
  // twelve warps for them, at the price of a stage (8192 x 16384: k 512 49 and
  // 52 us, 768 66 and 60; 8192 x 16383: k 1024 92 and 103, 1280 106 and 107).
  return steps <= (p.wide ? 2 : 5) ? run<192, 1, true, 3>(p, a, b, 1, st)
                                   : run<192, 1, true>(p, a, b, 1, st);
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
  p.k = k;
  p.y = y;
  p.stride = y_stride;
  p.type = y_type;
  p.wide = aligned(y, 16) && y_stride * type_size(y_type) % 16 == 0;
  return op_status(matmul(p, {a_codes, a_scales, m}, {b_codes, b_scales, n},
                          static_cast<cudaStream_t>(stream)));
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
