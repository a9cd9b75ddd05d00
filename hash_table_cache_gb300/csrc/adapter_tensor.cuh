// adapter_tensor.cuh -- the adapters' products of long requests with 16-bit matrices,
// on the tensor cores of tcgen05 with loads by TMA (the rest is in adapter.cuh).
//
// The first product: a block has 64 rows of one request and a part of their columns;
// one thread brings stages of 64 columns of x and of the adapter's first factor, one
// multiplies them into kRank columns of TMEM, and two warps read the sums out, which
// the blocks of a cluster join as in adapter.cuh.  The product is 128 rows high, the
// lowest that gives a row to a lane; what the 64 lanes below the tile's rows are
// multiplied with is whatever lies behind x in shared memory, and they are not read.
//
// The loads are the bound (x from memory, the factor from L2), and this way they cost
// no instructions of the warps.  Kernels alone, cold, 7935 rows of 4096 to 4096 by rank
// 64 bfloat16, here and with asynchronous copies and mma.sync: first product 19 us (3.4
// TB/s of x; 35), second 38 us (3.4 TB/s of base and y; 42), gradients 38 us (3.4 TB/s of x
// and dy; 73).  Half of a first product's time is its start and end: a block's search,
// its first loads, and the joining of the sums.
#pragma once

#include <cuda.h>

#include "adapter.cuh"

namespace hkv {
namespace tensor {

// Bounded wait for a phase of a barrier: false after kWaitNs, with this file's count
// of timeouts raised.
static __device__ unsigned long long g_wait_timeouts;
constexpr uint64_t kWaitNs = 4000000000ull;
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
static __device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity) {
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
// By a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}

__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

struct Maps {  // x: tokens x in; the first factor: adapters x rows x columns
  CUtensorMap x, first;
};

template <int kRank>
struct Shape {
  static constexpr int kTile = 64, kStep = 64, kThreads = 128;
  static constexpr int kX = kTile * 128, kFirst = kRank * 128, kStage = kX + kFirst;  // bytes, either order
  static constexpr int kStages = kRank == 64 ? 4 : 6;
  static constexpr int kPitch = kRank + 4;  // of the sums, which take the stages' place
  static constexpr int kColumns = kRank < 32 ? 32 : kRank;  // of TMEM
  // what the lowest lanes of the last stage's product read lies behind it
  static constexpr int kBytes = kStages * kStage + kX + 1024;
  static_assert(kTile * kPitch * 4 <= kStages * kStage, "room for the sums");
};

// Shared-memory descriptors, version 1; upper halves.  Rows of 128 bytes along k in the
// 128-byte swizzle, 1024 bytes from one group of 8 rows to the next.
constexpr uint32_t kAlongK = (1024 >> 4) | 1u << 14 | 2u << 29;
// The factor of the backward pass lies the other way: a row of kRank numbers for each k,
// in the swizzle of its length, groups of 8 of them.
template <int kRank>
__host__ __device__ constexpr uint32_t along_rank() {
  return (kRank * 16 >> 4) | 1u << 14 | (kRank == 64 ? 2u : kRank == 32 ? 4u : 6u) << 29;
}
// Instruction descriptor: float32 sums, both types bfloat16 or float16, 128 rows.
template <class T, int kRank, bool kBack>
__host__ __device__ constexpr uint32_t product_desc() {
  constexpr uint32_t kType = std::is_same_v<T, __nv_bfloat16> ? 1 : 0;
  return 1u << 4 | kType << 7 | kType << 10 | (kBack ? 1u : 0u) << 16 | (uint32_t)(kRank >> 3) << 17 | (128u >> 4) << 24;
}
template <int kRank, bool kBack>
__device__ __forceinline__ void product(uint32_t d, uint32_t x, uint32_t w, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(x), "r"(w), "r"(idesc), "r"(add), "n"(kAlongK), "n"(kBack ? along_rank<kRank>() : kAlongK)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

template <class T, int kRank, bool kBack>
__global__ void __launch_bounds__(Shape<kRank>::kThreads)
    first_tensor_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Chain<T> a) {
  using S = Shape<kRank>;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ uint64_t full[S::kStages], empty[S::kStages], done;
  __shared__ uint32_t tmem_base;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.x) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.first) : "memory");
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "n"(S::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  pdl_wait();
  pdl_trigger();  // what the second product reads before it waits is complete from here on

  const uint32_t part = blockIdx.x % a.parts;
  Tile t;
  const bool works = Tile::find<S::kTile>(a.q, blockIdx.x / a.parts, t) && t.adapter >= 0;  // the whole cluster's
  const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
  const uint32_t steps = works ? static_cast<uint32_t>((in1 - in0 + S::kStep - 1) / S::kStep) : 0;
  __syncwarp();

  if (warp == 0 && elect()) {
    bool ok = true;
    uint32_t step = 0;
    for (; step < steps; ++step) {
      const uint32_t s = step % S::kStages, round = step / S::kStages;
      if (round > 0 && !wait(&empty[s], (round + 1) & 1)) {
        ok = false;
        break;
      }
      uint8_t* const stage = smem + s * S::kStage;
      const int k = static_cast<int>(in0 + static_cast<uint64_t>(step) * S::kStep);
      mbar_arrive_expect_tx(&full[s], S::kStage);
      load_box(stage, &maps.x, k, static_cast<int>(t.row0), &full[s]);
      if constexpr (kBack) load_box(stage + S::kX, &maps.first, 0, k, static_cast<int>(t.adapter), &full[s]);
      else load_box(stage + S::kX, &maps.first, k, 0, static_cast<int>(t.adapter), &full[s]);
    }
    // before the block ends, the loads still in flight where a wait ran out
    if (!ok)
      for (uint32_t i = step - S::kStages; i < step; ++i)
        if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
  } else if (warp == 1 && elect()) {
    bool ok = true;
    const uint32_t units = (smem_u32(smem) & 0x3FFFF) >> 4;
    constexpr uint32_t kIdesc = product_desc<T, kRank, kBack>();
    uint32_t step = 0;
    for (; step < steps; ++step) {
      const uint32_t s = step % S::kStages;
      if (!wait(&full[s], step / S::kStages & 1)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t x = units + s * (S::kStage / 16), w = x + S::kX / 16 + (kBack ? (uint32_t)kRank << 16 : 0u);
#pragma unroll
      for (int i = 0; i < S::kStep / 16; ++i)  // 16 numbers of k: 32 bytes of a row, or 16 rows
        product<kRank, kBack>(tmem, x + 2 * i, w + i * (kBack ? kRank * 2 : 2), kIdesc, step > 0 || i > 0);
      commit(&empty[s]);
    }
    if (steps && ok) commit(&done);
    // the loading thread may have issued its last loads and be gone: where a wait ran
    // out, the loads that follow are waited for
    if (!ok)
      for (uint32_t i = step + 1; i < steps && i < step + S::kStages; ++i)
        if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
  }
  __syncwarp();
  // (steps is the same for all of the block)
  const bool summed = steps && wait_warp(&done, 0);
  float* const own = reinterpret_cast<float*>(smem);  // [tile][kPitch]
  if (summed) {
    // the stages are read: the sums take their place
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp < S::kTile / 32) {
      const uint32_t from = tmem + (warp * 32 << 16);
      float* const to = own + (warp * 32 + lane) * S::kPitch;
#pragma unroll
      for (int c = 0; c < kRank; c += 16) {
        uint32_t r[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(from + c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));  // used after the wait only
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<uint4*>(to + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns));
  if (!works) return;  // the whole cluster

  const float scale = a.q.scales ? a.q.scales[t.adapter] : 1.f;
  constexpr int kQuads = S::kTile * kRank / 4;
  const uint32_t used = static_cast<uint32_t>((a.in + a.part_in - 1) / a.part_in);  // parts with columns
  if (a.parts > 1) cluster_meet();
  const int each = kQuads / a.parts;
  for (int e = tid; e < each; e += S::kThreads) {
    const int i = part * each + e, row = i * 4 / kRank, col = i * 4 % kRank;
    if (row >= t.rows) break;
    const uint32_t at = smem_u32(own + row * S::kPitch + col);
    float4 v;
    if (a.parts == 1) {
      v = *reinterpret_cast<const float4*>(own + row * S::kPitch + col);
    } else {
      v = remote_f32x4(at, 0);
      for (uint32_t p = 1; p < used; ++p) v = v + remote_f32x4(at, p);
    }
    put_hidden<T, kRank>(a.hidden, t.row0 + row, col, v, scale);
  }
  if (a.parts > 1) cluster_meet();  // the others stay until their sums are read
}

// ---------------------------------------------------------------------------
// The second product of bfloat16 matrices: 128 columns of y in the lanes, the tile's 64
// rows in the columns of TMEM, so that a warp's lanes are neighbouring columns of a row
// and base and y are read and written row by row as they lie.  The two planes of c h (or
// dh) are multiplied by the same columns of the second factor and added up in TMEM.
// One thread loads (the factor's columns, base, and the planes once the first product is
// done), one multiplies, eight warps add onto base.  What bounds it is those warps'
// instructions (14 for an element) and how much base is on its way, which shared memory
// holds: 1447 rows to 131072 columns by rank 8 131 us, 73% of the memory's cycles; 7883
// rows to 8192 by rank 32 50 us.  Tried: four warps 68 us with the first product against
// 67; a third stage of rank 32 instead of a third block 77; sums put together in shared
// memory and stored 16 bytes at a time 75.
// ---------------------------------------------------------------------------
struct SecondMaps {  // the second factor; c h or dh: tokens x planes of kRank; base
  CUtensorMap second, hidden, base;
};

template <int kRank>
struct SecondShape {
  static constexpr int kTile = 64, kCols = 128;
  static constexpr int kGroups = 2, kAdding = 4 * kGroups, kThreads = 64 + 32 * kAdding;  // warps that add, by rows
  static constexpr int kFactor = kCols * kRank * 2, kBase = kTile * kCols * 2, kStage = kFactor + kBase;
  static constexpr int kPlane = kTile * kRank * 2, kPlanes = 2 * kPlane;
  static constexpr int kStages = kRank == 16 ? 3 : 2;
  static constexpr int kBytes = kPlanes + kStages * kStage + 1024;
  static_assert(kPlane % 1024 == 0 && kFactor % 1024 == 0, "swizzle");
};
// Upper halves: rows of kRank numbers along k, in the swizzle of their length, groups of
// 8 of them; and columns of y along the lanes in pieces of 64, a row of them for each k.
template <int kRank>
__host__ __device__ constexpr uint32_t rank_rows() { return along_rank<kRank>(); }

template <int kRank, bool kBack>
__global__ void __launch_bounds__(SecondShape<kRank>::kThreads, 3)
    second_tensor_kernel(const __grid_constant__ SecondMaps maps, const __grid_constant__ Chain<__nv_bfloat16> a) {
  using S = SecondShape<kRank>;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  uint8_t* const stages = smem + S::kPlanes;
  __shared__ uint64_t full[S::kStages], empty[S::kStages], planes, ready[2], drained[2];
  __shared__ uint32_t tmem_base;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.second) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.hidden) : "memory");
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1 + S::kAdding);  // multiplied, and base read
    }
    mbar_init(&planes, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ready[b], 1);
      mbar_init(&drained[b], S::kAdding);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_u32(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;

  // before the first product's end: its kernel lets this one start when all that came
  // before is complete, and it writes `hidden` alone
  const uint64_t col0 = static_cast<uint64_t>(blockIdx.x % a.groups) * a.group_out;
  const uint64_t col1 = min(col0 + a.group_out, a.out);
  Tile t;
  const bool any = Tile::find<S::kTile>(a.q, blockIdx.x / a.groups, t) && col0 < col1;
  const bool adapts = any && t.adapter >= 0;
  const uint32_t steps = any && (adapts || a.y != a.base) ? static_cast<uint32_t>((col1 - col0 + S::kCols - 1) / S::kCols) : 0;
  __syncwarp();
  const bool has_base = a.base != nullptr;

  if (warp == 0 && elect()) {
    bool ok = true;
    uint32_t step = 0;
    for (; step < steps; ++step) {
      const uint32_t s = step % S::kStages, round = step / S::kStages;
      if (round > 0 && !wait(&empty[s], (round + 1) & 1)) {
        ok = false;
        break;
      }
      uint8_t* const stage = stages + s * S::kStage;
      const int c = static_cast<int>(col0 + static_cast<uint64_t>(step) * S::kCols);
      const uint32_t bytes = (adapts ? S::kFactor : 0) + (has_base ? S::kBase : 0);
      mbar_arrive_expect_tx(&full[s], bytes);
      if (adapts) {
        if constexpr (kBack) {
          load_box(stage, &maps.second, c, 0, static_cast<int>(t.adapter), &full[s]);
          load_box(stage + S::kFactor / 2, &maps.second, c + 64, 0, static_cast<int>(t.adapter), &full[s]);
        } else {
          load_box(stage, &maps.second, 0, c, static_cast<int>(t.adapter), &full[s]);
        }
      }
      if (has_base) load_box(stage + S::kFactor, &maps.base, c, static_cast<int>(t.row0), &full[s]);
      if (step + 1 == S::kStages || (step + 1 == steps && steps < S::kStages)) {
        pdl_wait();  // the first product is done (limited waits begin here, in every role)
        if (adapts) {
          mbar_arrive_expect_tx(&planes, S::kPlanes);
          load_box(smem, &maps.hidden, 0, static_cast<int>(t.row0), &planes);
          load_box(smem + S::kPlane, &maps.hidden, kRank, static_cast<int>(t.row0), &planes);
        }
      }
    }
    // before the block ends, the loads still in flight where a wait ran out
    if (!ok) {
      if (adapts) wait(&planes, 0);
      for (uint32_t i = step - S::kStages; i < step; ++i)
        if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
    }
  } else if (warp == 1 && adapts && steps && elect()) {
    pdl_wait();
    bool ok = wait(&planes, 0);
    const uint32_t units = (smem_u32(smem) & 0x3FFFF) >> 4, factors = (smem_u32(stages) & 0x3FFFF) >> 4;
    constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (kBack ? 1u : 0u) << 15 | (uint32_t)(S::kTile >> 3) << 17 | (128u >> 4) << 24;
    uint32_t step = 0;
    for (; ok && step < steps; ++step) {
      const uint32_t s = step % S::kStages, b = step & 1;
      if ((step >= 2 && !wait(&drained[b], (step / 2 + 1) & 1)) || !wait(&full[s], step / S::kStages & 1)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // (a factor's pieces of 64 columns are kRank rows of 128 bytes)
      const uint32_t w = factors + s * (S::kStage / 16) + (kBack ? (uint32_t)(kRank * 8) << 16 : 0u);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < kRank / 16; ++i)
          asm volatile(
              "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n"
              " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
              " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(tmem + b * 64),
              "r"(w + i * (kBack ? 128 : 2)), "r"(units + p * (S::kPlane / 16) + 2 * i), "r"(kIdesc), "r"((uint32_t)(p + i)),
              "n"(kBack ? kAlongK : rank_rows<kRank>()), "n"(rank_rows<kRank>())
              : "memory");
      commit(&empty[s]);
      commit(&ready[b]);
    }
    // where a wait ran out, the loads that follow are waited for
    if (!ok) {
      wait(&planes, 0);
      for (uint32_t i = step; i < steps && i < step + S::kStages; ++i)
        if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
    }
  } else if (warp >= 2) {
    const uint32_t quarter = warp % 4;  // of the lanes, the only one that a warp can read
    constexpr int kRows = S::kTile / S::kGroups;
    const int first = (warp - 2) / 4 * kRows;
    pdl_wait();
    pdl_trigger();
    __nv_bfloat16* const y = a.y + t.row0 * a.y_stride;
    for (uint32_t step = 0; step < steps; ++step) {
      const uint32_t s = step % S::kStages, b = step & 1;
      const __nv_bfloat16* const base = reinterpret_cast<const __nv_bfloat16*>(stages + s * S::kStage + S::kFactor) + quarter * 32 + lane;
      const uint64_t col = col0 + static_cast<uint64_t>(step) * S::kCols + quarter * 32 + lane;
      if (!wait_warp(&full[s], step / S::kStages & 1)) break;
      if (adapts && !wait_warp(&ready[b], step / 2 & 1)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const bool mine = col < col1;
      __nv_bfloat16* to = y + col;
#pragma unroll
      for (int r = 0; r < kRows; r += 16) {
        const int r0 = first + r;
        if (r0 >= t.rows) break;
        __syncwarp();
        float v[16] = {};
        if (adapts) {
          uint32_t* const u = reinterpret_cast<uint32_t*>(v);
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
              : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
                "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
              : "r"(tmem + b * 64 + (quarter * 32 << 16) + r0));
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(v[i]));  // used after the wait only
        }
        if (has_base)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __bfloat162float(base[(r0 + i) * S::kCols]);
        const int rows = mine ? t.rows - r0 : 0;
        __nv_bfloat16* out = to + r0 * a.y_stride;
        if (rows >= 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i, out += a.y_stride) *out = __float2bfloat16_rn(v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i, out += a.y_stride)
            if (i < rows) *out = __float2bfloat16_rn(v[i]);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[s])) : "memory");
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&drained[b])) : "memory");
        // (a stage of a tile without an adapter is not multiplied)
        if (!adapts && warp == 2) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[s])) : "memory");
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem));
}

// ---------------------------------------------------------------------------
// The adapters' gradients of bfloat16 matrices: 128 columns of x or dy in the lanes, the
// ranks in the columns of TMEM, rows of the batch along k.  Both lie with their rows
// apart, which the tensor core takes as it is.  Rows of a tile that are another
// request's are made zeros in shared memory, of both operands.  Each of the (k + n) / 128
// blocks of an adapter reads the planes anew, from L2.
// ---------------------------------------------------------------------------
struct GradMaps {  // x and dy; dh and c h
  CUtensorMap m[2], p[2];
};

template <int kRank>
struct GradShape {
  static constexpr int kRows = 64, kCols = 128, kThreads = 128;
  static constexpr int kPiece = kRows * 128, kM = 2 * kPiece, kPlane = kRows * kRank * 2, kStage = kM + 2 * kPlane;
  static constexpr int kStages = kRank == 64 ? 2 : 3;
  static constexpr int kPitch = kRank + 4, kSums = kCols * kPitch * 4;  // [cols][kPitch]
  static constexpr int kColumns = kRank < 32 ? 32 : kRank;
  static constexpr int kBytes = (kStages * kStage > 2 * kSums ? kStages * kStage : 2 * kSums) + 1024;
};

template <int kRank>
__global__ void __launch_bounds__(GradShape<kRank>::kThreads)
    grads_tensor_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ Grads<__nv_bfloat16> a) {
  using S = GradShape<kRank>;
  constexpr int kThreads = S::kThreads;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ uint64_t full[S::kStages], empty[S::kStages], done;
  __shared__ uint32_t tmem_base, multiplied;
  __shared__ uint64_t from[kThreads], to[kThreads];  // rows of the adapter's requests
  __shared__ uint32_t counts[kThreads / 32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    multiplied = 0;
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "n"(S::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  pdl_trigger();
  pdl_wait();

  const uint32_t part = blockIdx.x % a.parts;
  const uint64_t all = a.blocks[0] + a.blocks[1];
  const int64_t adapter = adapter_at(a.q, a.by_request, blockIdx.x / a.parts / all);
  uint64_t block = blockIdx.x / a.parts % all;
  const int sel = block >= a.blocks[0];
  if (sel) block -= a.blocks[0];
  const uint64_t col0 = block * S::kCols, cols = a.cols[sel];

  uint64_t tile = 0;         // of the adapter's, counted over its requests
  uint32_t step = 0;         // of this block's tiles
  bool ok = true;            // the loading thread's, and the multiplying warp's
  for (uint64_t s0 = 0; s0 < a.q.requests; s0 += kThreads) {
    // the requests of this adapter among the next ones, in their order
    const uint64_t s = s0 + tid;
    const bool mine = s < a.q.requests && adapter >= 0 && a.q.adapter(s + 1) == adapter;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, mine);
    if (lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    uint32_t at = __popc(votes & ((1u << lane) - 1)), found = 0;
    for (uint32_t w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += counts[w];
      found += counts[w];
    }
    if (mine) {
      from[at] = a.q.start(s + 1);
      to[at] = a.q.start(s + 2);
    }
    __syncthreads();
    uint32_t i = 0;
    uint64_t row = found ? from[0] : 0;
    auto next = [&](uint64_t& row0, int& rows) {  // this block's next tile; false: none left
      while (i < found) {
        if (row >= to[i]) {
          if (++i < found) row = from[i];
          continue;
        }
        row0 = row;
        rows = static_cast<int>(min(to[i] - row, static_cast<uint64_t>(S::kRows)));
        row += S::kRows;
        if (tile++ % a.parts == part) return true;
      }
      return false;
    };
    uint64_t row0;
    int rows;
    if (warp == 0) {
      while (ok && next(row0, rows)) {
        const uint32_t st = step % S::kStages, round = step / S::kStages;
        if (round > 0 && !wait_warp(&empty[st], (round + 1) & 1)) {
          ok = false;
          break;
        }
        if (elect()) {
          uint8_t* const b = smem + st * S::kStage;
          const int y = static_cast<int>(row0), c = static_cast<int>(col0);
          mbar_arrive_expect_tx(&full[st], S::kStage);
          load_box(b, &maps.m[sel], c, y, &full[st]);
          load_box(b + S::kPiece, &maps.m[sel], c + 64, y, &full[st]);
          load_box(b + S::kM, &maps.p[sel], 0, y, &full[st]);
          load_box(b + S::kM + S::kPlane, &maps.p[sel], kRank, y, &full[st]);
        }
        __syncwarp();
        ++step;
      }
    } else if (warp == 1) {
      while (ok && next(row0, rows)) {
        const uint32_t st = step % S::kStages;
        if (!wait_warp(&full[st], step / S::kStages & 1)) {
          ok = false;
          break;
        }
        uint8_t* const b = smem + st * S::kStage;
        if (rows < S::kRows) {  // (a row's bytes change places within the row)
          const uint4 zero = make_uint4(0, 0, 0, 0);
          for (int e = rows * 8 + lane; e < S::kRows * 8; e += 32) {
            reinterpret_cast<uint4*>(b)[e] = zero;
            reinterpret_cast<uint4*>(b + S::kPiece)[e] = zero;
          }
          for (int e = rows * (kRank / 8) + lane; e < S::kRows * (kRank / 8); e += 32) {
            reinterpret_cast<uint4*>(b + S::kM)[e] = zero;
            reinterpret_cast<uint4*>(b + S::kM + S::kPlane)[e] = zero;
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (elect()) {
          constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | 3u << 15 | (uint32_t)(kRank >> 3) << 17 | (128u >> 4) << 24;
          const uint32_t m = ((smem_u32(b) & 0x3FFFF) >> 4) + ((uint32_t)(S::kPiece >> 4) << 16);
          const uint32_t h = ((smem_u32(b + S::kM) & 0x3FFFF) >> 4) + ((uint32_t)kRank << 16);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < S::kRows / 16; ++k)
              asm volatile(
                  "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n"
                  " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
                  " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(tmem),
                  "r"(m + k * 128), "r"(h + p * (S::kPlane / 16) + k * 2 * kRank), "r"(kIdesc), "r"(step + p + k),
                  "n"(kAlongK), "n"(along_rank<kRank>())
                  : "memory");
          commit(&empty[st]);
        }
        __syncwarp();
        ++step;
      }
    }
    __syncthreads();  // the lists are read
  }
  // before the block ends: the loads in flight where a wait ran out (the loading thread's
  // last ones, which the multiplying warp has not seen), and the products
  if (warp == 0 && !ok)
    for (uint32_t i = step - S::kStages; i < step; ++i)
      if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
  __syncwarp();
  if (warp == 1) {
    if (lane == 0) multiplied = ok && step > 0;
    if (ok && step > 0 && elect()) commit(&done);
    if (!ok && elect())
      for (uint32_t i = step + 1; i < step + S::kStages; ++i)
        if (!wait(&full[i % S::kStages], i / S::kStages & 1)) break;
    __syncwarp();
  }
  __syncthreads();
  // the sums of a column to a thread
  float* const sums = reinterpret_cast<float*>(smem);
  const bool summed = multiplied && wait_warp(&done, 0);
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
  for (int c = 0; c < kRank; c += 16) {
    uint32_t r[16] = {};
    if (summed) {
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
            "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
          : "r"(tmem + (warp * 32 << 16) + c));
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));  // used after the wait only
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint4*>(sums + tid * S::kPitch + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns));

  // the parts' sums in a fixed order, and the result: a part's share are whole ranks
  const int each = kRank / a.parts, r0 = part * each;
  const float* total = sums;
  if (a.parts > 1) {
    cluster_meet();
    float* const joined = sums + S::kSums / 4;
    const int quads = each / 4;  // (at least one: the launch sees to it)
    for (int e = tid; e < S::kCols * quads; e += kThreads) {
      const int at = e / quads * S::kPitch + r0 + e % quads * 4;
      float4 v = remote_f32x4(smem_u32(sums + at), 0);
      for (uint32_t q = 1; q < a.parts; ++q) v = v + remote_f32x4(smem_u32(sums + at), q);
      *reinterpret_cast<float4*>(joined + at) = v;
    }
    __syncthreads();
    total = joined;
  }
  if (adapter >= 0)
    put_grads<__nv_bfloat16, kThreads>(a, sel, adapter, col0,
                                       static_cast<uint32_t>(min(cols - col0, static_cast<uint64_t>(S::kCols))), r0,
                                       min(each, static_cast<int>(a.rank) - r0),
                                       [&](uint32_t r, uint32_t c) { return total[c * S::kPitch + r0 + r]; });
  if (a.parts > 1) cluster_meet();  // the others stay until their parts are read
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
inline EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// The matrices as TMA takes them: false where it does not take them as they lie
// (boundaries of 16 bytes, strides below 2^40 bytes and not 0).
template <class T, int kRank, bool kBack>
bool make_maps(Maps* maps, const Chain<T>& a) {
  using S = Shape<kRank>;
  if (!a.x_whole || !a.first.whole) return false;
  const EncodeFn f = encode_fn();
  if (!f) return false;
  constexpr CUtensorMapDataType kType =
      std::is_same_v<T, __nv_bfloat16> ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  constexpr CUtensorMapSwizzle kSwizzle = !kBack || kRank == 64 ? CU_TENSOR_MAP_SWIZZLE_128B
                                          : kRank == 32         ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                : CU_TENSOR_MAP_SWIZZLE_32B;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t x_dims[2] = {a.in, a.q.tokens}, x_strides[1] = {a.x_stride * sizeof(T)};
  const cuuint32_t x_box[2] = {S::kStep, S::kTile};
  const cuuint64_t w_dims[3] = {kBack ? a.rank : a.in, kBack ? a.in : a.rank, a.q.adapters};
  const cuuint64_t w_strides[2] = {a.first.stride * sizeof(T), a.first.step * sizeof(T)};
  const cuuint32_t w_box[3] = {kBack ? kRank : S::kStep, kBack ? S::kStep : kRank, 1};
  return f(&maps->x, kType, 2, const_cast<T*>(a.x), x_dims, x_strides, x_box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         f(&maps->first, kType, 3, const_cast<T*>(a.first.data), w_dims, w_strides, w_box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, kSwizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kRank, bool kBack>
bool make_maps(SecondMaps* maps, const Chain<__nv_bfloat16>& a) {
  using S = SecondShape<kRank>;
  if (!a.second.whole || (a.base && !a.base_whole)) return false;
  const EncodeFn f = encode_fn();
  if (!f) return false;
  constexpr CUtensorMapDataType kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr CUtensorMapSwizzle kRow =
      kRank == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : kRank == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t w_dims[3] = {kBack ? a.out : a.rank, kBack ? a.rank : a.out, a.q.adapters};
  const cuuint64_t w_strides[2] = {a.second.stride * 2, a.second.step * 2};
  const cuuint32_t w_box[3] = {kBack ? 64 : kRank, kBack ? kRank : S::kCols, 1};
  const cuuint64_t h_dims[2] = {2 * kRank, a.q.tokens}, h_strides[1] = {4 * kRank};
  const cuuint32_t h_box[2] = {kRank, S::kTile};
  const cuuint64_t b_dims[2] = {a.out, a.q.tokens}, b_strides[1] = {a.base_stride * 2};
  const cuuint32_t b_box[2] = {S::kCols, S::kTile};
  if (a.base && f(&maps->base, kType, 2, const_cast<__nv_bfloat16*>(a.base), b_dims, b_strides, b_box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  return f(&maps->second, kType, 3, const_cast<__nv_bfloat16*>(a.second.data), w_dims, w_strides, w_box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, kBack ? CU_TENSOR_MAP_SWIZZLE_128B : kRow, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         f(&maps->hidden, kType, 2, a.hidden, h_dims, h_strides, h_box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, kRow,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kRank>
bool make_maps(GradMaps* maps, const Grads<__nv_bfloat16>& a) {
  using S = GradShape<kRank>;
  const EncodeFn f = encode_fn();
  if (!f) return false;
  constexpr CUtensorMapDataType kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr CUtensorMapSwizzle kRow =
      kRank == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : kRank == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  const cuuint32_t ones[2] = {1, 1}, m_box[2] = {64, S::kRows}, p_box[2] = {kRank, S::kRows};
  const cuuint64_t p_dims[2] = {2 * kRank, a.q.tokens}, p_strides[1] = {4 * kRank};
  for (int i = 0; i < 2; ++i) {
    if (!a.out[i]) continue;
    const cuuint64_t m_dims[2] = {a.cols[i], a.q.tokens}, m_strides[1] = {a.stride[i] * 2};
    if (!a.whole[i] ||
        f(&maps->m[i], kType, 2, const_cast<__nv_bfloat16*>(a.m[i]), m_dims, m_strides, m_box, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        f(&maps->p[i], kType, 2, const_cast<__nv_bfloat16*>(a.p[i]), p_dims, p_strides, p_box, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, kRow, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

inline cudaError_t wait_timeouts(uint64_t* count) {
  unsigned long long v = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v));
  *count = v;
  return e;
}

}  // namespace tensor
}  // namespace hkv
