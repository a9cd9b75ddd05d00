// adapter_tensor.cuh -- the first product of long requests with 16-bit matrices, on
// the tensor cores of tcgen05 with loads by TMA (the rest is in adapter.cuh).
//
// A block has 64 rows of one request and a part of their columns: one thread brings
// stages of 64 columns of x and of the adapter's first factor, one multiplies them
// into kRank columns of TMEM, and two warps read the sums out, which the blocks of a
// cluster join as in adapter.cuh.  The product is 128 rows high, the lowest that
// gives a row to a lane; what the 64 lanes below the tile's rows are multiplied with
// is whatever lies behind x in shared memory, and they are not read.
//
// The loads are the bound (x from memory, the factor from L2), and this way they
// cost no instructions of the warps: with asynchronous copies and mma.sync 8224 rows
// of 4096 by rank 64 took 35 us.
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

inline cudaError_t wait_timeouts(uint64_t* count) {
  unsigned long long v = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v));
  *count = v;
  return e;
}

}  // namespace tensor
}  // namespace hkv
