// operators.cuh -- element types, reductions and argument checks shared by
// the operators on looked-up rows (mx_quantize.cu, mx_matmul.cu,
// preference.cu, clip.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "hkv.h"
#include "launch.h"

namespace hkv {

inline size_t type_size(int type) { return type == HKV_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == HKV_F32 || type == HKV_BF16 || type == HKV_F16; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline hkv_status op_status(cudaError_t e) {
  if (e == cudaSuccess) return HKV_OK;
  return e == cudaErrorMemoryAllocation ? HKV_ERR_OOM : HKV_ERR_CUDA;
}

// Call f with a null pointer of the element type `type` stands for.
template <class F>
auto with_type(int type, F&& f) {
  if (type == HKV_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  if (type == HKV_F16) return f(static_cast<__half*>(nullptr));
  return f(static_cast<float*>(nullptr));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// How eight neighbouring elements are moved: in one access of 16 bytes (32 of
// float32), in two of 16 (float32 alone), or, where rows start anywhere, in
// the 16-byte pieces around them that neighbouring threads share.
enum Move : int { kShifted = 0, kHalves = 1, kWhole = 2 };

// The widest move that an address and a row stride in bytes allow.
template <class T>
__host__ __device__ inline int widest(const void* p, uint64_t stride_bytes) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p) | stride_bytes;
  if (a % (8 * sizeof(T)) == 0) return kWhole;
  return sizeof(T) == 4 && a % 16 == 0 ? kHalves : kShifted;
}

// x[i] = the 32 bits that start `bytes` (even, below 16) into x[i]; the last
// four words are only taken from.
template <int N>
__device__ __forceinline__ void shift_bytes(uint32_t (&x)[N], uint32_t bytes) {
#pragma unroll
  for (int i = 0; i < N - 1; ++i) x[i] = bytes & 4 ? x[i + 1] : x[i];
#pragma unroll
  for (int i = 0; i < N - 2; ++i) x[i] = bytes & 8 ? x[i + 2] : x[i];
#pragma unroll
  for (int i = 0; i < N - 4; ++i) x[i] = __byte_perm(x[i], x[i + 1], bytes & 2 ? 0x5432 : 0x3210);
}

// Eight neighbouring elements of a row as they lie in memory.  `lo` and `hi`
// bound the row: elements lo .. hi - 1 from the thread's first one belong to
// it (hi may be above 8, or not above 0); the others read as zeros.  Sixteen neighbouring threads, a half-warp, `at` of it, hold 128
// neighbouring elements; all threads of a warp take part.  `move` is the same
// for all rows.
template <class T>
struct Eight {
  static constexpr int kVecs = sizeof(T) / 2;
  uint4 w[kVecs];

  // Whole moves without `move`, of memory that this kernel may also write.
  __device__ __forceinline__ void load_written(const T* p) {
    if constexpr (kVecs == 1)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w)
                   : "l"(p)
                   : "memory");
    else
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w),
                     "=r"(w[kVecs - 1].x), "=r"(w[kVecs - 1].y), "=r"(w[kVecs - 1].z),
                     "=r"(w[kVecs - 1].w)
                   : "l"(p)
                   : "memory");
  }
  // All eight, by one access or two.
  __device__ __forceinline__ void load_aligned(const T* p, int move) {
    if (kVecs == 2 && move == kWhole) {
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w),
                     "=r"(w[kVecs - 1].x), "=r"(w[kVecs - 1].y), "=r"(w[kVecs - 1].z),
                     "=r"(w[kVecs - 1].w)
                   : "l"(p));
    } else if (kVecs == 2) {
      // the halves of a sector come by two instructions: through L1
#pragma unroll
      for (int i = 0; i < kVecs; ++i) w[i] = ld_nc_v4(p + i * 4);
    } else {
      w[0] = ld_stream_v4(p);
    }
  }
  __device__ __forceinline__ void store_aligned(T* p, int move) const {
    if (kVecs == 2 && move == kWhole) {
      asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0].x),
                   "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[kVecs - 1].x),
                   "r"(w[kVecs - 1].y), "r"(w[kVecs - 1].z), "r"(w[kVecs - 1].w)
                   : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) st_stream_v4(p + i * (16 / sizeof(T)), w[i]);
    }
  }

  // The 16 bytes at p + from, a boundary.
  static __device__ __forceinline__ uint4 piece(const T* p, int from, int lo, int hi) {
    constexpr int kPer = 16 / sizeof(T);
    if (from >= lo && from + kPer <= hi) return ld_nc_v4(p + from);
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      e[i] = from + i >= lo && from + i < hi ? p[from + i] : from_f32<T>(0.f);
    return v;
  }

  __device__ __forceinline__ void load(const T* p, int lo, int hi, int move, int at) {
    constexpr int kPer = 16 / sizeof(T);
    if (move != kShifted) {
      if (hi >= 8) load_aligned(p, move);
      else
#pragma unroll
        for (int i = 0; i < kVecs; ++i) w[i] = piece(p, i * kPer, 0, hi);
      return;
    }
    // the pieces from the boundary below p on, and the next thread's first one
    const uint32_t off = reinterpret_cast<uintptr_t>(p) & 15;
    const int back = static_cast<int>(off / sizeof(T));
    uint32_t x[4 * kVecs + 4];
    uint4* v = reinterpret_cast<uint4*>(x);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = piece(p, i * kPer - back, lo, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * kVecs + i] = __shfl_down_sync(0xFFFFFFFFu, x[i], 1, 16);
    if (at == 15 && off) v[kVecs] = piece(p, kVecs * kPer - back, lo, hi);
    shift_bytes(x, off);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = v[i];
  }

  __device__ __forceinline__ void to(float (&v)[8]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void from(const float (&v)[8]) {
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
  }
};

// Thread-block clusters: a float in the shared memory of another block (at the
// same place there as `addr` here), and the barrier of all the blocks' threads.
__device__ __forceinline__ float remote_f32(uint32_t addr, uint32_t rank) {
  uint32_t far;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(far) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t addr, uint32_t rank) {
  uint32_t far;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(far) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Sums of N values over the block, the same bits in every thread (a fixed
// tree).  `red` holds N floats per warp; it is free again after the next
// __syncthreads().
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* red) {
  const int warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[(threadIdx.x >> 5) * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < warps; ++w) v[i] += red[w * N + i];
  }
}

}  // namespace hkv
