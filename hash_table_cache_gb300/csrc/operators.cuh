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
// float32), in two of 16 (float32 alone), or one by one.
enum Move : int { kSingly = 0, kHalves = 1, kWhole = 2 };

// The widest move that an address and a row stride in bytes allow.
template <class T>
__host__ __device__ inline int widest(const void* p, uint64_t stride_bytes) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p) | stride_bytes;
  if (a % (8 * sizeof(T)) == 0) return kWhole;
  return sizeof(T) == 4 && a % 16 == 0 ? kHalves : kSingly;
}

// Eight neighbouring elements as they lie in memory.  `valid` of them belong
// to the row; the others read as zeros and are not written.  Moves other
// than kSingly take all eight.
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
  __device__ __forceinline__ void load(const T* p, int valid, int move) {
    if (move == kWhole) {
      if constexpr (kVecs == 1)
        w[0] = ld_stream_v4(p);
      else
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w),
                       "=r"(w[kVecs - 1].x), "=r"(w[kVecs - 1].y), "=r"(w[kVecs - 1].z),
                       "=r"(w[kVecs - 1].w)
                     : "l"(p));
    } else if (move == kHalves) {
      // the halves of a sector come by two instructions: through L1
#pragma unroll
      for (int i = 0; i < kVecs; ++i) w[i] = ld_nc_v4(p + i * (16 / sizeof(T)));
    } else {
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < valid ? p[i] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void store(T* p, int valid, int move) const {
    if (move == kWhole) {
      if constexpr (kVecs == 1)
        st_stream_v4(p, w[0]);
      else
        asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0].x),
                     "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[kVecs - 1].x),
                     "r"(w[kVecs - 1].y), "r"(w[kVecs - 1].z), "r"(w[kVecs - 1].w)
                     : "memory");
    } else if (move == kHalves) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) st_stream_v4(p + i * (16 / sizeof(T)), w[i]);
    } else {
      const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) p[i] = e[i];
    }
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
