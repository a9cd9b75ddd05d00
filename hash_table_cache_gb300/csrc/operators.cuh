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

// Sum over the block, the same bits in every thread (a fixed tree).
// `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int warps = (blockDim.x + 31) >> 5;
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();  // red may still be read from an earlier call
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; ++w) s += red[w];
  return s;
}

}  // namespace hkv
