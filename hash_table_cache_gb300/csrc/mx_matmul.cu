// mx_matmul.cu -- hkv_mx_matmul: the product of two 4-bit microscaled matrices.
#include "mx.cuh"

namespace hkv {
namespace {

constexpr int kTile = 32;  // rows of A and of B per thread block

__device__ unsigned long long g_wait_timeouts;

// A 32 x 32 tile of y per thread block, 32 columns of k at a time.
template <class T>
__global__ void __launch_bounds__(256)
    matmul_kernel(uint64_t m, uint64_t n, uint64_t k, const uint8_t* __restrict__ a_codes,
                  const uint8_t* __restrict__ a_scales, const uint8_t* __restrict__ b_codes,
                  const uint8_t* __restrict__ b_scales, T* y, uint64_t stride) {
  __shared__ float a[kTile][33], b[kTile][33];
  const uint64_t blocks = (k + 31) / 32, groups = (blocks + 3) / 4;
  const uint64_t m0 = static_cast<uint64_t>(blockIdx.y) * kTile;
  const uint64_t n0 = static_cast<uint64_t>(blockIdx.x) * kTile;
  float acc[4] = {};
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  for (uint64_t kb = 0; kb < blocks; ++kb) {
    for (int i = threadIdx.x; i < kTile * 16; i += 256) {
      const int r = i / 16, c = i % 16;
      uint32_t ca = 0, cb = 0;
      float sa = 0.f, sb = 0.f;
      if (m0 + r < m) {
        ca = a_codes[((m0 + r) * blocks + kb) * 16 + c];
        sa = mx_scale_value(a_scales[mx_scale_at(m0 + r, kb, groups)]);
      }
      if (n0 + r < n) {
        cb = b_codes[((n0 + r) * blocks + kb) * 16 + c];
        sb = mx_scale_value(b_scales[mx_scale_at(n0 + r, kb, groups)]);
      }
      a[r][2 * c] = mx_code_value(ca & 15) * sa;
      a[r][2 * c + 1] = mx_code_value(ca >> 4) * sa;
      b[r][2 * c] = mx_code_value(cb & 15) * sb;
      b[r][2 * c + 1] = mx_code_value(cb >> 4) * sb;
    }
    __syncthreads();
    for (int q = 0; q < 32; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += a[ty + 8 * j][q] * b[tx][q];
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (m0 + ty + 8 * j < m && n0 + tx < n)
      y[(m0 + ty + 8 * j) * stride + n0 + tx] = from_f32<T>(acc[j]);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>((n + kTile - 1) / kTile),
                  static_cast<unsigned>((m + kTile - 1) / kTile));
  return op_status(with_type(y_type, [&](auto* t) {
    matmul_kernel<<<grid, 256, 0, st>>>(m, n, k, a_codes, a_scales, b_codes, b_scales,
                                        static_cast<decltype(t)>(y), y_stride);
    return cudaGetLastError();
  }));
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
