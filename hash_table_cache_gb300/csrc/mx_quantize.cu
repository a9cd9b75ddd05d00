// mx_quantize.cu -- hkv_mx_quantize and hkv_mx_dequantize: 4-bit microscaled
// copies of a matrix's rows and columns, and their values.
#include "mx.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;

// One thread per block of 32 elements, `step` elements apart in x; blocks and
// rows of the padding get a zero scale byte.
template <class T>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(uint64_t rows, uint64_t cols, const T* __restrict__ x, uint64_t row_step,
                    uint64_t col_step, uint8_t* codes, uint8_t* scales) {
  const uint64_t blocks = (cols + kMxBlock - 1) / kMxBlock, groups = (blocks + 3) / 4;
  const uint64_t padded_rows = (rows + 127) / 128 * 128;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint64_t row = row_step == 1 ? i % padded_rows : i / (groups * 4);
  const uint64_t block = row_step == 1 ? i / padded_rows : i % (groups * 4);
  if (row >= padded_rows || block >= groups * 4) return;
  uint32_t byte = 0;
  if (row < rows && block < blocks) {
    float v[kMxBlock];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kMxBlock; ++k) {
      const uint64_t c = block * kMxBlock + k;
      v[k] = c < cols ? to_f32(x[row * row_step + c * col_step]) : 0.f;
      most = max(most, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    }
    byte = mx_scale_byte(most);
    const float inv = mx_inverse(byte);
    uint4 out;
    uint32_t* word = &out.x;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = byte == 255 ? 0.f : v[8 * w + k] * inv;
      word[w] = mx_codes8(u);
    }
    *reinterpret_cast<uint4*>(codes + (row * blocks + block) * 16) = out;
  }
  scales[mx_scale_at(row, block, groups)] = static_cast<uint8_t>(byte);
}

// One thread per two elements.
template <class T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(uint64_t rows, uint64_t cols, const uint8_t* __restrict__ codes,
                      const uint8_t* __restrict__ scales, T* y, uint64_t stride) {
  const uint64_t blocks = (cols + kMxBlock - 1) / kMxBlock, groups = (blocks + 3) / 4;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint64_t row = i / (blocks * 16), c = i % (blocks * 16) * 2;
  if (row >= rows) return;
  const float s = mx_scale_value(scales[mx_scale_at(row, c / kMxBlock, groups)]);
  const uint32_t two = codes[row * blocks * 16 + c / 2];
  if (c < cols) y[row * stride + c] = from_f32<T>(mx_code_value(two & 15) * s);
  if (c + 1 < cols) y[row * stride + c + 1] = from_f32<T>(mx_code_value(two >> 4) * s);
}

template <class T>
cudaError_t quantize(uint64_t rows, uint64_t cols, const T* x, uint64_t row_step,
                     uint64_t col_step, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const uint64_t threads = (rows + 127) / 128 * 128 * ((cols + 127) / 128 * 4);
  quantize_kernel<T><<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(
      rows, cols, x, row_step, col_step, codes, scales);
  return cudaGetLastError();
}

bool shape_ok(uint64_t rows, uint64_t cols, uint64_t stride, int type) {
  return rows <= HKV_MAX_BATCH && cols <= HKV_MAX_BATCH && stride >= cols && type_ok(type);
}

}  // namespace
}  // namespace hkv

extern "C" {

hkv_status hkv_mx_quantize(uint64_t rows, uint64_t cols, const void* x, int x_type,
                           uint64_t x_stride, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                           uint8_t* scales_t, void* stream) {
  using namespace hkv;
  if (!shape_ok(rows, cols, x_stride, x_type)) return HKV_ERR_INVALID;
  if (rows == 0 || cols == 0) return HKV_OK;
  if (!x || !codes != !scales || !codes_t != !scales_t || (!codes && !codes_t))
    return HKV_ERR_INVALID;
  if (!aligned(x, type_size(x_type)) || !aligned(codes, 16) || !aligned(scales, 16) ||
      !aligned(codes_t, 16) || !aligned(scales_t, 16))
    return HKV_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return op_status(with_type(x_type, [&](auto* t) {
    auto* in = static_cast<decltype(t)>(const_cast<void*>(x));
    cudaError_t e = cudaSuccess;
    if (codes) e = quantize(rows, cols, in, x_stride, 1, codes, scales, st);
    if (e == cudaSuccess && codes_t) e = quantize(cols, rows, in, 1, x_stride, codes_t, scales_t, st);
    return e;
  }));
}

hkv_status hkv_mx_dequantize(uint64_t rows, uint64_t cols, const uint8_t* codes,
                             const uint8_t* scales, void* y, int y_type, uint64_t y_stride,
                             void* stream) {
  using namespace hkv;
  if (!shape_ok(rows, cols, y_stride, y_type)) return HKV_ERR_INVALID;
  if (rows == 0 || cols == 0) return HKV_OK;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(scales, 16) ||
      !aligned(y, type_size(y_type)))
    return HKV_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint64_t threads = rows * ((cols + 31) / 32) * 16;
  return op_status(with_type(y_type, [&](auto* t) {
    dequantize_kernel<<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        rows, cols, codes, scales, static_cast<decltype(t)>(y), y_stride);
    return cudaGetLastError();
  }));
}

}  // extern "C"
