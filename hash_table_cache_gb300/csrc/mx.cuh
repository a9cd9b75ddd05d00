// mx.cuh -- the 4-bit microscaled format (include/hkv.h) in device code.
#pragma once

#include "operators.cuh"

namespace hkv {

constexpr int kMxBlock = HKV_MX_BLOCK;  // columns that share a scale

// Position of the scale byte of (row, block) in a matrix of `groups` 4-block
// groups per row: 512-byte groups of 128 rows by 4 blocks, in the order in
// which the tensor cores read a group's scales (32 lanes of 16 bytes).
__host__ __device__ inline uint64_t mx_scale_at(uint64_t row, uint64_t block, uint64_t groups) {
  return ((row >> 7) * groups + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// Scale byte of a block whose largest magnitude has these float32 bits (sign
// cleared).  The bits of a NaN are the largest of all, so the maximum over
// the magnitudes' bits finds NaNs and infinities too.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t most) {
  const uint32_t e = most >> 23;
  return e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
}
// 1 / scale as a float32, a power of two (0 for the NaN scale, whose codes
// are 0; byte 253 and 254 do not occur).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255 ? 0.f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 1u << 22 : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Eight floats (already divided by their scale) as eight e2m1 codes, the
// first in the lowest bits: nearest, ties to the even code, 6 above it.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight e2m1 codes, the first in the lowest bits.
__device__ __forceinline__ void mx_values8(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n"
      " mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n"
      " cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

}  // namespace hkv
