// mx_quantize.cu -- hkv_mx_quantize and hkv_mx_dequantize: 4-bit microscaled
// copies of a matrix's rows and columns, and their values.
//
// Both are bound by memory.  A thread block takes a tile of 128 rows by 128
// columns, which is one 512-byte group of scales in either direction: 16
// threads read 128 neighbouring columns of a row, 8 each, and every thread
// has the rows r, r + 32, r + 64 and r + 96 in flight together, because those
// four rows' scales are 16 neighbouring bytes of the group.  Four threads
// share a block of 32 and agree on its largest magnitude by two shuffles.
// For a copy along the columns the tile goes through shared memory as it was
// read, and four threads take the 128 rows of a column (or of two neighbouring
// 16-bit columns), so that they write 64 neighbouring bytes of codes; both
// copies come from one read of x.
//
// Times (GB300): rows of 1000003 x 128 float32 81 us, 7.2 TB/s, their columns 95
// us, both 110 us, and the rows' values as bfloat16 48 us, 6.7 TB/s; 8192 x 8192
// bfloat16 rows 26 us, 6.5 TB/s, columns 32 us, 5.4 TB/s, both copies 42 us, 5.0
// TB/s, where the conversions and maxima of two copies take longer than the
// memory.  Rows that start off 16-byte boundaries: 8200 x 4095 bfloat16 rows 33
// us, columns 34, both 39, values 23 us.
#include <type_traits>

#include "mx.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;

// The end of a row of `cols` elements as seen from element c, within -32 .. 32:
// what Eight takes.
__device__ __forceinline__ int limit(uint64_t cols, uint64_t c) {
  const int64_t d = static_cast<int64_t>(cols) - static_cast<int64_t>(c);
  return static_cast<int>(min(max(d, static_cast<int64_t>(-32)), static_cast<int64_t>(32)));
}

// Running maxima of magnitudes.  A word holds one float32 (compared as an
// integer, which puts NaNs above infinity) or two 16-bit elements, whose maxima
// are kept apart until the end: one instruction for two elements.  A NaN stays.
template <class T>
__device__ __forceinline__ uint32_t most(uint32_t m, uint32_t word) {
  if constexpr (sizeof(T) == 4) {
    return max(m, word & 0x7FFFFFFFu);
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __nv_bfloat16>, __nv_bfloat162, __half2>;
    const T2 r = __hmax2_nan(*reinterpret_cast<const T2*>(&m), __habs2(*reinterpret_cast<const T2*>(&word)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
// Of two of them.
template <class T>
__device__ __forceinline__ uint32_t most_of(uint32_t m, uint32_t other) {
  if constexpr (sizeof(T) == 4) return max(m, other);
  return __vmaxu2(m, other);
}
// One of them as float32 bits: of a float32, or of the lower (0) or upper (1)
// elements of the words.
template <class T>
__device__ __forceinline__ uint32_t magnitude(uint32_t m, int k) {
  if constexpr (sizeof(T) == 4) return m;
  const uint32_t h = k ? m >> 16 : m & 0xFFFFu;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t byte, float inverse) {
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = v[i] * inverse;
  const uint32_t code = mx_codes8(u);
  return byte == 255 ? 0 : code;
}

// While one block waits for its tile another encodes: five per SM for 16-bit
// elements (rows of 8200 x 4095: 33 us, with four 38), four for float32
// (both copies of 8192 x 8192: 62 us, with five 71).
template <class T, bool kRowCopy, bool kColCopy>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4)
    quantize_kernel(uint64_t rows, uint64_t cols, const T* __restrict__ x, uint64_t stride,
                    int move, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                    uint8_t* scales_t) {
  // The tile in 32-bit words; word w of a row in the tile's quarter q lies at
  // w ^ 8q, which spreads the four quarters of a column over the banks.
  constexpr int kWords = kTile * sizeof(T) / 4;
  extern __shared__ uint32_t tile[];
  pdl_trigger();
  pdl_wait();
  const uint64_t blocks = (cols + 31) / 32, groups = (cols + 127) / 128;
  const uint64_t blocks_t = (rows + 31) / 32, groups_t = (rows + 127) / 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (uint64_t t = blockIdx.x; t < groups * groups_t; t += gridDim.x) {
    const uint64_t tile_c = t % groups, tile_r = t / groups;
    const uint64_t c = tile_c * kTile + tx * 8, row0 = tile_r * kTile;
    const int lo = tile_c ? -16 : -8 * tx, hi = limit(cols, c);
    const int rows_here = rows - row0 < kTile ? static_cast<int>(rows - row0) : kTile;
    const bool inside = move != kShifted && hi >= 8 && rows_here == kTile;
    const T* in = x + (row0 + ty) * stride + c;
    uint8_t* out = codes + (row0 + ty) * blocks * 16 + c / 2;
#pragma unroll
    for (int h = 0; h < 2; ++h, in += 16 * stride, out += 256 * blocks) {
      const int r = ty + 16 * h;
      Eight<T> e[4];
      if (inside) {
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q].load_aligned(in + q * (32 * stride), move);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool row = r + 32 * q < rows_here;
          e[q].load(in + q * (32 * stride), row ? lo : 0, row ? hi : 0, move, tx);
        }
      }
      if (kColCopy) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t* line = tile + (r + 32 * q) * kWords;
#pragma unroll
          for (int i = 0; i < Eight<T>::kVecs; ++i)
            *reinterpret_cast<uint4*>(line + ((tx * 4 * Eight<T>::kVecs) ^ (8 * q)) + 4 * i) = e[q].w[i];
        }
      }
      if (kRowCopy) {
        // this block's scale bytes of the four rows, one byte each
        uint32_t four = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t* words = reinterpret_cast<const uint32_t*>(e[q].w);
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4 * Eight<T>::kVecs; ++i) m = most<T>(m, words[i]);
          m = most_of<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = most_of<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const uint32_t byte = mx_scale_byte(max(magnitude<T>(m, 0), magnitude<T>(m, 1)));
          float v[8];
          e[q].to(v);
          const uint32_t code = encode8(v, byte, mx_inverse(byte));
          if (inside || (r + 32 * q < rows_here && (c >> 5) < blocks))
            *reinterpret_cast<uint32_t*>(out + q * (512 * blocks)) = code;
          four |= byte << (8 * q);
        }
        // four blocks' bytes of a row are neighbours in the group
        const uint32_t b1 = __shfl_down_sync(0xFFFFFFFFu, four, 4);
        const uint32_t b2 = __shfl_down_sync(0xFFFFFFFFu, four, 8);
        const uint32_t b3 = __shfl_down_sync(0xFFFFFFFFu, four, 12);
        if (tx == 0) {
          const uint32_t a01 = __byte_perm(four, b1, 0x5140), a23 = __byte_perm(b2, b3, 0x5140);
          const uint32_t c01 = __byte_perm(four, b1, 0x7362), c23 = __byte_perm(b2, b3, 0x7362);
          *reinterpret_cast<uint4*>(scales + t * 512 + r * 16) =
              make_uint4(__byte_perm(a01, a23, 0x5410), __byte_perm(a01, a23, 0x7632),
                         __byte_perm(c01, c23, 0x5410), __byte_perm(c01, c23, 0x7632));
        }
      }
    }
    if (kColCopy) {
      __syncthreads();
      const int q = threadIdx.x & 3;
      constexpr int kPer = 4 / sizeof(T);  // columns in a word
      for (int w = threadIdx.x >> 2; w < kWords; w += kThreads / 4) {
        uint32_t word[32], m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          word[i] = tile[(32 * q + i) * kWords + (w ^ (8 * q))];
          m = most<T>(m, word[i]);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const uint32_t byte = mx_scale_byte(magnitude<T>(m, k));
          const float inverse = mx_inverse(byte);
          uint32_t code[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32(reinterpret_cast<const T*>(&word[8 * g + i])[k]);
            code[g] = encode8(v, byte, inverse);
          }
          const uint4 all = make_uint4(code[0], code[1], code[2], code[3]);
          const uint64_t col = tile_c * kTile + w * kPer + k, block = tile_r * 4 + q;
          if (col < cols && block < blocks_t)
            *reinterpret_cast<uint4*>(codes_t + (col * blocks_t + block) * 16) = all;
          uint32_t packed = byte << (8 * q);
          packed |= __shfl_xor_sync(0xFFFFFFFFu, packed, 1);
          packed |= __shfl_xor_sync(0xFFFFFFFFu, packed, 2);
          if (q == 0)
            *reinterpret_cast<uint32_t*>(scales_t + mx_scale_at(col, block, groups_t)) = packed;
        }
      }
      __syncthreads();
    }
  }
}

// kShifted: y's rows start anywhere.  A thread then takes, instead of its eight
// columns, the eight that lie between boundaries in y, `tail` of them before
// its own: the codes are shifted, not the values.
template <class T, bool kShifted>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(uint64_t rows, uint64_t cols, const uint8_t* __restrict__ codes,
                      const uint8_t* __restrict__ scales, T* y, uint64_t stride, int move) {
  pdl_trigger();
  pdl_wait();
  const uint64_t blocks = (cols + 31) / 32, groups = (cols + 127) / 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const uint64_t tiles = groups * ((rows + 127) / 128);
  for (uint64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint64_t tile_c = t % groups, c = tile_c * kTile + tx * 8, row0 = t / groups * kTile;
    const bool own = c < cols, left = kShifted && c > 0 && c - 8 < cols;
    if (!own && !left) continue;
    uint32_t code[8], code_left[8];
    uint4 scale[2], scale_left[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t at = t * 512 + (ty + 16 * h) * 16;
      scale[h] = scale_left[h] = ld_nc_v4(scales + at);
      if (kShifted && tx == 0 && left) scale_left[h] = ld_nc_v4(scales + at - 512);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t row = row0 + ty + 16 * h + 32 * q;
        const uint32_t* word = reinterpret_cast<const uint32_t*>(codes + row * blocks * 16 + c / 2);
        code[4 * h + q] = own && row < rows ? __ldg(word) : 0;
        code_left[4 * h + q] = left && row < rows ? __ldg(word - 1) : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t row = row0 + ty + 16 * (i >> 2) + 32 * (i & 3);
      if (row >= rows) continue;
      T* out = y + row * stride + c;
      const uint32_t four = reinterpret_cast<const uint32_t*>(&scale[i >> 2])[i & 3];
      const float s = mx_scale_value(four >> (8 * (tx >> 2)) & 255);
      float v[8];
      Eight<T> e;
      if constexpr (!kShifted) {
        mx_values8(code[i], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= s;
        e.from(v);
        if (c + 8 <= cols) {
          e.store_aligned(out, move);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < cols) out[k] = from_f32<T>(v[k]);
        }
      } else {
        const int tail = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
        const uint32_t four_left = reinterpret_cast<const uint32_t*>(&scale_left[i >> 2])[i & 3];
        const float s_left = mx_scale_value(four_left >> (8 * ((tx + 15 & 15) >> 2)) & 255);
        mx_values8(__funnelshift_l(code_left[i], code[i], 4 * tail), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= k < tail ? s_left : s;
        e.from(v);
        out -= tail;
        // the columns of out[0 .. 7] that lie in the row
        const int lo = c ? 0 : tail, hi = limit(cols, c) + tail;
        if (lo == 0 && hi >= 8) {
          e.store_aligned(out, kHalves);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k >= lo && k < hi) out[k] = from_f32<T>(v[k]);
        }
        // a row that ends with this tile has no thread for what is left of it
        if (tx == 15 && tile_c == groups - 1 && tail && own) {
          mx_values8(code[i], v);
#pragma unroll
          for (int k = 1; k < 8; ++k)
            if (k >= 8 - tail && c + k < cols) out[tail + k] = from_f32<T>(v[k] * s);
        }
      }
    }
  }
}

unsigned tile_grid(uint64_t rows, uint64_t cols) {
  const uint64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
  return static_cast<unsigned>(tiles < 0x7FFFFFFF ? tiles : 0x7FFFFFFF);
}

template <class T, bool kRowCopy, bool kColCopy>
cudaError_t quantize(uint64_t rows, uint64_t cols, const T* x, uint64_t stride, uint8_t* codes,
                     uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, cudaStream_t st) {
  const int move = widest<T>(x, stride * sizeof(T));
  const size_t smem = kColCopy ? kTile * kTile * sizeof(T) : 0;
  auto* kernel = quantize_kernel<T, kRowCopy, kColCopy>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_chained(kernel, tile_grid(rows, cols), kThreads, smem, st, rows, cols, x, stride,
                        move, codes, scales, codes_t, scales_t);
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
    using T = std::remove_pointer_t<decltype(t)>;
    const T* in = static_cast<const T*>(x);
    return (!codes_t ? quantize<T, true, false>
            : !codes ? quantize<T, false, true>
                     : quantize<T, true, true>)(rows, cols, in, x_stride, codes, scales, codes_t,
                                                scales_t, st);
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
  return op_status(with_type(y_type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const int move = widest<T>(y, y_stride * sizeof(T));
    return launch_chained(move == kShifted ? dequantize_kernel<T, true> : dequantize_kernel<T, false>,
                          tile_grid(rows, cols), kThreads, 0, st, rows, cols, codes, scales,
                          static_cast<T*>(y), y_stride, move);
  }));
}

}  // extern "C"
