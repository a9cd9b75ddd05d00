// logits.cuh -- rows of logits: what the kernels that take log probabilities
// from them share (preference.cu, token_logps.cu).
#pragma once

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "operators.cuh"

namespace hkv {

constexpr int kThreads = 256;       // a row's or a piece's, where a block takes it
constexpr int kWarpThreads = 128;   // four rows, where a warp takes one
constexpr int kMaxParts = 8;  // blocks of a cluster that share a row
// 16-byte loads in flight per thread where kLanes threads share a row
__host__ __device__ constexpr int unroll(int lanes) { return lanes == 32 ? 8 : 4; }
// log2 e in two floats: one alone is off by 1e-8 of it, which leans one way in
// every exponential
constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;
// Below this maximum exp(x - max) is taken as 2^(x log2 e - c) 2^(c - max log2
// e), c the rounded max log2 e: the second exponent is half a unit of c, at most
// 0.0013 here, and its power three terms of a series (left out: 1.2e-10).  It
// grows with the maximum (a mask such as -1e10 where a thread has met nothing
// else), past 127 from 2e9 on, where one factor would be infinite and the other 0.
constexpr float kFactored = 16384.f;
// 2^-x for |x| below 0.002 (the gradient of token_logps.cu has in x what a float leaves
// out of the log sum as well, up to 0.0007): three terms, and below 4.5e-10 left out
__device__ __forceinline__ float exp2_of_minus(float x) {
  return fmaf(x * x, 0.240226507f, fmaf(-x, 0.693147181f, 1.f));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats in one 64-bit register: one instruction works on both.
__device__ __forceinline__ uint64_t both(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 parts(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_both(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_both(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Neighbouring elements in 16 bytes.
template <class T>
struct Chunk {
  static constexpr int kN = 16 / sizeof(T);
  uint4 w;
  __device__ __forceinline__ float at(int i) const {
    return to_f32(reinterpret_cast<const T*>(&w)[i]);
  }
  __device__ __forceinline__ void fill_lowest() {  // -inf
    const uint32_t v = sizeof(T) == 4                         ? 0xFF800000u
                       : std::is_same_v<T, __nv_bfloat16> ? 0xFF80FF80u
                                                          : 0xFC00FC00u;
    w = make_uint4(v, v, v, v);
  }
};
// The largest of N chunks' elements; 16-bit ones two at a time.  NaNs are
// passed over: the sum of exponentials brings them in.
template <class T, int N>
__device__ __forceinline__ float largest(const Chunk<T> (&c)[N]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, c[u].at(i));
    return m;
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __nv_bfloat16>, __nv_bfloat162, __half2>;
    T2 m = *reinterpret_cast<const T2*>(&c[0].w.x);
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __hmax2(m, reinterpret_cast<const T2*>(&c[u].w)[i]);
    return fmaxf(to_f32(m.x), to_f32(m.y));
  }
}
template <class T>
__device__ __forceinline__ uint32_t to_boundary(const T* p, uint64_t n) {
  const uint32_t head = (16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T);
  return n < head ? static_cast<uint32_t>(n) : head;
}

// A running maximum m and s = sum exp(x - m).  Nothing seen, or only -inf:
// m = -inf, s = 0.  A NaN or +inf among the values makes s NaN.
struct Running {
  float m = -INFINITY, s = 0.f;

  // Raises the maximum to that of the next values, and returns what to
  // subtract from them (0 while all are -inf: their exponentials are 0).
  __device__ __forceinline__ float raise(float top) {
    if (top > m) {
      s *= expf(m - top);
      m = top;
    }
    return m == -INFINITY ? 0.f : m;
  }
  __device__ __forceinline__ void one(float x) {
    const float base = raise(x);
    s += __expf(x - base);
  }
  __device__ __forceinline__ void join(float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = (m == top ? s : s * expf(m - top)) + (m2 == top ? s2 : s2 * expf(m2 - top));
    m = top;
  }
  // m + log s as a float and what it leaves out.  With s = 2^e f the product
  // of e and the upper digits of log 2 is exact (Cody and Waite), and so is
  // what the addition to m rounds off.
  __device__ __forceinline__ float log_sum(float& rest) const {
    rest = 0.f;
    if (!(s >= FLT_MIN && s <= FLT_MAX && fabsf(m) <= FLT_MAX))
      return m == -INFINITY && s == 0.f ? -INFINITY : m + logf(s);
    const int bits = __float_as_int(s), e = (bits >> 23) - 127;
    const float f = __int_as_float((bits & 0x7FFFFF) | 0x3F800000);
    const float a = static_cast<float>(e) * 0.693145751953125f;
    const float hi = m + a, back = hi - m;
    const float lo = (m - (hi - back)) + (a - back) +
                     (logf(f) + static_cast<float>(e) * 1.42860682e-6f);
    const float l = hi + lo;
    rest = lo - (l - hi);
    return l;
  }
};

__device__ __forceinline__ bool counts(int64_t label, uint64_t vocab) {
  return label >= 0 && static_cast<uint64_t>(label) < vocab;
}

// A warp takes a row (not a block) of at most 4 KB, a few rounds of its loads,
// or of 16 KB where there are enough rows for every warp of the GPU.  Forward
// and backward, by warps and by blocks: 64 rows of 4000 bytes 5.3 and 3.0 us, 5.6
// and 2.3; 64 of 16000 7.2 and 3.0, 5.7 and 3.0; 4096 of 4000 10.1 and 7.1, 22.0 and
// 12.0; 16384 of 16000 58.5 and 77.0, 76.6 and 76.5; 4096 of 64000 56.2 and 76.3, 52.3
// and 76.1.
inline bool by_warps(uint64_t rows, uint64_t row_bytes) {
  return row_bytes <= 4096 || (row_bytes <= 16384 && rows >= 32ull * sm_count());
}

}  // namespace hkv
