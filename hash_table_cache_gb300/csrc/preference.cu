// preference.cu -- hkv_preference_loss and hkv_preference_loss_backward: the
// logistic loss of paired log ratios, from logits, and its gradient.
//
// The logits are what costs: the forward call reads them once, keeping a
// running maximum and the sum of exponentials relative to it (one pass over
// a row, no second one for the maximum), and the backward call reads and
// writes once.  A hidden token's row is not read.  Rows are taken by a warp
// or by a block, depending on their length; a few long rows are shared by
// the blocks of a cluster, which join their parts through distributed shared
// memory in a fixed order, so no partial result goes through global memory.
//
// Times (GB300): 8192 x 131072 bfloat16, a quarter of the tokens hidden,
// forward 253 us (6.4 TB/s of what is read), backward 540 us (6.9 TB/s); 4096
// x 32768 forward 42 us (4.8 TB/s: 8 blocks per SM take the rows in two and a
// half rounds, and the exponentials alone would take 20 us), backward 70 us;
// 32768 x 2000 27 and 37 us; 96 x 1000 float32 5.0 and 2.7 us.  4096 x 50257 as
// the first columns of 50304 forward 62 us, backward 106 us into a matrix of the
// same stride and 326 us, element by element, into a contiguous one.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "operators.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;       // a row's or a piece's, where a block takes it
constexpr int kWarpThreads = 128;   // four rows, where a warp takes one
constexpr int kPairThreads = 256;
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
// 2^-x for |x| below 0.0013
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

// One thread's share of a row of n elements, taken by kLanes threads.
template <class T, int kLanes>
__device__ __forceinline__ Running row_pass(const T* x, uint64_t n, int lane) {
  constexpr int kN = Chunk<T>::kN, kUnroll = unroll(kLanes);
  Running r;
  const uint32_t head = to_boundary(x, n);
  if (lane < static_cast<int>(head)) r.one(to_f32(x[lane]));
  const T* body = x + head;
  const uint64_t chunks = (n - head) / kN;
  for (uint64_t k = lane; k < chunks; k += kUnroll * kLanes) {
    Chunk<T> c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (k + u * kLanes < chunks) c[u].w = ld_stream_v4(body + (k + u * kLanes) * kN);
      else c[u].fill_lowest();
    }
    const float base = r.raise(largest(c));
    if (fabsf(base) < kFactored) {
      // exp(x - base) as 2^(x log2 e - base log2 e), by two multiply-adds.  The
      // same rounded base log2 e is in every term; what it is off by is taken
      // out of their sum.
      const float scaled = base * kLog2e;
      const float off = fmaf(base, kLog2eRest, fmaf(base, kLog2e, -scaled));
      const uint64_t l = both(kLog2e, kLog2e), rest = both(kLog2eRest, kLog2eRest);
      const uint64_t minus = both(-scaled, -scaled);
      uint64_t sum[2] = {};
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const uint64_t x2 = both(c[u].at(i), c[u].at(i + 1));
          const float2 a = parts(fma_both(x2, rest, fma_both(x2, l, minus)));
          sum[i / 2 & 1] = add_both(sum[i / 2 & 1], both(exp2_approx(a.x), exp2_approx(a.y)));
        }
      const float2 t = parts(add_both(sum[0], sum[1]));
      r.s = fmaf(t.x + t.y, exp2_of_minus(off), r.s);
    } else {
      float part = 0.f;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i) part += __expf(c[u].at(i) - base);
      r.s += part;
    }
  }
  const uint64_t tail = head + chunks * kN + lane;
  if (tail < n) r.one(to_f32(x[tail]));
  return r;
}

__device__ __forceinline__ bool counts(int64_t label, uint64_t vocab) {
  return label >= 0 && static_cast<uint64_t>(label) < vocab;
}

// A warp's lanes: the maximum first, so that each sum is brought to it once.
__device__ __forceinline__ Running join_lanes(Running r) {
  float top = r.m;
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (r.m != top) r.s *= expf(r.m - top);
  r.m = top;
  for (int o = 16; o > 0; o >>= 1) r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
  return r;
}

__device__ __forceinline__ void finish_row(const Running& r, float chosen, uint64_t t, float* logps,
                                           float* lse) {
  float rest;
  const float l = r.log_sum(rest);
  lse[t] = l;
  logps[t] = (chosen - l) - rest;
}

// A warp per row: short rows.
template <class T>
__global__ void __launch_bounds__(kWarpThreads)
    short_rows_kernel(uint64_t rows, uint64_t vocab, const T* __restrict__ logits, uint64_t stride,
                      const int64_t* __restrict__ labels, float* logps, float* lse,
                      float* row_grad, int32_t* row_pair) {
  pdl_trigger();
  pdl_wait();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * (kWarpThreads / 32) + threadIdx.x / 32;
  if (t >= rows) return;
  const int lane = threadIdx.x & 31;
  const int64_t label = labels[t];
  if (lane == 0) {
    row_grad[t] = 0.f;
    row_pair[t] = -1;
  }
  const T* x = logits + t * stride;
  if (!counts(label, vocab)) {
    if (lane == 0) logps[t] = lse[t] = 0.f;
    return;
  }
  const float chosen = lane == 0 ? to_f32(x[label]) : 0.f;
  const Running r = join_lanes(row_pass<T, 32>(x, vocab, lane));
  if (lane == 0) finish_row(r, chosen, t, logps, lse);
}

// A block per row, or the `parts` blocks of a cluster.
template <class T>
__global__ void __launch_bounds__(kThreads, 8)
    long_rows_kernel(uint64_t vocab, const T* __restrict__ logits, uint64_t stride, uint32_t parts,
                     const int64_t* __restrict__ labels, float* logps, float* lse, float* row_grad,
                     int32_t* row_pair) {
  __shared__ float ms[2][kThreads / 32 + 1];  // [maximum or sum][warp, then the block]
  pdl_trigger();
  pdl_wait();
  const uint64_t t = blockIdx.x / parts;
  const uint32_t part = blockIdx.x % parts;
  const int64_t label = labels[t];
  const bool writes = part == 0 && threadIdx.x == 0;
  if (writes) {
    row_grad[t] = 0.f;
    row_pair[t] = -1;
  }
  if (!counts(label, vocab)) {
    if (writes) logps[t] = lse[t] = 0.f;
    return;  // every block of the cluster
  }
  const T* x = logits + t * stride;
  const float chosen = writes ? to_f32(x[label]) : 0.f;  // on its way while the row is read
  // parts start at multiples of 64 elements of the row
  const uint64_t size = ((vocab + parts - 1) / parts + 63) / 64 * 64;
  const uint64_t lo = min(part * size, vocab), hi = min(lo + size, vocab);
  Running r = join_lanes(row_pass<T, kThreads>(x + lo, hi - lo, threadIdx.x));
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    ms[0][warp] = r.m;
    ms[1][warp] = r.s;
  }
  __syncthreads();
  if (warp == 0) {
    r = Running{};
    if (threadIdx.x < kThreads / 32) {
      r.m = ms[0][threadIdx.x];
      r.s = ms[1][threadIdx.x];
    }
    r = join_lanes(r);
    if (threadIdx.x == 0) {
      ms[0][kThreads / 32] = r.m;
      ms[1][kThreads / 32] = r.s;
    }
  }
  if (parts > 1) {
    __syncwarp();
    cluster_sync();
    if (writes)
      for (uint32_t p = 1; p < parts; ++p)
        r.join(remote_f32(smem_u32(&ms[0][kThreads / 32]), p),
               remote_f32(smem_u32(&ms[1][kThreads / 32]), p));
    __syncwarp();
    cluster_sync();  // the others stay until their parts are read
  }
  if (writes) finish_row(r, chosen, t, logps, lse);
}

// One pair per block: the sums of both sequences, the loss, and the loss's
// slope for each of their tokens.
__global__ void __launch_bounds__(kPairThreads)
    pair_kernel(uint64_t pairs, uint64_t rows, uint64_t vocab, const int64_t* __restrict__ labels,
                const int64_t* __restrict__ offsets, const float* __restrict__ ref, float beta,
                float smoothing, int average, float* losses, float* ratios,
                const float* logps, float* row_grad, int32_t* row_pair) {
  __shared__ float red[kPairThreads / 32 * 4];
  pdl_trigger();
  pdl_wait();
  const uint64_t p = blockIdx.x;
  uint64_t lo[2], hi[2];
  float sums[4] = {};  // ratio and number of counted tokens, of either side
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint64_t s = p + side * pairs;
    const int64_t a = offsets[s], b = offsets[s + 1];
    lo[side] = a <= 0 ? 0 : min(static_cast<uint64_t>(a), rows);
    hi[side] = b <= 0 ? 0 : min(static_cast<uint64_t>(b), rows);
  }
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (uint64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) {
      const float lp = logps[t], re = ref ? ref[t] : 0.f;
      if (counts(labels[t], vocab)) {
        sums[2 * side] += lp - re;
        sums[2 * side + 1] += 1.f;
      }
    }
  block_sums(sums, red);
  float r[2], inv[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const float n = sums[2 * side + 1];
    inv[side] = average ? (n > 0.f ? 1.f / n : 0.f) : 1.f;
    r[side] = average ? sums[2 * side] * inv[side] : sums[2 * side];
  }
  const float h = beta * (r[0] - r[1]);
  // a side with weight 0 is left out: its logarithm may be infinite
  const float tail = log1pf(expf(-fabsf(h)));
  float loss = 0.f, slope = 0.f;
  if (smoothing < 1.f) {
    loss += (1.f - smoothing) * (tail + fmaxf(-h, 0.f));
    slope -= (1.f - smoothing) / (1.f + expf(h));
  }
  if (smoothing > 0.f) {
    loss += smoothing * (tail + fmaxf(h, 0.f));
    slope += smoothing / (1.f + expf(-h));
  }
  if (isnan(h)) loss = slope = h;
  slope *= beta;
  if (threadIdx.x == 0) {
    losses[p] = loss;
    ratios[p] = r[0];
    ratios[pairs + p] = r[1];
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const float g = (side ? -slope : slope) * inv[side];
#pragma unroll 4
    for (uint64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) {
      row_pair[t] = static_cast<int32_t>(p);
      if (counts(labels[t], vocab)) row_grad[t] = g;
    }
  }
}

// The log-sum-exp in one float is off by half a unit of itself, and so are all
// the exponentials of its row: 6e-5 at 1024.  Logits as large are masks, in a
// row whose mask leaves nothing (at -1e10 each of its exponentials would come
// out as 1 instead of 1 / vocab), and such rows are taken by their maximum.
constexpr float kOneFloat = 1024.f;
__device__ __forceinline__ bool is_far(float lse) {
  return fabsf(lse) >= kOneFloat && fabsf(lse) <= FLT_MAX;
}

// Such a row as a whole by kLanes threads, each with elements of its own that it
// alone reads and writes.
template <class T, int kLanes>
__device__ __forceinline__ void far_row(const T* x, T* d, uint64_t vocab, uint64_t label, float g,
                                        uint32_t lane) {
  __shared__ float red[2][kThreads / 32];
  float m = -INFINITY, s = 0.f;
#pragma unroll 1
  for (uint64_t k = lane; k < vocab; k += kLanes) m = fmaxf(m, to_f32(x[k]));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if constexpr (kLanes > 32) {
    if (lane % 32 == 0) red[0][lane / 32] = m;
    __syncthreads();
    for (int w = 0; w < kLanes / 32; ++w) m = fmaxf(m, red[0][w]);
  }
#pragma unroll 1
  for (uint64_t k = lane; k < vocab; k += kLanes) s += expf(to_f32(x[k]) - m);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if constexpr (kLanes > 32) {
    if (lane % 32 == 0) red[1][lane / 32] = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < kLanes / 32; ++w) s += red[1][w];
    __syncthreads();  // red is free for the block's next row
  }
#pragma unroll 1
  for (uint64_t k = lane; k < vocab; k += kLanes) {
    const float soft = expf(to_f32(x[k]) - m) / s;
    d[k] = from_f32<T>(k == label ? g * (1.f - soft) : -g * soft);
  }
}

// A piece of a row for every kLanes threads, as many chunks of 16 bytes per
// thread as it keeps in flight.  Rows run from the last to the first, so that
// what the forward call read last is taken from L2 while it is there.  (72 and 32
// registers; 32768 x 2000 bfloat16 takes 36.7 us with 72, 37.6 with 64.)
template <class T, int kLanes>
__global__ void __launch_bounds__(kLanes == 32 ? kWarpThreads : kThreads, kLanes == 32 ? 7 : 8)
    backward_kernel(uint64_t pairs, uint64_t rows, uint64_t vocab, const T* logits, uint64_t stride,
                    uint64_t pieces, const int64_t* __restrict__ labels,
                    const float* __restrict__ lse, const float* __restrict__ row_grad,
                    const int32_t* __restrict__ row_pair, const float* __restrict__ dlosses,
                    T* dlogits, uint64_t dstride) {
  constexpr int kN = Chunk<T>::kN, kUnroll = unroll(kLanes);
  constexpr int kTeams = (kLanes == 32 ? kWarpThreads : kThreads) / kLanes;
  constexpr uint64_t kPiece = kLanes * kUnroll * kN;
  const uint32_t lane = threadIdx.x % kLanes;
  pdl_trigger();
  pdl_wait();
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kTeams;
  const uint64_t begin = static_cast<uint64_t>(blockIdx.x) * kTeams + threadIdx.x / kLanes;
  bool far = false;  // a row of which this team has the first piece
  for (uint64_t b = begin; b < rows * pieces; b += step) {
    const uint64_t t = rows - 1 - b / pieces, lo = b % pieces * kPiece;
    const int64_t label = labels[t];
    const int32_t p = row_pair[t];
    const bool counted = p >= 0 && static_cast<uint64_t>(p) < pairs && counts(label, vocab);
    const float g = counted ? row_grad[t] * (dlosses ? dlosses[p] : 1.f) : 0.f;
    const float l = counted ? lse[t] : 0.f;
    const uint64_t hit = counted && static_cast<uint64_t>(label) >= lo
                             ? static_cast<uint64_t>(label) - lo : ~0ull;
    const T* x = logits + t * stride + lo;
    T* d = dlogits + t * dstride + lo;
    const uint64_t n = min(vocab - lo, kPiece);
    auto value = [&](float v, uint64_t at) {
      const float soft = __expf(v - l);
      return at == hit ? g * (1.f - soft) : -g * soft;
    };
    auto one = [&](uint64_t at) { d[at] = from_f32<T>(counted ? value(to_f32(x[at]), at) : 0.f); };
    const uint32_t head = to_boundary(d, n);
    const bool alike = to_boundary(x, n) == head;
    const uint32_t chunks = static_cast<uint32_t>((n - head) / kN);
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t k = lane + u * kLanes;
      if (counted && alike && k < chunks) w[u] = __ldcs(reinterpret_cast<const uint4*>(x + head + k * kN));
    }
    if (is_far(l)) {  // asked when the logits are on their way
      far |= lo == 0;
      continue;
    }
    if (counted && !alike) {  // the two lie differently: one by one
      for (uint64_t k = lane; k < n; k += kLanes) one(k);
      continue;
    }
    if (lane < head) one(lane);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t k = lane + u * kLanes;
      if (k >= chunks) break;
      Chunk<T> out;
      T* e = reinterpret_cast<T*>(&out.w);
      if (!counted) {
        out.w = make_uint4(0, 0, 0, 0);
      } else {
        Chunk<T> in;
        in.w = w[u];
        const uint64_t at = head + k * kN;
        if (hit - at < kN) {
#pragma unroll
          for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(value(in.at(i), at + i));
        } else {
#pragma unroll
          for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(-g * __expf(in.at(i) - l));
        }
      }
      st_stream_v4(d + head + k * kN, out.w);
    }
    const uint64_t tail = head + static_cast<uint64_t>(chunks) * kN + lane;
    if (tail < n) one(tail);
  }
  if (!far) return;
  // whole rows, in a loop of their own that leaves the registers of the one above alone
  for (uint64_t b = begin; b < rows * pieces; b += step) {
    const uint64_t t = rows - 1 - b / pieces;
    const int64_t label = labels[t];
    const int32_t p = row_pair[t];
    if (b % pieces || p < 0 || static_cast<uint64_t>(p) >= pairs || !counts(label, vocab) ||
        !is_far(lse[t]))
      continue;
    far_row<T, kLanes>(logits + t * stride, dlogits + t * dstride, vocab,
                       static_cast<uint64_t>(label), row_grad[t] * (dlosses ? dlosses[p] : 1.f), lane);
  }
}

// A warp takes a row (not a block) of at most 4 KB, a few rounds of its loads,
// or of 16 KB where there are enough rows for every warp of the GPU.  Forward
// and backward, by warps and by blocks: 64 rows of 4000 bytes 5.3 and 3.0 us, 5.6
// and 2.3; 64 of 16000 7.2 and 3.0, 5.7 and 3.0; 4096 of 4000 10.1 and 7.1, 22.0 and
// 12.0; 16384 of 16000 58.5 and 77.0, 76.6 and 76.5; 4096 of 64000 56.2 and 76.3, 52.3
// and 76.1.
bool by_warps(uint64_t rows, uint64_t row_bytes) {
  return row_bytes <= 4096 || (row_bytes <= 16384 && rows >= 32ull * sm_count());
}

bool logits_ok(uint64_t pairs, uint64_t rows, uint64_t vocab, const void* logits, int type,
               uint64_t stride) {
  return pairs <= HKV_MAX_BATCH / 2 && rows <= HKV_MAX_BATCH && vocab >= 1 &&
         vocab <= HKV_MAX_BATCH && type_ok(type) && stride >= vocab &&
         (rows == 0 || (logits && aligned(logits, type_size(type))));
}

template <class T>
cudaError_t forward_rows(uint64_t rows, uint64_t vocab, const T* logits, uint64_t stride,
                         const int64_t* labels, float* logps, float* lse, float* row_grad,
                         int32_t* row_pair, cudaStream_t st) {
  const uint64_t sms = sm_count();
  if (by_warps(rows, vocab * sizeof(T)))
    return launch_chained(short_rows_kernel<T>, static_cast<unsigned>((rows + 3) / 4), kWarpThreads,
                          0, st, rows, vocab, logits, stride, labels, logps, lse, row_grad, row_pair);
  // few rows: clusters share them while there is room on the SMs and a part
  // keeps a round of its block's loads
  uint32_t parts = 1;
  while (parts < kMaxParts && rows * parts <= sms &&
         vocab * sizeof(T) >= 2ull * parts * kThreads * unroll(kThreads) * 16)
    parts *= 2;
  if (rows > 0x7FFFFFFFull / parts) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, long_rows_kernel<T>, vocab, logits, stride, parts, labels, logps,
                            lse, row_grad, row_pair);
}

}  // namespace
}  // namespace hkv

extern "C" {

hkv_status hkv_preference_loss(uint64_t pairs, uint64_t rows, uint64_t vocab, const void* logits,
                               int type, uint64_t stride, const int64_t* labels,
                               const int64_t* offsets, const float* ref_logps, float beta,
                               float label_smoothing, int average, float* losses, float* ratios,
                               float* logps, float* lse, float* row_grad, int32_t* row_pair,
                               void* stream) {
  using namespace hkv;
  if (!logits_ok(pairs, rows, vocab, logits, type, stride)) return HKV_ERR_INVALID;
  if (!std::isfinite(beta) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return HKV_ERR_INVALID;
  if (rows && (!labels || !logps || !lse || !row_grad || !row_pair)) return HKV_ERR_INVALID;
  if (pairs && (!offsets || !losses || !ratios)) return HKV_ERR_INVALID;
  if (!aligned(labels, 8) || !aligned(offsets, 8) || !aligned(ref_logps, 4) ||
      !aligned(losses, 4) || !aligned(ratios, 4) || !aligned(logps, 4) || !aligned(lse, 4) ||
      !aligned(row_grad, 4) || !aligned(row_pair, 4))
    return HKV_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (rows)
    e = with_type(type, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      return forward_rows(rows, vocab, static_cast<const T*>(logits), stride, labels, logps, lse,
                          row_grad, row_pair, st);
    });
  if (e == cudaSuccess && pairs)
    e = launch_chained(pair_kernel, static_cast<unsigned>(pairs), kPairThreads, 0, st, pairs, rows,
                       vocab, labels, offsets, ref_logps, beta, label_smoothing, average, losses,
                       ratios, logps, row_grad, row_pair);
  return op_status(e);
}

hkv_status hkv_preference_loss_backward(uint64_t pairs, uint64_t rows, uint64_t vocab,
                                        const void* logits, int type, uint64_t stride,
                                        const int64_t* labels, const float* lse,
                                        const float* row_grad, const int32_t* row_pair,
                                        const float* dlosses, void* dlogits, uint64_t dstride,
                                        void* stream) {
  using namespace hkv;
  if (!logits_ok(pairs, rows, vocab, logits, type, stride) || dstride < vocab)
    return HKV_ERR_INVALID;
  if (rows == 0) return HKV_OK;
  if (!labels || !lse || !row_grad || !row_pair || !dlogits || !aligned(dlogits, type_size(type)))
    return HKV_ERR_INVALID;
  if (dlogits == logits && dstride != stride) return HKV_ERR_INVALID;
  if (!aligned(labels, 8) || !aligned(lse, 4) || !aligned(row_grad, 4) || !aligned(row_pair, 4) ||
      !aligned(dlosses, 4))
    return HKV_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return op_status(with_type(type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const bool warps = by_warps(rows, vocab * sizeof(T));
    const int lanes = warps ? 32 : kThreads;
    const uint64_t piece = static_cast<uint64_t>(lanes) * unroll(lanes) * Chunk<T>::kN;
    const uint64_t pieces = (vocab + piece - 1) / piece;
    const int threads = warps ? kWarpThreads : kThreads;
    const uint64_t blocks = (rows * pieces * lanes + threads - 1) / threads;
    return launch_chained(warps ? backward_kernel<T, 32> : backward_kernel<T, kThreads>,
                          static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF), threads,
                          0, st, pairs, rows, vocab, static_cast<const T*>(logits), stride, pieces,
                          labels, lse, row_grad, row_pair, dlosses, static_cast<T*>(dlogits), dstride);
  }));
}

}  // extern "C"
