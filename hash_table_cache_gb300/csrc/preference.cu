// preference.cu -- hkv_preference_loss and hkv_preference_loss_backward: the
// logistic loss of paired log ratios, from logits, and its gradient.
#include <cmath>

#include "operators.cuh"

namespace hkv {
namespace {

constexpr int kRowThreads = 256;
constexpr int kPairThreads = 512;

// Joins a running maximum and the sum of exp(x - maximum) with another pair.
// An empty or all -inf part has m = -inf and s = 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float a = m == top ? 1.f : __expf(m - top);
  const float b = m2 == top ? 1.f : __expf(m2 - top);
  s = s * a + s2 * b;
  m = top;
}

// A row's log-sum-exp in one pass, and its label's log probability.
template <class T>
__global__ void __launch_bounds__(kRowThreads)
    row_kernel(uint64_t vocab, const T* __restrict__ logits, uint64_t stride,
               const int64_t* __restrict__ labels, float* logps, float* lse, float* row_grad,
               int32_t* row_pair) {
  __shared__ float ms[kRowThreads / 32], ss[kRowThreads / 32];
  const uint64_t t = blockIdx.x;
  const int64_t label = labels[t];
  const bool counted = label >= 0 && static_cast<uint64_t>(label) < vocab;
  if (threadIdx.x == 0) {
    row_grad[t] = 0.f;
    row_pair[t] = -1;
    if (!counted) logps[t] = lse[t] = 0.f;
  }
  if (!counted) return;
  const T* x = logits + t * stride;
  float m = -INFINITY, s = 0.f;
  for (uint64_t v = threadIdx.x; v < vocab; v += kRowThreads) {
    const float f = to_f32(x[v]);
    if (f > m) {
      s *= __expf(m - f);
      m = f;
    }
    if (f != -INFINITY) s += __expf(f - m);
  }
  for (int o = 16; o > 0; o >>= 1)
    join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  if ((threadIdx.x & 31) == 0) {
    ms[threadIdx.x >> 5] = m;
    ss[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kRowThreads / 32; ++w) join(m, s, ms[w], ss[w]);
    const float l = m + logf(s);
    lse[t] = l;
    logps[t] = to_f32(x[label]) - l;
  }
}

// One pair per thread block: the sums of both sequences, the loss, and the
// loss's slope for each of their tokens.
__global__ void __launch_bounds__(kPairThreads)
    pair_kernel(uint64_t pairs, uint64_t rows, uint64_t vocab, const int64_t* __restrict__ labels,
                const int64_t* __restrict__ offsets, const float* __restrict__ ref, float beta,
                float smoothing, int average, float* losses, float* ratios,
                const float* __restrict__ logps, float* row_grad, int32_t* row_pair) {
  __shared__ float red[kPairThreads / 32];
  const uint64_t p = blockIdx.x;
  float r[2], inv[2];
  uint64_t lo[2], hi[2];
  for (int side = 0; side < 2; ++side) {
    const uint64_t s = p + side * pairs;
    const int64_t a = offsets[s], b = offsets[s + 1];
    hi[side] = b <= 0 ? 0 : min(static_cast<uint64_t>(b), rows);
    lo[side] = a <= 0 ? 0 : min(static_cast<uint64_t>(a), rows);
    float sum = 0.f, count = 0.f;
    for (uint64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) {
      const int64_t label = labels[t];
      if (label < 0 || static_cast<uint64_t>(label) >= vocab) continue;
      sum += logps[t] - (ref ? ref[t] : 0.f);
      count += 1.f;
    }
    sum = block_sum(sum, red);
    count = block_sum(count, red);
    inv[side] = average ? (count > 0.f ? 1.f / count : 0.f) : 1.f;
    r[side] = average ? sum * inv[side] : sum;
  }
  const float h = beta * (r[0] - r[1]);
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
  for (int side = 0; side < 2; ++side) {
    const float g = (side ? -slope : slope) * inv[side];
    for (uint64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) {
      const int64_t label = labels[t];
      row_pair[t] = static_cast<int32_t>(p);
      if (label >= 0 && static_cast<uint64_t>(label) < vocab) row_grad[t] = g;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
    backward_kernel(uint64_t pairs, uint64_t vocab, const T* logits, uint64_t stride,
                    const int64_t* __restrict__ labels, const float* __restrict__ lse,
                    const float* __restrict__ row_grad, const int32_t* __restrict__ row_pair,
                    const float* __restrict__ dlosses, T* dlogits, uint64_t dstride) {
  const uint64_t t = blockIdx.x;
  const int64_t label = labels[t];
  const int32_t p = row_pair[t];
  T* d = dlogits + t * dstride;
  if (p < 0 || static_cast<uint64_t>(p) >= pairs || label < 0 ||
      static_cast<uint64_t>(label) >= vocab) {
    for (uint64_t v = threadIdx.x; v < vocab; v += kRowThreads) d[v] = from_f32<T>(0.f);
    return;
  }
  const float g = row_grad[t] * (dlosses ? dlosses[p] : 1.f), l = lse[t];
  const T* x = logits + t * stride;
  for (uint64_t v = threadIdx.x; v < vocab; v += kRowThreads) {
    const float hit = v == static_cast<uint64_t>(label) ? 1.f : 0.f;
    d[v] = from_f32<T>(g * (hit - __expf(to_f32(x[v]) - l)));
  }
}

bool logits_ok(uint64_t pairs, uint64_t rows, uint64_t vocab, const void* logits, int type,
               uint64_t stride) {
  return pairs <= HKV_MAX_BATCH / 2 && rows <= HKV_MAX_BATCH && vocab >= 1 &&
         vocab <= HKV_MAX_BATCH && type_ok(type) && stride >= vocab &&
         (rows == 0 || (logits && aligned(logits, type_size(type))));
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
      row_kernel<<<static_cast<unsigned>(rows), kRowThreads, 0, st>>>(
          vocab, static_cast<decltype(t)>(const_cast<void*>(logits)), stride, labels, logps, lse,
          row_grad, row_pair);
      return cudaGetLastError();
    });
  if (e == cudaSuccess && pairs) {
    pair_kernel<<<static_cast<unsigned>(pairs), kPairThreads, 0, st>>>(
        pairs, rows, vocab, labels, offsets, ref_logps, beta, label_smoothing, average, losses,
        ratios, logps, row_grad, row_pair);
    e = cudaGetLastError();
  }
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
    using P = decltype(t);
    backward_kernel<<<static_cast<unsigned>(rows), kRowThreads, 0, st>>>(
        pairs, vocab, static_cast<P>(const_cast<void*>(logits)), stride, labels, lse, row_grad,
        row_pair, dlosses, static_cast<P>(dlogits), dstride);
    return cudaGetLastError();
  }));
}

}  // extern "C"
