// clip.cu -- hkv_clip_grad_norm: the norm of many gradients taken as one
// vector, and clipping to it.
//
// The gradients are cut into chunks of one size; a fixed grid of thread
// blocks takes the chunks in turn and leaves one partial sum of squares per
// block, so the sum's order depends on the sizes alone.  The second kernel
// adds the partials again in every block (a few hundred floats) instead of
// in a kernel of its own, and scales.
#include <cmath>

#include "operators.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxPartials = HKV_CLIP_WORK_BYTES / 4;

// One launch's gradients, passed as a kernel argument (no copy to the device
// that a caller's buffer or a graph capture would have to outlive).
struct Entry {
  const void* data;
  void* out;
  uint64_t n_types;  // n | type << 56 | out_type << 60
};
template <int N>
struct Batch {
  Entry e[N];
  uint32_t first[N + 1];  // number of chunks before entry i
  uint32_t count;
  uint64_t chunk;         // elements of a chunk
};

template <int N>
__device__ __forceinline__ uint32_t entry_of(const Batch<N>& b, uint32_t c) {
  uint32_t lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) / 2;
    if (b.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <class F>
__device__ __forceinline__ void for_type(uint32_t type, F&& f) {
  if (type == HKV_F32) f(static_cast<float*>(nullptr));
  else if (type == HKV_BF16) f(static_cast<__nv_bfloat16*>(nullptr));
  else f(static_cast<__half*>(nullptr));
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    norm_kernel(const __grid_constant__ Batch<N> b, float* partial, bool more) {
  __shared__ float red[kThreads / 32];
  float s = 0.f;
  const uint32_t chunks = b.first[b.count];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t i = entry_of(b, c);
    const uint64_t n = b.e[i].n_types & ((1ull << 56) - 1);
    const uint64_t lo = (c - b.first[i]) * b.chunk, hi = min(lo + b.chunk, n);
    for_type(b.e[i].n_types >> 56 & 15, [&](auto* t) {
      const auto* x = static_cast<decltype(t)>(const_cast<void*>(b.e[i].data));
      for (uint64_t k = lo + threadIdx.x; k < hi; k += kThreads) {
        const float v = to_f32(x[k]);
        s = fmaf(v, v, s);
      }
    });
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = more ? partial[blockIdx.x] + s : s;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ Batch<N> b, const float* partial, int partials,
                float max_norm, float* norm_out) {
  __shared__ float red[kThreads / 32];
  float s = 0.f;
  for (int k = threadIdx.x; k < partials; k += kThreads) s += partial[k];
  const float norm = sqrtf(block_sum(s, red));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float f = norm <= max_norm ? 1.f : max_norm / norm;
  const uint32_t chunks = b.count ? b.first[b.count] : 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t i = entry_of(b, c);
    const Entry& e = b.e[i];
    const uint32_t type = e.n_types >> 56 & 15, out_type = e.n_types >> 60;
    if (!e.out || (f == 1.f && e.out == e.data && type == out_type)) continue;
    const uint64_t n = e.n_types & ((1ull << 56) - 1);
    const uint64_t lo = (c - b.first[i]) * b.chunk, hi = min(lo + b.chunk, n);
    for_type(type, [&](auto* t) {
      for_type(out_type, [&](auto* u) {
        const auto* x = static_cast<decltype(t)>(const_cast<void*>(e.data));
        auto* y = static_cast<decltype(u)>(e.out);
        for (uint64_t k = lo + threadIdx.x; k < hi; k += kThreads) {
          const float v = to_f32(x[k]) * f;
          y[k] = from_f32<std::remove_pointer_t<decltype(u)>>(v);
        }
      });
    });
  }
}

template <int N, class F>
cudaError_t for_batches(uint64_t count, const hkv_grad* g, uint64_t chunk, F&& f) {
  Batch<N> b{};
  b.chunk = chunk;
  auto flush = [&](bool last) {
    cudaError_t e = f(b, last);
    b.count = 0;
    b.first[0] = 0;
    return e;
  };
  for (uint64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uint64_t chunks = (g[i].n + chunk - 1) / chunk;
    if (b.count == N || b.first[b.count] + chunks > 0x7FFFFFFFull) {
      cudaError_t e = flush(false);
      if (e != cudaSuccess) return e;
    }
    b.e[b.count] = {g[i].data, g[i].out,
                    g[i].n | static_cast<uint64_t>(g[i].type) << 56 |
                        static_cast<uint64_t>(g[i].out ? g[i].out_type : 0) << 60};
    b.first[b.count + 1] = b.first[b.count] + static_cast<uint32_t>(chunks);
    ++b.count;
  }
  return flush(true);
}

template <int N>
cudaError_t clip(uint64_t count, const hkv_grad* g, uint64_t total, float max_norm,
                 float* norm_out, float* work, cudaStream_t st) {
  const int grid_max = std::min(kMaxPartials, sm_count() * 4);
  uint64_t chunk = 4096;
  while (chunk < 65536 && total / chunk > static_cast<uint64_t>(grid_max) * 4) chunk *= 2;
  bool more = false;
  int partials = 0;
  cudaError_t e = for_batches<N>(count, g, chunk, [&](const Batch<N>& b, bool) {
    if (!more) partials = std::max(1, std::min<int>(grid_max, b.first[b.count]));
    if (b.count == 0 && more) return cudaSuccess;
    norm_kernel<N><<<more ? std::min<int>(partials, b.first[b.count]) : partials, kThreads, 0, st>>>(
        b, work, more);
    more = true;
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  return for_batches<N>(count, g, chunk, [&](const Batch<N>& b, bool) {
    clip_kernel<N><<<std::max(1, std::min<int>(grid_max, b.first[b.count])), kThreads, 0, st>>>(
        b, work, partials, max_norm, norm_out);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace hkv

extern "C" hkv_status hkv_clip_grad_norm(uint64_t count, const hkv_grad* grads, float max_norm,
                                         float* norm_out, void* work, void* stream) {
  using namespace hkv;
  if (count > HKV_MAX_BATCH || (count && !grads) || !norm_out || !work || !(max_norm >= 0.f) ||
      !aligned(norm_out, 4) || !aligned(work, 4))
    return HKV_ERR_INVALID;
  uint64_t total = 0;
  for (uint64_t i = 0; i < count; ++i) {
    const hkv_grad& g = grads[i];
    if (!type_ok(g.type) || (g.out && !type_ok(g.out_type)) || g.n >= 1ull << 40)
      return HKV_ERR_INVALID;
    if (g.n && (!g.data || !aligned(g.data, type_size(g.type)) ||
                (g.out && !aligned(g.out, type_size(g.out_type)))))
      return HKV_ERR_INVALID;
    if (g.n && g.out == g.data && g.out_type != g.type) return HKV_ERR_INVALID;
    total += g.n;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* w = static_cast<float*>(work);
  return op_status(count <= 64 ? clip<64>(count, grads, total, max_norm, norm_out, w, st)
                               : clip<1024>(count, grads, total, max_norm, norm_out, w, st));
}
