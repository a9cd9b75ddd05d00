// clip.cu -- hkv_clip_grad_norm: the norm of many gradients taken as one
// vector, and clipping to it.
//
// Bound by memory: the gradients are read once for the norm and once more,
// and written, where they are clipped.  They are cut into chunks of one size
// that a fixed number of thread blocks share evenly, each a run of
// neighbouring chunks, and every block leaves one partial sum of squares: the
// order of the sum depends on the sizes, on where the tensors start within 32
// bytes, and on the number of SMs, and not on the order in which blocks run.  The
// second kernel adds the
// partials again in every block (a few hundred floats) instead of in a launch
// of its own, and takes each run from its end, where the first kernel left
// off and L2 still holds it.
//
// Times (GB300): the norm of 10^8 float32 in 300 tensors 66 us, 6.0 TB/s; 10^9
// bfloat16 in 400 tensors into float32 1,258 us, 6.4 TB/s of two reads and a
// write, and clipped in place 913 us, 6.6 TB/s; 10^8 float32 in place 185 us; 10^5
// elements in 24 tensors 5.9 us, two launches.  Outs that do not lie as their
// gradients do within 8 elements go one element at a time: the 10^9 into a
// float32 buffer without padding take 3,600 us.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>

#include "operators.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;
constexpr int kPerSm = 4;  // blocks
// groups of eight elements in flight per thread: 128 bytes
template <class T>
constexpr int kUnroll = sizeof(T) == 4 ? 4 : 8;
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
  uint32_t chunk;         // elements of a chunk
};

template <class F>
__device__ __forceinline__ void for_type(uint32_t type, F&& f) {
  if (type == HKV_F32) f(static_cast<float*>(nullptr));
  else if (type == HKV_BF16) f(static_cast<__nv_bfloat16*>(nullptr));
  else f(static_cast<__half*>(nullptr));
}

// The chunks of this block, lo .. hi - 1, by calls of f(entry, first element,
// number of elements); from the last to the first if kBackwards.
template <bool kBackwards, int N, class F>
__device__ __forceinline__ void for_chunks(const Batch<N>& b, F&& f) {
  const uint64_t chunks = b.count ? b.first[b.count] : 0;
  const uint32_t lo = chunks * blockIdx.x / gridDim.x, hi = chunks * (blockIdx.x + 1) / gridDim.x;
  if (lo == hi) return;
  const uint32_t begin = kBackwards ? hi - 1 : lo;
  uint32_t i = 0, end = b.count - 1;
  while (i < end) {  // the entry that holds `begin`
    const uint32_t mid = (i + end + 1) / 2;
    if (b.first[mid] <= begin) i = mid;
    else end = mid - 1;
  }
  for (uint32_t k = 0; k < hi - lo; ++k) {
    const uint32_t c = kBackwards ? hi - 1 - k : lo + k;
    if (kBackwards) {
      while (c < b.first[i]) --i;
    } else {
      while (c >= b.first[i + 1]) ++i;
    }
    const uint64_t n = b.e[i].n_types & ((1ull << 56) - 1);
    const uint64_t at = static_cast<uint64_t>(c - b.first[i]) * b.chunk;
    f(b.e[i], at, static_cast<uint32_t>(min(n - at, static_cast<uint64_t>(b.chunk))));
  }
}

// Elements up to the first place from which both arrays take whole moves of
// eight, or -1 where there is none.
template <class T, class U>
__device__ __forceinline__ int lead(const T* x, const U* y) {
  const uint32_t a = (reinterpret_cast<uintptr_t>(x) / sizeof(T)) & 7;
  const uint32_t b = (reinterpret_cast<uintptr_t>(y) / sizeof(U)) & 7;
  return a == b ? static_cast<int>((8 - a) & 7) : -1;
}

// A sum of many terms: what each addition rounds off is taken into the next.
// Squares of 16-bit numbers have so few digits that the roundings of a plain
// sum lean one way: 4e-6 of 3200 terms, on average over threads.
struct LongSum {
  float s = 0.f, off = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float y = v - off, t = s + y;
    off = fabsf(t) <= FLT_MAX ? (t - s) - y : 0.f;  // infinities stay
    s = t;
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm)
    norm_kernel(const __grid_constant__ Batch<N> b, float* partial, bool more) {
  __shared__ float red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  LongSum s;
  for_chunks<false>(b, [&](const Entry& e, uint64_t at, uint32_t n) {
    for_type(e.n_types >> 56 & 15, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      const T* x = static_cast<const T*>(e.data) + at;
      const uint32_t head = min(static_cast<uint32_t>(lead(x, x)), n);
      if (threadIdx.x < head) {
        const float v = to_f32(x[threadIdx.x]);
        s.add(v * v);
      }
      const uint32_t eights = (n - head) / 8;
      x += head;
      auto add = [&](float (&part)[4], const Eight<T>& in) {
        float v[8];
        in.to(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[i & 3] = fmaf(v[i], v[i], part[i & 3]);
      };
      uint32_t k = threadIdx.x;
      for (; k + (kUnroll<T> - 1) * kThreads < eights; k += kUnroll<T> * kThreads) {
        Eight<T> in[kUnroll<T>];
        float part[4] = {};
#pragma unroll
        for (int u = 0; u < kUnroll<T>; ++u) in[u].load_aligned(x + (k + u * kThreads) * 8, kWhole);
#pragma unroll
        for (int u = 0; u < kUnroll<T>; ++u) add(part, in[u]);
        s.add((part[0] + part[1]) + (part[2] + part[3]));
      }
      for (; k < eights; k += kThreads) {
        Eight<T> in;
        in.load_aligned(x + k * 8, kWhole);
        float part[4] = {};
        add(part, in);
        s.add((part[0] + part[1]) + (part[2] + part[3]));
      }
      const uint32_t tail = eights * 8 + threadIdx.x;
      if (tail < n - head) {
        const float v = to_f32(x[tail]);
        s.add(v * v);
      }
    });
  });
  float sum[1] = {s.s};
  block_sums(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = more ? partial[blockIdx.x] + sum[0] : sum[0];
}

template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm)
    clip_kernel(const __grid_constant__ Batch<N> b, const float* partial, int partials,
                float max_norm, float* norm_out) {
  __shared__ float red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  float sum[1] = {};
  for (int k = threadIdx.x; k < partials; k += kThreads) sum[0] += partial[k];
  block_sums(sum, red);
  const float norm = sqrtf(sum[0]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float f = norm <= max_norm ? 1.f : max_norm / norm;
  for_chunks<true>(b, [&](const Entry& e, uint64_t at, uint32_t n) {
    const uint32_t type = e.n_types >> 56 & 15, out_type = e.n_types >> 60;
    if (!e.out || (f == 1.f && e.out == e.data && type == out_type)) return;
    for_type(type, [&](auto* t) {
      for_type(out_type, [&](auto* u) {
        using T = std::remove_pointer_t<decltype(t)>;
        using U = std::remove_pointer_t<decltype(u)>;
        const T* x = static_cast<const T*>(e.data) + at;
        U* y = static_cast<U*>(e.out) + at;
        const int ahead = lead(x, y);
        const uint32_t head = ahead < 0 ? n : min(static_cast<uint32_t>(ahead), n);
        for (uint32_t k = threadIdx.x; k < head; k += kThreads)
          y[k] = from_f32<U>(to_f32(x[k]) * f);
        const uint32_t eights = (n - head) / 8;
        x += head;
        y += head;
        auto scale = [&](const Eight<T>& in, uint32_t k) {
          float v[8];
          in.to(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= f;
          Eight<U> out;
          out.from(v);
          out.store_aligned(y + k * 8, kWhole);
        };
        uint32_t k = threadIdx.x;
        for (; k + (kUnroll<T> - 1) * kThreads < eights; k += kUnroll<T> * kThreads) {
          Eight<T> in[kUnroll<T>];
#pragma unroll
          for (int q = 0; q < kUnroll<T>; ++q) in[q].load_written(x + (k + q * kThreads) * 8);
#pragma unroll
          for (int q = 0; q < kUnroll<T>; ++q) scale(in[q], k + q * kThreads);
        }
        for (; k < eights; k += kThreads) {
          Eight<T> in;
          in.load_written(x + k * 8);
          scale(in, k);
        }
        const uint32_t tail = eights * 8 + threadIdx.x;
        if (tail < n - head) y[tail] = from_f32<U>(to_f32(x[tail]) * f);
      });
    });
  });
}

// Calls f(batch) for the gradients in runs of at most N.
template <int N, class F>
cudaError_t for_batches(uint64_t count, const hkv_grad* g, uint32_t chunk, F&& f) {
  Batch<N> b{};
  b.chunk = chunk;
  for (uint64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uint64_t chunks = (g[i].n + chunk - 1) / chunk;
    if (b.count == N || b.first[b.count] + chunks > 0x7FFFFFFFull) {
      cudaError_t e = f(b);
      if (e != cudaSuccess) return e;
      b.count = 0;
    }
    b.e[b.count] = {g[i].data, g[i].out,
                    g[i].n | static_cast<uint64_t>(g[i].type) << 56 |
                        static_cast<uint64_t>(g[i].out ? g[i].out_type : 0) << 60};
    b.first[b.count + 1] = b.first[b.count] + static_cast<uint32_t>(chunks);
    ++b.count;
  }
  return f(b);
}

template <int N>
cudaError_t clip(uint64_t count, const hkv_grad* g, uint64_t total, bool writes, float max_norm,
                 float* norm_out, float* work, cudaStream_t st) {
  // every block resident, so that none starts when others end; small totals
  // are cut finer, so that every SM has some.  Chunks of 1024, 4096, 16384 and
  // 65536: 10^5 elements 6.2, 6.1, 6.5 and 7.0 us, 3 * 10^6 13.1, 10.5, 9.9 and 14.0
  // (9.4 by this rule), 10^9 2919, 1412, 1237 and 1232.
  const int grid = std::min(kMaxPartials, sm_count() * kPerSm);
  uint32_t chunk = 4096;
  while (chunk < 16384 && total / chunk > static_cast<uint64_t>(grid)) chunk *= 2;
  auto blocks = [&](const Batch<N>& b) {
    return std::max(1, static_cast<int>(std::min<uint32_t>(grid, b.count ? b.first[b.count] : 0)));
  };
  int partials = 0;
  cudaError_t e = for_batches<N>(count, g, chunk, [&](const Batch<N>& b) {
    // the first launch sets its partials; later ones add to those that are
    // there, so they keep to its number of blocks
    const bool more = partials > 0;
    if (!more) partials = blocks(b);
    return launch_chained(norm_kernel<N>, std::min(partials, blocks(b)), kThreads, 0, st, b, work,
                          more);
  });
  if (e != cudaSuccess) return e;
  if (!writes)
    return launch_chained(clip_kernel<1>, 1, kThreads, 0, st, Batch<1>{}, work, partials, max_norm,
                          norm_out);
  return for_batches<N>(count, g, chunk, [&](const Batch<N>& b) {
    return launch_chained(clip_kernel<N>, blocks(b), kThreads, 0, st, b, work, partials, max_norm,
                          norm_out);
  });
}

// Whether memory that the call writes is written once and read by nothing else:
// blocks take the gradients in no fixed order, so one that is listed twice, or
// lies in another's out, would be scaled once or twice by chance.  Outs that
// follow one another in memory, away from the gradients, are seen in one pass;
// others are sorted.
hkv_status written_once(uint64_t count, const hkv_grad* g) {
  struct Range {
    uintptr_t begin, end;
    bool out;
  };
  auto of = [](const void* p, uint64_t n, int type, bool out) {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(p);
    return Range{begin, begin + n * type_size(type), out};
  };
  auto join = [](Range& all, const Range& r) {
    all.begin = std::min(all.begin, r.begin);
    all.end = std::max(all.end, r.end);
  };
  Range outs{UINTPTR_MAX, 0, true}, data{UINTPTR_MAX, 0, false};
  uint64_t ranges = 0;
  bool ascending = true;
  for (uint64_t i = 0; i < count; ++i) {
    if (!g[i].data || g[i].n == 0) continue;
    if (g[i].out != g[i].data) {
      join(data, of(g[i].data, g[i].n, g[i].type, false));
      ++ranges;
    }
    if (!g[i].out) continue;
    const Range out = of(g[i].out, g[i].n, g[i].out_type, true);
    ascending &= out.begin >= outs.end;
    join(outs, out);
    ++ranges;
  }
  if (ascending && (data.begin >= outs.end || outs.begin >= data.end)) return HKV_OK;
  Range* all = new (std::nothrow) Range[ranges];
  if (!all) return HKV_ERR_OOM;
  uint64_t k = 0;
  for (uint64_t i = 0; i < count; ++i) {
    if (!g[i].data || g[i].n == 0) continue;
    if (g[i].out != g[i].data) all[k++] = of(g[i].data, g[i].n, g[i].type, false);
    if (g[i].out) all[k++] = of(g[i].out, g[i].n, g[i].out_type, true);
  }
  std::sort(all, all + ranges, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t any_end = 0, out_end = 0;
  bool once = true;
  for (k = 0; k < ranges; ++k) {
    once &= all[k].begin >= (all[k].out ? any_end : out_end);
    any_end = std::max(any_end, all[k].end);
    if (all[k].out) out_end = std::max(out_end, all[k].end);
  }
  delete[] all;
  return once ? HKV_OK : HKV_ERR_INVALID;
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
  bool writes = false;
  for (uint64_t i = 0; i < count; ++i) {
    const hkv_grad& g = grads[i];
    if (!type_ok(g.type) || (g.out && !type_ok(g.out_type)) || g.n >= 1ull << 40)
      return HKV_ERR_INVALID;
    if (g.n == 0) continue;
    if (!g.data || !aligned(g.data, type_size(g.type))) return HKV_ERR_INVALID;
    if (g.out && !aligned(g.out, type_size(g.out_type))) return HKV_ERR_INVALID;
    if (g.out == g.data && g.out_type != g.type) return HKV_ERR_INVALID;
    total += g.n;
    writes |= g.out != nullptr;
  }
  if (writes) {
    const hkv_status apart = written_once(count, grads);
    if (apart != HKV_OK) return apart;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* w = static_cast<float*>(work);
  return op_status(
      count <= 64 ? clip<64>(count, grads, total, writes, max_norm, norm_out, w, st)
                  : clip<1024>(count, grads, total, writes, max_norm, norm_out, w, st));
}
