// token_logps.cu -- hkv_token_logps and hkv_token_logps_backward: log
// probabilities of given tokens, the entropy and the largest entries of their
// rows of logits, and the gradient of the first two.
//
// With m the row's maximum, s = sum exp(x - m) and w = sum exp(x - m) (x - m),
//   log p_v = x_v - m - log s     entropy = log s - w / s
// so one pass with a running maximum gives both; when the maximum rises by d,
// w becomes (w - s d) exp(-d) and s becomes s exp(-d).  Rows are taken by a
// warp, a block or a cluster's blocks, as in preference.cu.
#include "logits.cuh"

namespace hkv {
namespace {

// x - max of an entry whose exponential is 0 in any case (-inf, and masks far
// below the maximum): finite, so that its product with 0 is 0.
constexpr float kLeast = -1e30f;
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A running maximum m, s = sum exp(x - m) and w = sum exp(x - m) (x - m).
// Nothing seen, or only -inf: m = -inf, s = w = 0.  A NaN or +inf among the
// values makes s NaN.
struct Moments {
  float m = -INFINITY, s = 0.f, w = 0.f;

  __device__ __forceinline__ void bring(float top) {
    const float d = m - top, f = expf(d);
    w = f > 0.f ? (w + s * d) * f : 0.f;  // d may be -inf where f is 0
    s *= f;
    m = top;
  }
  // Raises the maximum to that of the next values, and returns what to
  // subtract from them (0 while all are -inf).
  __device__ __forceinline__ float raise(float top) {
    if (top > m) bring(top);
    return m == -INFINITY ? 0.f : m;
  }
  __device__ __forceinline__ void add(float x, float base) {
    const float d = max_nan(x - base, kLeast), e = __expf(d);
    s += e;
    w = fmaf(e, d, w);
  }
  __device__ __forceinline__ void one(float x) { add(x, raise(x)); }
  __device__ __forceinline__ void join(Moments o) {
    const float top = fmaxf(m, o.m);
    if (m != top) bring(top);
    if (o.m != top) o.bring(top);
    s += o.s;
    w += o.w;
  }
  __device__ __forceinline__ float entropy() const {
    const float h = logf(s) - w / s;
    return h < 0.f ? 0.f : h;
  }
};

__device__ __forceinline__ Moments join_lanes(Moments r) {
  float top = r.m;
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (r.m != top) r.bring(top);
  for (int o = 16; o > 0; o >>= 1) {
    r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
    r.w += __shfl_xor_sync(0xFFFFFFFFu, r.w, o);
  }
  return r;
}

// One thread's share of a row of n elements, taken by kLanes threads.
template <class T, int kLanes>
__device__ __forceinline__ Moments row_pass(const T* x, uint64_t n, int lane) {
  constexpr int kN = Chunk<T>::kN, kUnroll = unroll(kLanes);
  Moments r;
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
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) r.add(c[u].at(i), base);
  }
  const uint64_t tail = head + chunks * kN + lane;
  if (tail < n) r.one(to_f32(x[tail]));
  return r;
}

// An entry as a whole number: ordered by its logit (-0 as 0), then by the lower
// index.  0 stands for none.
__device__ __forceinline__ uint64_t key_of(float x, uint64_t at) {
  const int32_t b = __float_as_int(x + 0.f);
  const uint32_t order = b < 0 ? ~static_cast<uint32_t>(b) : static_cast<uint32_t>(b) | 0x80000000u;
  return static_cast<uint64_t>(order) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(at));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t order = static_cast<uint32_t>(key >> 32);
  return __int_as_float(static_cast<int32_t>(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order));
}
__device__ __forceinline__ int64_t index_of(uint64_t key) {
  return 0xFFFFFFFFu - static_cast<uint32_t>(key);
}
__device__ __forceinline__ uint64_t largest_of_warp(uint64_t key) {
  for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
  return key;
}

// The largest entry of x[lo .. hi) below `limit` among this thread's.
template <class T, int kLanes>
__device__ __forceinline__ uint64_t largest_below(const T* x, uint64_t lo, uint64_t hi,
                                                  uint64_t limit, int lane) {
  uint64_t best = 0;
  for (uint64_t i = lo + lane; i < hi; i += kLanes) {
    const uint64_t key = key_of(to_f32(x[i]), i);
    if (key < limit) best = max(best, key);
  }
  return best;
}

__device__ __forceinline__ uint64_t remote_u64(uint32_t addr, uint32_t rank) {
  uint32_t far;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(far) : "memory");
  return v;
}

struct Out {
  float *logps, *entropy, *top_logps, *lse;
  int64_t* top_ids;
};

// What a row's sums give.  A row with a NaN, +inf or nothing above -inf has
// NaNs (and no alternatives).
struct Row {
  float lse, rest;
  bool bad;
  __device__ __forceinline__ explicit Row(const Moments& r) {
    lse = Running{r.m, r.s}.log_sum(rest);
    bad = !(r.s > 0.f);
  }
  __device__ __forceinline__ float logp(float x) const { return (x - lse) - rest; }
};

__device__ __forceinline__ void finish_row(const Moments& r, const Row& row, bool has, float chosen,
                                           uint64_t t, const Out& out) {
  if (out.logps) out.logps[t] = row.bad ? NAN : has ? row.logp(chosen) : 0.f;
  out.entropy[t] = row.bad ? NAN : r.entropy();
  if (out.lse) {
    out.lse[2 * t] = row.bad ? NAN : row.lse;
    out.lse[2 * t + 1] = row.rest;
  }
}
__device__ __forceinline__ void no_row(uint64_t t, const Out& out) {
  if (out.logps) out.logps[t] = 0.f;
  out.entropy[t] = 0.f;
  if (out.lse) out.lse[2 * t] = out.lse[2 * t + 1] = 0.f;
}
__device__ __forceinline__ void put_top(uint64_t at, uint64_t key, const Row& row, const Out& out) {
  out.top_ids[at] = row.bad ? -1 : index_of(key);
  out.top_logps[at] = row.bad ? NAN : row.logp(logit_of(key));
}

// A warp per row: short rows.
template <class T>
__global__ void __launch_bounds__(kWarpThreads)
    short_rows_kernel(uint64_t rows, uint64_t vocab, const T* __restrict__ logits, uint64_t stride,
                      const int64_t* __restrict__ labels, uint32_t top, Out out) {
  pdl_trigger();
  pdl_wait();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * (kWarpThreads / 32) + threadIdx.x / 32;
  if (t >= rows) return;
  const uint32_t lane = threadIdx.x & 31;
  const int64_t label = labels ? labels[t] : 0;
  if (!counts(label, vocab)) {
    if (lane == 0) no_row(t, out);
    if (lane < top) {
      out.top_ids[t * top + lane] = -1;
      out.top_logps[t * top + lane] = -INFINITY;
    }
    return;
  }
  const T* x = logits + t * stride;
  const float chosen = to_f32(x[label]);
  const Moments r = join_lanes(row_pass<T, 32>(x, vocab, lane));
  const Row row(r);
  if (lane == 0) finish_row(r, row, true, chosen, t, out);
  uint64_t limit = ~0ull;
  for (uint32_t j = 0; j < top; ++j) {
    limit = largest_of_warp(largest_below<T, 32>(x, 0, vocab, limit, lane));
    if (lane == 0) put_top(t * top + j, limit, row, out);
  }
}

// A block per row, or the `parts` blocks of a cluster.
template <class T>
__global__ void __launch_bounds__(kThreads)
    long_rows_kernel(uint64_t vocab, const T* __restrict__ logits, uint64_t stride, uint32_t parts,
                     const int64_t* __restrict__ labels, uint32_t top, Out out) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float ms[3][kWarps + 1];  // [maximum, sum, weighted sum][warp, then the block]
  __shared__ uint64_t red[2][kWarps];
  __shared__ uint64_t mine[HKV_MAX_TOP], all[HKV_MAX_TOP * kMaxParts];
  pdl_trigger();
  pdl_wait();
  const uint64_t t = blockIdx.x / parts;
  const uint32_t part = blockIdx.x % parts;
  const int64_t label = labels ? labels[t] : 0;
  const bool writes = part == 0 && threadIdx.x == 0;
  if (!counts(label, vocab)) {
    if (writes) no_row(t, out);
    if (part == 0 && threadIdx.x < top) {
      out.top_ids[t * top + threadIdx.x] = -1;
      out.top_logps[t * top + threadIdx.x] = -INFINITY;
    }
    return;  // every block of the cluster
  }
  const T* x = logits + t * stride;
  const float chosen = writes ? to_f32(x[label]) : 0.f;  // on its way while the row is read
  // parts start at multiples of 64 elements of the row
  const uint64_t size = ((vocab + parts - 1) / parts + 63) / 64 * 64;
  const uint64_t lo = min(part * size, vocab), hi = min(lo + size, vocab);
  Moments r = join_lanes(row_pass<T, kThreads>(x + lo, hi - lo, threadIdx.x));
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    ms[0][warp] = r.m;
    ms[1][warp] = r.s;
    ms[2][warp] = r.w;
  }
  __syncthreads();
  if (warp == 0) {
    r = Moments{};
    if (threadIdx.x < kWarps) r = Moments{ms[0][threadIdx.x], ms[1][threadIdx.x], ms[2][threadIdx.x]};
    r = join_lanes(r);
    if (threadIdx.x == 0) {
      ms[0][kWarps] = r.m;
      ms[1][kWarps] = r.s;
      ms[2][kWarps] = r.w;
    }
  }
  uint64_t limit = ~0ull;
  for (uint32_t j = 0; j < top; ++j) {
    const uint64_t best =
        largest_of_warp(largest_below<T, kThreads>(x, lo, hi, limit, threadIdx.x));
    if ((threadIdx.x & 31) == 0) red[j & 1][warp] = best;
    __syncthreads();
    limit = red[j & 1][0];
    for (int i = 1; i < kWarps; ++i) limit = max(limit, red[j & 1][i]);
    if (threadIdx.x == 0) mine[j] = limit;
  }
  __syncthreads();
  if (parts > 1) {
    cluster_sync();
    if (part == 0) {
      r = Moments{ms[0][kWarps], ms[1][kWarps], ms[2][kWarps]};
      for (uint32_t p = 1; p < parts; ++p)
        r.join(Moments{remote_f32(smem_u32(&ms[0][kWarps]), p), remote_f32(smem_u32(&ms[1][kWarps]), p),
                       remote_f32(smem_u32(&ms[2][kWarps]), p)});
      if (threadIdx.x < parts * top)
        all[threadIdx.x] = remote_u64(smem_u32(&mine[threadIdx.x % top]), threadIdx.x / top);
    }
    cluster_sync();  // the others stay until their parts are read
    if (part) return;
    const Row row(r);
    if (writes) finish_row(r, row, true, chosen, t, out);
    if (threadIdx.x < parts * top) {
      const uint64_t key = all[threadIdx.x];
      uint32_t rank = 0;
      for (uint32_t i = 0; i < parts * top; ++i) rank += all[i] > key;
      if (key && rank < top) put_top(t * top + rank, key, row, out);
    }
    return;
  }
  r = Moments{ms[0][kWarps], ms[1][kWarps], ms[2][kWarps]};
  const Row row(r);
  if (writes) finish_row(r, row, true, chosen, t, out);
  if (threadIdx.x < top) put_top(t * top + threadIdx.x, mine[threadIdx.x], row, out);
}

// A piece of a row for every kLanes threads, rows from the last to the first, so
// that what the forward call read last is taken from L2 while it is there.
template <class T, int kLanes>
__global__ void __launch_bounds__(kLanes == 32 ? kWarpThreads : kThreads)
    backward_kernel(uint64_t rows, uint64_t vocab, const T* logits, uint64_t stride, uint64_t pieces,
                    const int64_t* __restrict__ labels, const float* __restrict__ lse,
                    const float* __restrict__ entropy, const float* __restrict__ dlogps,
                    const float* __restrict__ dentropy, T* dlogits, uint64_t dstride) {
  constexpr int kN = Chunk<T>::kN, kUnroll = unroll(kLanes);
  constexpr int kTeams = (kLanes == 32 ? kWarpThreads : kThreads) / kLanes;
  constexpr uint64_t kPiece = kLanes * kUnroll * kN;
  const uint32_t lane = threadIdx.x % kLanes;
  pdl_trigger();
  pdl_wait();
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kTeams;
  const uint64_t begin = static_cast<uint64_t>(blockIdx.x) * kTeams + threadIdx.x / kLanes;
  for (uint64_t b = begin; b < rows * pieces; b += step) {
    const uint64_t t = rows - 1 - b / pieces, lo = b % pieces * kPiece;
    const int64_t label = labels ? labels[t] : -1;
    const bool counted = !labels || counts(label, vocab);
    const float g = counted && dlogps ? dlogps[t] : 0.f;
    const float h = counted && dentropy ? dentropy[t] : 0.f;
    const float l = lse[2 * t], rest = lse[2 * t + 1], ent = entropy[t];
    const uint64_t hit = static_cast<uint64_t>(label) >= lo ? static_cast<uint64_t>(label) - lo : ~0ull;
    const T* x = logits + t * stride + lo;
    T* d = dlogits + t * dstride + lo;
    const uint64_t n = min(vocab - lo, kPiece);
    // p (-g - h (log p + H)), and g (1 - p) - h p (log p + H) for the label
    auto value = [&](float v, uint64_t at) {
      const float lp = (v - l) - rest, p = __expf(lp);
      const float slope = -h * (max_nan(lp, -200.f) + ent);
      return at == hit ? fmaf(p, slope, g * (1.f - p)) : p * (slope - g);
    };
    auto one = [&](uint64_t at) { d[at] = from_f32<T>(counted ? value(to_f32(x[at]), at) : 0.f); };
    const uint32_t head = to_boundary(d, n);
    const bool alike = to_boundary(x, n) == head;
    if (counted && !alike) {  // the two lie differently: one by one
      for (uint64_t k = lane; k < n; k += kLanes) one(k);
      continue;
    }
    const uint32_t chunks = static_cast<uint32_t>((n - head) / kN);
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t k = lane + u * kLanes;
      if (counted && k < chunks) w[u] = __ldcs(reinterpret_cast<const uint4*>(x + head + k * kN));
    }
    if (lane < head) one(lane);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t k = lane + u * kLanes;
      if (k >= chunks) break;
      Chunk<T> o;
      T* e = reinterpret_cast<T*>(&o.w);
      if (!counted) {
        o.w = make_uint4(0, 0, 0, 0);
      } else {
        Chunk<T> in;
        in.w = w[u];
#pragma unroll
        for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(value(in.at(i), head + k * kN + i));
      }
      st_stream_v4(d + head + k * kN, o.w);
    }
    const uint64_t tail = head + static_cast<uint64_t>(chunks) * kN + lane;
    if (tail < n) one(tail);
  }
}

bool logits_ok(uint64_t rows, uint64_t vocab, const void* logits, int type, uint64_t stride) {
  return rows <= HKV_MAX_BATCH && vocab >= 1 && vocab <= HKV_MAX_BATCH && type_ok(type) &&
         stride >= vocab &&
         (rows == 0 || (logits && aligned(logits, type_size(type))));
}

template <class T>
cudaError_t forward_rows(uint64_t rows, uint64_t vocab, const T* logits, uint64_t stride,
                         const int64_t* labels, uint32_t top, const Out& out, cudaStream_t st) {
  const uint64_t sms = sm_count();
  if (by_warps(rows, vocab * sizeof(T)))
    return launch_chained(short_rows_kernel<T>, static_cast<unsigned>((rows + 3) / 4), kWarpThreads,
                          0, st, rows, vocab, logits, stride, labels, top, out);
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
  return cudaLaunchKernelEx(&cfg, long_rows_kernel<T>, vocab, logits, stride, parts, labels, top, out);
}

}  // namespace
}  // namespace hkv

extern "C" {

hkv_status hkv_token_logps(uint64_t rows, uint64_t vocab, const void* logits, int type,
                           uint64_t stride, const int64_t* labels, uint32_t top, float* logps,
                           float* entropy, float* top_logps, int64_t* top_ids, float* lse,
                           void* stream) {
  using namespace hkv;
  if (!logits_ok(rows, vocab, logits, type, stride)) return HKV_ERR_INVALID;
  if (top > HKV_MAX_TOP || top > vocab) return HKV_ERR_INVALID;
  if (rows == 0) return HKV_OK;
  if (!labels != !logps || !entropy || (top && (!top_logps || !top_ids))) return HKV_ERR_INVALID;
  if (!aligned(labels, 8) || !aligned(logps, 4) || !aligned(entropy, 4) || !aligned(top_logps, 4) ||
      !aligned(top_ids, 8) || !aligned(lse, 4))
    return HKV_ERR_INVALID;
  const Out out{logps, entropy, top_logps, lse, top_ids};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return op_status(with_type(type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return forward_rows(rows, vocab, static_cast<const T*>(logits), stride, labels, top, out, st);
  }));
}

hkv_status hkv_token_logps_backward(uint64_t rows, uint64_t vocab, const void* logits, int type,
                                    uint64_t stride, const int64_t* labels, const float* lse,
                                    const float* entropy, const float* dlogps, const float* dentropy,
                                    void* dlogits, uint64_t dstride, void* stream) {
  using namespace hkv;
  if (!logits_ok(rows, vocab, logits, type, stride) || dstride < vocab)
    return HKV_ERR_INVALID;
  if (rows == 0) return HKV_OK;
  if (!lse || !entropy || !dlogits || !aligned(dlogits, type_size(type)) || (dlogps && !labels))
    return HKV_ERR_INVALID;
  if (dlogits == logits && dstride != stride) return HKV_ERR_INVALID;
  if (!aligned(labels, 8) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(dlogps, 4) ||
      !aligned(dentropy, 4))
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
                          0, st, rows, vocab, static_cast<const T*>(logits), stride, pieces, labels,
                          lse, entropy, dlogps, dentropy, static_cast<T*>(dlogits), dstride);
  }));
}

}  // extern "C"
