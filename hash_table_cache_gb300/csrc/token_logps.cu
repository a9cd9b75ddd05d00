// token_logps.cu -- hkv_token_logps and hkv_token_logps_backward: log
// probabilities of given tokens, the entropy and the largest entries of their
// rows of logits, and the gradient of the first two.
//
// With m the row's maximum, s = sum exp(x - m) and w = sum exp(x - m) (x - m),
//   log p_v = x_v - m - log s     entropy = log s - w / s
// so one pass with a running maximum gives both; when the maximum rises by d,
// w becomes (w - s d) exp(-d) and s becomes s exp(-d).  Rows are taken by a
// warp, a block or a cluster's blocks, as in preference.cu.
//
// The `top` largest entries come from the same pass.  Lanes of equal number in
// all warps form one of 32 groups; the top-th largest of the groups' maxima is a
// value that at least `top` entries reach, and few more do: 32 log(32 / (32 -
// top)) of a row without order, 31 for 20, about 130 for 32.  Each thread keeps
// the maximum of each of its rounds of loads (a cell: 32 16-bit entries), so that
// only cells that reach the value are read again, and the entries found there are
// ranked by counting.  Rows with too many entries that reach it (ties at a mask)
// are read once more for the groups' largest entries by value and index, and rows
// where that is not enough (entries that repeat with the groups) once for each
// alternative.
//
// Times (GB300, CUDA graph replays): 4096 x 131072 bfloat16, a tenth of the tokens
// hidden, with 20 alternatives 161 us (6.0 TB/s of what is read, 76% of the memory's
// cycles); 4096 x 32768 without 43 us (5.6 TB/s), its gradient 75 us (6.8 TB/s with what
// L2 keeps; both bound by memory); 256 x 50257 10.3 us, with 20 14 to 18 (a row to a block,
// 256 of them on 152 SMs), with 32 22 to 25, with all but 5 entries masked 42, entries that
// repeat with the groups 369; one row of 131072 with 5 7.5 us; 32768 x 2000 37, 79 with 20
// and 46; 4096 x 32768 float32 79, 91 with 20 and 154.  A gradient that lies otherwise
// than its logits within 16 bytes, 4096 x 50257 of 50304 into a contiguous matrix: 200 us
// for 119.  Before: alternatives by a pass each 6205 us for the first of these; powers with
// subnormals 215; 64-bit steps and tests in whole rounds 173.
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

// 2^x, 0 below 2^-126: one instruction, where powers down to 2^-149 take four.  In sums of
// powers whose largest is 1, where neither that nor the power's error of some 2^-22 shows: the
// results for 256 rows of 50257 are off by 5.2e-8 of themselves against 64 bits, for one row of
// 131072 by 1.1e-7 (elementary operations in 32 bits: 6.4e-8 and 8.2e-8).  The same holds
// for __expf, which takes what lies before and behind the whole loads and rows far from 0.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// The clamp that keeps products of 0 and an infinity out of w and out of the gradient:
// masks below it (float16's lowest, for all types) have exponential 0 in any case where
// it is used (a maximum or a log sum within kFactored).
constexpr float kLowest = -65504.f;
template <class T>
__device__ __forceinline__ void clamp(Chunk<T>& c) {
  if constexpr (sizeof(T) == 4) {
    float* e = reinterpret_cast<float*>(&c.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = max_nan(e[i], kLowest);
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __nv_bfloat16>, __nv_bfloat162, __half2>;
    T2* e = reinterpret_cast<T2*>(&c.w);
    T2 least;
    if constexpr (std::is_same_v<T, __nv_bfloat16>) least = __float2bfloat162_rn(kLowest);
    else least = __float2half2_rn(kLowest);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = __hmax2_nan(e[i], least);
  }
}

// 16-byte loads of a round, in flight together.
constexpr int kLoads = 4;

// Cells that a thread keeps at most of a row (a cell is one round of loads or, of
// longer rows, several).
template <class T, int kLanes>
constexpr int cells_of() { return kLanes == 32 ? 4 : 256 / kLoads / static_cast<int>(sizeof(T)); }

// One thread's share of a row of n elements, taken by kLanes threads.  With kTop
// cells[i * kLanes] gets the maximum of its rounds i * per .. (i + 1) * per - 1.
template <class T, int kLanes, bool kTop>
__device__ __forceinline__ Moments row_pass(const T* x, uint64_t n, int lane, T* cells, uint32_t per,
                                            uint32_t count) {
  constexpr int kN = Chunk<T>::kN, kUnroll = kLoads;
  Moments r;
  const uint32_t head = to_boundary(x, n);
  if (lane < static_cast<int>(head)) r.one(to_f32(x[lane]));
  const uint32_t chunks = static_cast<uint32_t>((n - head) / kN);
  const T* from = x + head + static_cast<uint64_t>(lane) * kN;
  float cell = -INFINITY;
  uint32_t in_cell = 0, kept = 0;
  auto round = [&](Chunk<T>(&c)[kUnroll]) {
    const float top = largest(c);
    const float base = r.raise(top);
    if constexpr (kTop) {
      cell = fmaxf(cell, top);
      if (++in_cell == per) {
        cells[kept++ * kLanes] = from_f32<T>(cell);
        cell = -INFINITY;
        in_cell = 0;
      }
    }
    if (fabsf(base) < kFactored) {
      // exp(x - base) as 2^a, a = x log2 e - base log2 e by two multiply-adds.  The
      // same rounded base log2 e is in every a; what it is off by is taken out of
      // the sums.
      const float scaled = base * kLog2e;
      const float off = fmaf(base, kLog2eRest, fmaf(base, kLog2e, -scaled));
      const uint64_t l = both(kLog2e, kLog2e), rest = both(kLog2eRest, kLog2eRest);
      const uint64_t minus = both(-scaled, -scaled);
      uint64_t sum[2] = {}, wsum[2] = {};
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        clamp(c[u]);
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const uint64_t x2 = both(c[u].at(i), c[u].at(i + 1));
          const uint64_t a2 = fma_both(x2, rest, fma_both(x2, l, minus));
          const float2 a = parts(a2);
          const uint64_t e2 = both(exp2_of(a.x), exp2_of(a.y));
          sum[i / 2 & 1] = add_both(sum[i / 2 & 1], e2);
          wsum[i / 2 & 1] = fma_both(e2, a2, wsum[i / 2 & 1]);
        }
      }
      const float2 t = parts(add_both(sum[0], sum[1])), v = parts(add_both(wsum[0], wsum[1]));
      const float back = exp2_of_minus(off), total = t.x + t.y;
      r.s = fmaf(total, back, r.s);
      r.w = fmaf((v.x + v.y) - off * total, back * 0.693147181f, r.w);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i) r.add(c[u].at(i), base);
    }
  };
  uint32_t k = lane;
  for (; k + (kUnroll - 1) * kLanes < chunks; k += kUnroll * kLanes, from += kUnroll * kLanes * kN) {
    Chunk<T> c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) c[u].w = ld_stream_v4(from + u * kLanes * kN);
    round(c);
  }
  if (k < chunks) {
    Chunk<T> c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (k + u * kLanes < chunks) c[u].w = ld_stream_v4(from + u * kLanes * kN);
      else c[u].fill_lowest();
    }
    round(c);
  }
  if constexpr (kTop)
    for (; kept < count; ++kept) {
      cells[kept * kLanes] = from_f32<T>(cell);
      cell = -INFINITY;
    }
  const uint64_t tail = head + static_cast<uint64_t>(chunks) * kN + lane;
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

// The threads of a row or a part of one, and what they share to find its
// largest entries.
template <class T, int kLanes>
struct Team {
  static constexpr int kCells = cells_of<T, kLanes>(), kKeys = kLanes == 32 ? 384 : 512;
  static constexpr int kItems = kLanes == 32 ? 128 : 512;
  uint64_t keys[kKeys];
  uint64_t best[kLanes];
  uint64_t list[HKV_MAX_TOP];  // the result: largest first, 0 where there are no more
  T cells[kCells * kLanes];
  float most[kLanes];
  uint16_t items[kItems];  // cell * kLanes + lane
  uint32_t items_found, keys_found;
  float bound;
  uint64_t limit;

  static __device__ __forceinline__ void sync() {
    if constexpr (kLanes == 32) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ void add(uint64_t key) {
    const uint32_t i = atomicAdd(&keys_found, 1);
    if (i < kKeys) keys[i] = key;
  }
  // Ranks the keys found (which are all different) and keeps the first `top`.
  __device__ __forceinline__ void rank(uint32_t top, uint32_t lane) {
    const uint32_t n = keys_found;
    for (uint32_t i = lane; i < n; i += kLanes) {
      const uint64_t key = keys[i];
      uint32_t above = 0;
      for (uint32_t j = 0; j < n; ++j) above += keys[j] > key;
      if (above < top) list[above] = key;
    }
  }
  // Rounds of loads to a cell, and cells, of n elements from x on.
  static __device__ __forceinline__ void plan(const T* x, uint64_t n, uint32_t& per, uint32_t& count) {
    constexpr uint64_t kRound = kLanes * kLoads;
    const uint64_t chunks = (n - to_boundary(x, n)) / Chunk<T>::kN;
    const uint64_t rounds = (chunks + kRound - 1) / kRound;
    per = 1;
    if (rounds > kCells) per = static_cast<uint32_t>((rounds + kCells - 1) / kCells);
    count = static_cast<uint32_t>(per == 1 ? rounds : (rounds + per - 1) / per);
  }

  // The `top` largest of x[lo .. hi), m being this thread's maximum of them and
  // cells written.  All of the team's threads call it.
  __device__ __forceinline__ void pick(const T* x, uint64_t lo, uint64_t hi, float m, uint32_t per,
                                       uint32_t count, uint32_t top, uint32_t lane) {
    constexpr int kN = Chunk<T>::kN, kUnroll = kLoads;
    most[lane] = m;
    if (lane < HKV_MAX_TOP) list[lane] = 0;
    if (lane == 0) items_found = keys_found = 0;
    sync();
    if (lane < 32) {
      float v = m;
      for (uint32_t i = lane + 32; i < kLanes; i += 32) v = fmaxf(v, most[i]);
      uint32_t above = 0;
      for (int i = 0; i < 32; ++i) above += __shfl_sync(0xFFFFFFFFu, v, i) > v;
      float least = above < top ? v : INFINITY;
      for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
      if (lane == 0) bound = least;
    }
    sync();
    const float b = bound;
    const T* part = x + lo;
    const uint64_t n = hi - lo;
    const uint32_t head = to_boundary(part, n);
    const uint64_t chunks = (n - head) / kN;
    for (uint32_t i = 0; i < count; ++i)
      if (to_f32(cells[i * kLanes + lane]) >= b) {
        const uint32_t at = atomicAdd(&items_found, 1);
        if (at < kItems) items[at] = static_cast<uint16_t>(i * kLanes + lane);
      }
    // what lies before the first and behind the last whole chunk
    if (lane < head && to_f32(part[lane]) >= b) add(key_of(to_f32(part[lane]), lo + lane));
    const uint64_t tail = head + chunks * kN + lane;
    if (tail < n && to_f32(part[tail]) >= b) add(key_of(to_f32(part[tail]), lo + tail));
    sync();
    const uint32_t found = items_found;
    bool done = found <= kItems;
    if (done) {
      const uint32_t each = per * kUnroll;
      for (uint32_t j = lane; j < found * each; j += kLanes) {
        const uint32_t item = items[j / each];
        const uint64_t k = (static_cast<uint64_t>(item / kLanes) * each + j % each) * kLanes + item % kLanes;
        if (k >= chunks) continue;
        Chunk<T> c;
        c.w = ld_nc_v4(part + head + k * kN);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (c.at(i) >= b) add(key_of(c.at(i), lo + head + k * kN + i));
      }
      sync();
      done = keys_found <= kKeys;
    }
    if (!done) {
      done = pick_by_keys(x, lo, hi, top, lane);
      if (!done) {
        pick_each(x, lo, hi, top, lane);
        return;
      }
    }
    rank(top, lane);
    sync();
  }

  // The same with the groups' largest entries by value and index.  False where
  // too many entries are left all the same.
  __device__ __noinline__ bool pick_by_keys(const T* x, uint64_t lo, uint64_t hi, uint32_t top,
                                            uint32_t lane) {
    uint64_t mine = 0;
#pragma unroll 8
    for (uint64_t i = lo + lane; i < hi; i += kLanes) mine = max(mine, key_of(to_f32(x[i]), i));
    best[lane] = mine;
    sync();  // all have read keys_found
    if (lane == 0) keys_found = 0;
    if (lane < 32) {
      for (uint32_t i = lane + 32; i < kLanes; i += 32) mine = max(mine, best[i]);
      uint32_t above = 0;
      for (int i = 0; i < 32; ++i) above += __shfl_sync(0xFFFFFFFFu, mine, i) > mine;
      uint64_t least = above < top ? mine : ~0ull;
      for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
      if (lane == 0) limit = least;
    }
    sync();
    const uint64_t l = limit;
#pragma unroll 8
    for (uint64_t i = lo + lane; i < hi; i += kLanes) {
      const uint64_t key = key_of(to_f32(x[i]), i);
      if (key >= l) add(key);
    }
    sync();
    return keys_found <= kKeys;
  }

  // The largest, the largest below it, and so on.
  __device__ __noinline__ void pick_each(const T* x, uint64_t lo, uint64_t hi, uint32_t top,
                                         uint32_t lane) {
    uint64_t below = ~0ull;
    for (uint32_t j = 0; j < top && below; ++j) {
      uint64_t key = 0;
#pragma unroll 8
      for (uint64_t i = lo + lane; i < hi; i += kLanes) {
        const uint64_t other = key_of(to_f32(x[i]), i);
        if (other < below) key = max(key, other);
      }
      best[lane] = key;
      sync();
      if (lane < 32) {
        for (uint32_t i = lane + 32; i < kLanes; i += 32) key = max(key, best[i]);
        key = largest_of_warp(key);
        if (lane == 0) list[j] = limit = key;
      }
      sync();
      below = limit;
    }
  }
};

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

__device__ __forceinline__ void no_top(uint64_t t, uint32_t top, uint32_t lane, const Out& out) {
  if (lane < top) {
    out.top_ids[t * top + lane] = -1;
    out.top_logps[t * top + lane] = -INFINITY;
  }
}

// A warp per row: short rows.  Ten blocks to an SM: 32768 x 2000 bfloat16 took 35 us, and
// 51 with 5 and 75 with 20 alternatives (37 and 79 on another GPU, for 35 and 75); eight blocks 37, 54 and 83, twelve 34, 56
// and 80.  With eight loads in flight and as many registers as they want it was 44, 75 and 99.
template <class T, bool kTop>
__global__ void __launch_bounds__(kWarpThreads, 10)
    short_rows_kernel(uint64_t rows, uint64_t vocab, const T* __restrict__ logits, uint64_t stride,
                      const int64_t* __restrict__ labels, uint32_t top, Out out) {
  using Warp = Team<T, 32>;
  extern __shared__ uint64_t smem[];
  pdl_trigger();
  pdl_wait();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * (kWarpThreads / 32) + threadIdx.x / 32;
  if (t >= rows) return;
  const uint32_t lane = threadIdx.x & 31;
  const int64_t label = labels ? labels[t] : 0;
  if (!counts(label, vocab)) {
    if (lane == 0) no_row(t, out);
    if (kTop) no_top(t, top, lane, out);
    return;
  }
  const T* x = logits + t * stride;
  const float chosen = to_f32(x[label]);
  Warp* team = reinterpret_cast<Warp*>(smem) + threadIdx.x / 32;
  uint32_t per = 0, count = 0;
  if constexpr (kTop) Warp::plan(x, vocab, per, count);
  const Moments own = row_pass<T, 32, kTop>(x, vocab, lane, kTop ? team->cells + lane : nullptr, per, count);
  const Moments r = join_lanes(own);
  const Row row(r);
  if (lane == 0) finish_row(r, row, true, chosen, t, out);
  if constexpr (kTop) {
    if (!row.bad) team->pick(x, 0, vocab, own.m, per, count, top, lane);
    if (lane < top) put_top(t * top + lane, row.bad ? 0 : team->list[lane], row, out);
  }
}

// A block per row, or the `parts` blocks of a cluster.
template <class T, bool kTop>
__global__ void __launch_bounds__(kThreads, 6)
    long_rows_kernel(uint64_t vocab, const T* __restrict__ logits, uint64_t stride, uint32_t parts,
                     const int64_t* __restrict__ labels, uint32_t top, Out out) {
  constexpr int kWarps = kThreads / 32;
  using Block = Team<T, kThreads>;
  extern __shared__ uint64_t smem[];
  __shared__ float ms[3][kWarps + 1];  // [maximum, sum, weighted sum][warp, then the block]
  Block* team = reinterpret_cast<Block*>(smem);
  pdl_trigger();
  pdl_wait();
  const uint64_t t = blockIdx.x / parts;
  const uint32_t part = blockIdx.x % parts, lane = threadIdx.x;
  const int64_t label = labels ? labels[t] : 0;
  const bool writes = part == 0 && lane == 0;
  if (!counts(label, vocab)) {
    if (writes) no_row(t, out);
    if (kTop && part == 0) no_top(t, top, lane, out);
    return;  // every block of the cluster
  }
  const T* x = logits + t * stride;
  const float chosen = writes ? to_f32(x[label]) : 0.f;  // on its way while the row is read
  // parts start at multiples of 64 elements of the row
  const uint64_t size = ((vocab + parts - 1) / parts + 63) / 64 * 64;
  const uint64_t lo = min(part * size, vocab), hi = min(lo + size, vocab);
  uint32_t per = 0, count = 0;
  if constexpr (kTop) Block::plan(x + lo, hi - lo, per, count);
  Moments r = row_pass<T, kThreads, kTop>(x + lo, hi - lo, lane, kTop ? team->cells + lane : nullptr, per, count);
  const float own = r.m;
  r = join_lanes(r);
  const int warp = lane >> 5;
  if ((lane & 31) == 0) {
    ms[0][warp] = r.m;
    ms[1][warp] = r.s;
    ms[2][warp] = r.w;
  }
  __syncthreads();
  if (warp == 0) {
    r = Moments{};
    if (lane < kWarps) r = Moments{ms[0][lane], ms[1][lane], ms[2][lane]};
    r = join_lanes(r);
    if (lane == 0) {
      ms[0][kWarps] = r.m;
      ms[1][kWarps] = r.s;
      ms[2][kWarps] = r.w;
    }
  }
  if constexpr (kTop) team->pick(x, lo, hi, own, per, count, top, lane);
  if (parts > 1) {
    __syncthreads();
    cluster_sync();
    if (part == 0) {
      r = Moments{ms[0][kWarps], ms[1][kWarps], ms[2][kWarps]};
      for (uint32_t p = 1; p < parts; ++p)
        r.join(Moments{remote_f32(smem_u32(&ms[0][kWarps]), p), remote_f32(smem_u32(&ms[1][kWarps]), p),
                       remote_f32(smem_u32(&ms[2][kWarps]), p)});
      if constexpr (kTop)  // the parts' entries, each where no other thread's is
        if (lane < parts * top) team->keys[lane] = remote_u64(smem_u32(&team->list[lane % top]), lane / top);
    }
    cluster_sync();  // the others stay until their parts are read
    if (part) return;
    const Row row(r);
    if (writes) finish_row(r, row, true, chosen, t, out);
    if constexpr (kTop)
      if (lane < parts * top) {
        const uint64_t key = team->keys[lane];
        uint32_t above = 0;
        for (uint32_t i = 0; i < parts * top; ++i) above += team->keys[i] > key;
        if (row.bad ? lane < top : key && above < top) put_top(t * top + (row.bad ? lane : above), key, row, out);
      }
    return;
  }
  __syncthreads();
  r = Moments{ms[0][kWarps], ms[1][kWarps], ms[2][kWarps]};
  const Row row(r);
  if (writes) finish_row(r, row, true, chosen, t, out);
  if (kTop && lane < top) put_top(t * top + lane, team->list[lane], row, out);
}

// Two neighbouring elements of a chunk.
__device__ __forceinline__ void put_both(float* e, float a, float b) {
  e[0] = a;
  e[1] = b;
}
__device__ __forceinline__ void put_both(__nv_bfloat16* e, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(e) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void put_both(__half* e, float a, float b) {
  *reinterpret_cast<__half2*>(e) = __floats2half2_rn(a, b);
}

// From here on dlogps and dentropy may be too large to meet an exponent before its power.
constexpr float kSteep = 1e30f;

// A piece of a row for every kLanes threads, rows from the last to the first, so
// that what the forward call read last is taken from L2 while it is there.
// kAlike: every row of the gradient lies as the logits' does within 16 bytes.
template <class T, int kLanes, bool kAlike>
__global__ void __launch_bounds__(kLanes == 32 ? kWarpThreads : kThreads, kAlike ? 7 : 5)
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
    // -p g - h p (log p + H), and g (1 - p) - h p (log p + H) for the label; p first, so
    // that no product is larger than the gradient's terms are
    auto value = [&](float v, uint64_t at) {
      const float lp = (v - l) - rest, p = __expf(lp);
      return fmaf(-h, p * (max_nan(lp, -200.f) + ent), at == hit ? g * (1.f - p) : -p * g);
    };
    // The others in pairs: p = 2^(a - off), a = v log2 e - l log2 e by two multiply-adds,
    // off what the rounded l log2 e (the same in every a) and l leave out; then the
    // entry is 2^a (slope a + level).  (a is above -120000, so that the bracket is finite
    // where g and h are below kSteep.)
    const bool factored = fabsf(l) < kFactored && fabsf(g) < kSteep && fabsf(h) < kSteep;
    const float scaled = l * kLog2e;
    const float off = fmaf(rest, kLog2e, fmaf(l, kLog2eRest, fmaf(l, kLog2e, -scaled)));
    const float back = exp2_of_minus(off);
    const uint64_t log2e = both(kLog2e, kLog2e), more = both(kLog2eRest, kLog2eRest), minus = both(-scaled, -scaled);
    const float slope1 = -h * 0.693147181f * back, level1 = (-h * fmaf(off, -0.693147181f, ent) - g) * back;
    const uint64_t slope2 = both(slope1, slope1), level2 = both(level1, level1);
    auto one = [&](uint64_t at) { d[at] = from_f32<T>(counted ? value(to_f32(x[at]), at) : 0.f); };
    const uint32_t head = to_boundary(d, n);
    const uint32_t chunks = static_cast<uint32_t>((n - head) / kN);
    auto emit = [&](uint32_t k, uint4 w) {  // chunk k of the gradient from the logits there
      Chunk<T> o;
      T* e = reinterpret_cast<T*>(&o.w);
      if (!counted) {
        o.w = make_uint4(0, 0, 0, 0);
      } else {
        Chunk<T> in;
        in.w = w;
        if (!factored || hit - (head + k * kN) < kN) {
#pragma unroll
          for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(value(in.at(i), head + k * kN + i));
        } else {
          clamp(in);
#pragma unroll
          for (int i = 0; i < kN; i += 2) {
            const uint64_t x2 = both(in.at(i), in.at(i + 1));
            const uint64_t a2 = fma_both(x2, more, fma_both(x2, log2e, minus));
            const float2 a = parts(a2), m = parts(fma_both(a2, slope2, level2));
            put_both(e + i, exp2_approx(a.x) * m.x, exp2_approx(a.y) * m.y);
          }
        }
      }
      st_stream_v4(d + head + k * kN, o.w);
    };
    if (lane < head) one(lane);
    if (!kAlike && counted) {
      // the two may lie differently: the logits from the pieces of 16 bytes around them,
      // which the next thread reads as well
      const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x + head) & 15);
      const uint4* const from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x + head) - off);
#pragma unroll 1
      for (uint32_t k = lane; k < chunks; k += kLanes) {
        const uint4 lo = from[k], hi = off ? from[k + 1] : lo;
        uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        shift_bytes(v, off);
        emit(k, make_uint4(v[0], v[1], v[2], v[3]));
      }
    } else {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t k = lane + u * kLanes;
        if (counted && k < chunks) w[u] = __ldcs(reinterpret_cast<const uint4*>(x + head + k * kN));
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t k = lane + u * kLanes;
        if (k >= chunks) break;
        emit(k, w[u]);
      }
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
    return launch_chained(top ? short_rows_kernel<T, true> : short_rows_kernel<T, false>,
                          static_cast<unsigned>((rows + 3) / 4), kWarpThreads,
                          top ? kWarpThreads / 32 * sizeof(Team<T, 32>) : 0, st, rows, vocab, logits,
                          stride, labels, top, out);
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
  cfg.dynamicSmemBytes = top ? sizeof(Team<T, kThreads>) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, top ? long_rows_kernel<T, true> : long_rows_kernel<T, false>, vocab, logits, stride, parts, labels, top, out);
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
  const Matrix from{logits, rows, vocab, stride, type_size(type)}, to{dlogits, rows, vocab, dstride, type_size(type)};
  if (meet(to, from) && !(dlogits == logits && dstride == stride)) return HKV_ERR_INVALID;
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
    const bool alike = (reinterpret_cast<uintptr_t>(dlogits) - reinterpret_cast<uintptr_t>(logits)) % 16 == 0 &&
                       (dstride - stride) * sizeof(T) % 16 == 0;
    return launch_chained(alike ? warps ? backward_kernel<T, 32, true> : backward_kernel<T, kThreads, true>
                                : warps ? backward_kernel<T, 32, false> : backward_kernel<T, kThreads, false>,
                          static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF), threads,
                          0, st, rows, vocab, static_cast<const T*>(logits), stride, pieces, labels,
                          lse, entropy, dlogps, dentropy, static_cast<T*>(dlogits), dstride);
  }));
}

}  // extern "C"
