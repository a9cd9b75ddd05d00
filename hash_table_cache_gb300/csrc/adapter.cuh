// adapter.cuh -- the kernels of hkv_adapter_matmul and its backward pass: low-rank
// adapters of many requests beside a shared projection.
//
// A request s is the rows offsets[s] .. offsets[s + 1] - 1 of the batch and has
// the adapter a = which[s], two thin matrices D (rank x k) and U (n x rank) and a
// scale c:
//   h = D x,  y = base + c U h            dh = c U^T dy,  dx = base + D^T dh
//   dD = sum_t dh_t x_t^T                 dU = sum_t c dy_t h_t^T
// Both chains are one kernel: a tile of rows of one request is multiplied by the
// first factor along its whole length, which the blocks of a cluster share and
// join through distributed shared memory in a fixed order, and the tile's rank
// numbers a row, which never leave the SM, go through the second factor, whose
// columns the same blocks share.
//
// The products are thin: 2 rank operations for each element that is read or
// written, 16 to 128 where the tensor cores could take 280 and more, so memory is
// the bound and mma.sync, which takes ragged tiles, either order of either factor
// and sums in registers, is enough.  It multiplies bfloat16 (float16 in the first
// product of float16 matrices); what has more digits is split into two or three
// bfloat16 numbers (planes), whose products are added in float32:
//   float32 = three planes exactly, products of planes i + j <= 2 (what is left
//   out is below 2^-23 of a term); float16 = two planes exactly; the float32 h and
//   dh in two planes where matrices have 16 bits (2^-16 of it is left out, where
//   the result is rounded to 2^-8 or 2^-11), in three where they have 32.
#pragma once

#include <type_traits>

#include "operators.cuh"

namespace hkv {

constexpr int kAdapterThreads = 256;
constexpr int kAdapterParts = 8;  // blocks of a cluster at most

// Planes of the first product's operands, of the second factor, and of h.
template <class T>
struct Planes {
  static constexpr int kIn = sizeof(T) == 4 ? 3 : 1;
  static constexpr int kW = sizeof(T) == 4 ? 3 : std::is_same_v<T, __half> ? 2 : 1;
  static constexpr int kP = sizeof(T) == 4 ? 3 : 2;
  // Whether the product of planes i and j is taken.
  static __device__ __forceinline__ constexpr bool takes(int i, int j) {
    return sizeof(T) != 4 || i + j <= 2;
  }
};

// What the requests are, as the kernels take it.
struct Requests {
  uint64_t tokens, requests, adapters;
  const int64_t *offsets, *which;
  const float* scales;
  // First row of segment s: the rows before the first request are segment 0, the
  // requests 1 .. requests, the rows behind the last one requests + 1.
  __device__ __forceinline__ uint64_t start(uint64_t s) const {
    if (s == 0) return 0;
    if (s > requests + 1) return tokens;
    if (!offsets) return 0;
    const int64_t v = offsets[s - 1];
    return v <= 0 ? 0 : min(static_cast<uint64_t>(v), tokens);
  }
  __device__ __forceinline__ int64_t adapter(uint64_t s) const {
    if (s == 0 || s > requests) return -1;
    const int64_t a = which[s - 1];
    return a >= 0 && static_cast<uint64_t>(a) < adapters ? a : -1;
  }
};

// Tiles of kTile rows: segment s has the slots start(s) / kTile + s up to
// start(s + 1) / kTile + s + 1, at least as many as it has tiles, so that a block
// finds its rows by one search and no list of tiles has to be made.
template <int kTile>
__device__ __forceinline__ uint64_t find_segment(const Requests& q, uint64_t slot) {
  const uint32_t lane = threadIdx.x & 31;
  uint64_t lo = 0, hi = q.requests + 2;
  while (hi - lo > 1) {  // every turn leaves a thirty-second part
    const uint64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool before = at < hi && q.start(at) / kTile + at <= slot;
    const uint64_t n = __popc(__ballot_sync(0xFFFFFFFFu, before));
    lo += n * step;
    hi = min(lo + step, hi);
  }
  return lo;
}
inline uint64_t slots_of(uint64_t tokens, uint64_t requests, int tile) {
  return tokens / tile + requests + 2;
}

// Eight neighbouring elements as they lie in memory, the first `n` of them.
template <class T>
struct Raw {
  static constexpr int kVecs = sizeof(T) / 2;
  uint4 v[kVecs];
  // kWritten: of memory that the kernel may also write (by the same thread, later).
  template <bool kWritten = false>
  __device__ __forceinline__ void load(const T* p, int64_t n, bool whole) {
    if (n >= 8 && whole) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if constexpr (kWritten)
          asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                       : "l"(p + i * (16 / sizeof(T)))
                       : "memory");
        else
          v[i] = ld_nc_v4(p + i * (16 / sizeof(T)));
    } else {
      T* e = reinterpret_cast<T*>(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void store(T* p, int64_t n, bool whole) const {
    if (n >= 8 && whole) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) st_stream_v4(p + i * (16 / sizeof(T)), v[i]);
    } else {
      const T* e = reinterpret_cast<const T*>(v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = e[i];
    }
  }
  __device__ __forceinline__ float at(int i) const { return to_f32(reinterpret_cast<const T*>(v)[i]); }
};

// Two floats as kN planes of two bfloat16 each: all but the last cut off, which
// leaves an exact rest, the last rounded.
template <int kN>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&out)[kN]) {
#pragma unroll
  for (int p = 0; p + 1 < kN; ++p) {
    out[p] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
    b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
  }
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  out[kN - 1] = *reinterpret_cast<const uint32_t*>(&r);
}
// Eight elements as planes of eight; one plane is the 16-bit elements as they are.
template <class T, int kN>
__device__ __forceinline__ void split(const Raw<T>& r, uint4 (&out)[kN]) {
  if constexpr (kN == 1) {
    out[0] = r.v[0];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t pair[kN];
      split_pair<kN>(r.at(2 * i), r.at(2 * i + 1), pair);
#pragma unroll
      for (int p = 0; p < kN; ++p) w[4 * p + i] = pair[p];
    }
  }
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The cluster's barrier, for warps whose threads may have parted.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  cluster_sync();
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 operator+(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// A factor of the adapters: adapter a's row r starts a * step + r * stride
// elements in.  whole: rows of eight elements may be taken by 16-byte loads.
template <class T>
struct Factor {
  const T* data;
  uint64_t step, stride;
  bool whole;
};

template <class T>
struct Chain {
  Requests q;
  uint64_t in, out;  // columns of the matrix read and of the one written
  uint32_t rank;
  const T* x;        // tokens x in
  uint64_t x_stride;
  Factor<T> first, second;
  const T* base;     // tokens x out, or null
  uint64_t base_stride;
  T* y;
  uint64_t y_stride;
  float* hidden;     // tokens x rank, or null
  uint32_t parts, groups;  // blocks of a cluster, and clusters that share a tile's columns
  uint64_t part_in, part_out;  // columns of x to a block, columns of y to a block
  bool x_whole, base_whole, y_whole;
};

// Shared memory of a chain, in bytes.
template <class T, int kRank, int kTile, bool kBack>
struct ChainShape {
  using P = Planes<T>;
  static constexpr int kRowWarps = kTile / 16, kOther = 8 / kRowWarps;
  static constexpr int kStep = kTile == 64 ? 64 : 128;   // columns of x to a stage
  static constexpr int kCols = kOther * (kTile == 64 ? 64 : 32);  // columns of y to a step
  static constexpr int kInPitch = kStep + 8, kRankPitch = kRank + 8, kColPitch = kCols + 8;
  static constexpr int kX = P::kIn * kTile * kInPitch * 2;
  static constexpr int kFirst = P::kIn * (kBack ? kStep * kRankPitch : kRank * kInPitch) * 2;
  static constexpr int kStage = kX + kFirst;
  static constexpr int kSecond = P::kW * (kBack ? kRank * kColPitch : kCols * kRankPitch) * 2;
  static constexpr int kSums = kOther * kTile * kRank * 4;
  static constexpr int most(int a, int b) { return a > b ? a : b; }
  static constexpr int kWork = most(most(2 * kStage, 2 * kSecond), kSums);
  // this block's part of the sums.  A few are read from all parts by every block;
  // many are shared out first, and their planes take this part's place.
  static constexpr bool kDirect = kTile * kRank <= 1024;
  static constexpr int kOwn = kTile * kRank * 4;
  static constexpr int kPlanes = P::kP * kTile * kRankPitch * 2;
  static constexpr int kPlanesAt = kWork + (kDirect ? kOwn : 0);
  static constexpr int kShareAt = kWork + most(kOwn, kPlanes);
  static constexpr int kBytes = kDirect ? kPlanesAt + kPlanes : kShareAt + kOwn / 2;
};

// Where column c of 32 stands in shared memory, so that the tensor core's result
// gives a thread eight neighbouring columns.
__device__ __forceinline__ int place(int c) { return (c >> 1 & 3) * 8 + (c >> 3 & 3) * 2 + (c & 1); }

template <class T, int kRank, int kTile, bool kBack>
__global__ void __launch_bounds__(kAdapterThreads)
    chain_kernel(const __grid_constant__ Chain<T> a) {
  using S = ChainShape<T, kRank, kTile, kBack>;
  using P = Planes<T>;
  constexpr int kThreads = kAdapterThreads;
  constexpr bool kF16 = std::is_same_v<T, __half>;
  constexpr int kXLoads = (kTile * S::kStep / 8 + kThreads - 1) / kThreads;
  constexpr int kFirstChunks = kRank * S::kStep / 8, kFirstLoads = (kFirstChunks + kThreads - 1) / kThreads;
  constexpr int kSecondChunks = kRank * S::kCols / 8, kSecondLoads = (kSecondChunks + kThreads - 1) / kThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const sums = reinterpret_cast<float*>(smem);             // [other][tile][rank]
  float* const own = reinterpret_cast<float*>(smem + S::kWork);   // [tile][rank]
  float* const share = reinterpret_cast<float*>(smem + S::kShareAt);
  uint8_t* const planes = smem + S::kPlanesAt;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t row_warp = warp % S::kRowWarps, other = warp / S::kRowWarps;
  pdl_trigger();
  pdl_wait();

  const uint32_t part = blockIdx.x % a.parts;
  const uint32_t group = blockIdx.x / a.parts % a.groups;
  const uint64_t slot = blockIdx.x / a.parts / a.groups;
  const uint64_t seg = find_segment<kTile>(a.q, slot);
  const uint64_t seg_start = a.q.start(seg), seg_end = a.q.start(seg + 1);
  const uint64_t row0 = seg_start + (slot - (seg_start / kTile + seg)) * kTile;
  if (row0 >= seg_end) return;  // the cluster's other blocks as well
  const int rows = static_cast<int>(min(seg_end - row0, static_cast<uint64_t>(kTile)));
  const int64_t adapter = a.q.adapter(seg);
  const uint64_t col0 = (static_cast<uint64_t>(group) * a.parts + part) * a.part_out;
  const uint64_t col1 = min(col0 + a.part_out, a.out);

  if (adapter < 0) {  // base as it is
    if (a.hidden && group == 0 && part == 0)
      for (uint64_t i = tid; i < rows * static_cast<uint64_t>(a.rank); i += kThreads) a.hidden[row0 * a.rank + i] = 0.f;
    if (a.y == a.base || col0 >= col1) return;
    const uint64_t eights = (col1 - col0 + 7) / 8;
    for (uint64_t i = tid; i < rows * eights; i += kThreads) {
      const uint64_t row = row0 + i / eights, col = col0 + i % eights * 8;
      const int64_t n = col1 - col;
      Raw<T> r;
      r.template load<true>(a.base + row * a.base_stride + col, a.base ? n : 0, a.base_whole);
      r.store(a.y + row * a.y_stride + col, n, a.y_whole);
    }
    return;
  }
  const T* const first = a.first.data + adapter * a.first.step;
  const T* const second = a.second.data + adapter * a.second.step;
  const float scale = a.q.scales ? a.q.scales[adapter] : 1.f;

  // ---- the first product: this block's part of the columns of x
  const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
  Raw<T> x_raw[kXLoads], first_raw[kFirstLoads], second_raw[kSecondLoads];
  auto load_stage = [&](uint64_t k) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int at = tid + i * kThreads, row = at / (S::kStep / 8);
      const uint64_t col = k + at % (S::kStep / 8) * 8;
      x_raw[i].load(a.x + (row0 + row) * a.x_stride + col, row < rows ? static_cast<int64_t>(in1 - col) : 0, a.x_whole);
    }
#pragma unroll
    for (int i = 0; i < kFirstLoads; ++i) {
      const int at = tid + i * kThreads;
      if (kFirstChunks % kThreads && at >= kFirstChunks) break;
      if constexpr (kBack) {
        const uint64_t row = k + at / (kRank / 8);
        const int col = at % (kRank / 8) * 8;
        first_raw[i].load(first + row * a.first.stride + col, row < in1 ? static_cast<int64_t>(a.rank) - col : 0, a.first.whole);
      } else {
        const uint32_t row = at / (S::kStep / 8);
        const uint64_t col = k + at % (S::kStep / 8) * 8;
        first_raw[i].load(first + row * a.first.stride + col, row < a.rank ? static_cast<int64_t>(in1 - col) : 0, a.first.whole);
      }
    }
  };
  auto store_stage = [&](int buffer) {
    uint8_t* const to = smem + buffer * S::kStage;
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int at = tid + i * kThreads, row = at / (S::kStep / 8), col = at % (S::kStep / 8) * 8;
      uint4 v[P::kIn];
      split<T, P::kIn>(x_raw[i], v);
#pragma unroll
      for (int p = 0; p < P::kIn; ++p)
        *reinterpret_cast<uint4*>(to + ((p * kTile + row) * S::kInPitch + col) * 2) = v[p];
    }
#pragma unroll
    for (int i = 0; i < kFirstLoads; ++i) {
      const int at = tid + i * kThreads;
      if (kFirstChunks % kThreads && at >= kFirstChunks) break;
      constexpr int kPer = (kBack ? kRank : S::kStep) / 8, kRows = kBack ? S::kStep : kRank;
      constexpr int kPitch = kBack ? S::kRankPitch : S::kInPitch;
      const int row = at / kPer, col = at % kPer * 8;
      uint4 v[P::kIn];
      split<T, P::kIn>(first_raw[i], v);
#pragma unroll
      for (int p = 0; p < P::kIn; ++p)
        *reinterpret_cast<uint4*>(to + S::kX + ((p * kRows + row) * kPitch + col) * 2) = v[p];
    }
  };
  // the second factor's first columns are on their way while the sums are joined
  auto load_second = [&](uint64_t c) {
#pragma unroll
    for (int i = 0; i < kSecondLoads; ++i) {
      const int at = tid + i * kThreads;
      if (kSecondChunks % kThreads && at >= kSecondChunks) break;
      if constexpr (kBack) {
        const uint32_t row = at / (S::kCols / 8);
        const uint64_t col = c + at % (S::kCols / 8) * 8;
        second_raw[i].load(second + row * a.second.stride + col, row < a.rank ? static_cast<int64_t>(col1 - col) : 0, a.second.whole);
      } else {
        const uint64_t row = c + at / (kRank / 8);
        const int col = at % (kRank / 8) * 8;
        second_raw[i].load(second + row * a.second.stride + col, row < col1 ? static_cast<int64_t>(a.rank) - col : 0, a.second.whole);
      }
    }
  };
  auto store_second = [&](int buffer) {
    uint8_t* const to = smem + buffer * S::kSecond;
#pragma unroll
    for (int i = 0; i < kSecondLoads; ++i) {
      const int at = tid + i * kThreads;
      if (kSecondChunks % kThreads && at >= kSecondChunks) break;
      uint4 v[P::kW];
      split<T, P::kW>(second_raw[i], v);
      if constexpr (kBack) {
        const int row = at / (S::kCols / 8), col = at % (S::kCols / 8) * 8;
#pragma unroll
        for (int p = 0; p < P::kW; ++p) {
          uint8_t* const r = to + (p * kRank + row) * S::kColPitch * 2;
          const uint32_t* const w = reinterpret_cast<const uint32_t*>(&v[p]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint32_t*>(r + ((col & ~31) + place((col & 31) + 2 * j)) * 2) = w[j];
        }
      } else {
        const int row = at / (kRank / 8), col = at % (kRank / 8) * 8;
        const int placed = (row & ~31) + place(row & 31);
#pragma unroll
        for (int p = 0; p < P::kW; ++p)
          *reinterpret_cast<uint4*>(to + ((p * S::kCols + placed) * S::kRankPitch + col) * 2) = v[p];
      }
    }
  };

  float acc[kRank / 8][4] = {};
  const int steps = static_cast<int>((in1 - in0 + S::kStep - 1) / S::kStep);
  if (steps) {
    load_stage(in0);
    store_stage(0);
    __syncthreads();
  }
  for (int step = 0; step < steps; ++step) {
    if (step + 1 < steps) load_stage(in0 + static_cast<uint64_t>(step + 1) * S::kStep);
    const uint32_t xs = smem_u32(smem) + (step & 1) * S::kStage, ws = xs + S::kX;
    // sums of 32 bits in the tensor core are cut, not rounded: short chains, added
    // up by rounding additions, where the result has 32 bits
    float chain[kRank / 8][4] = {};
    constexpr bool kShort = sizeof(T) == 4;
    constexpr int kEach = S::kStep / 16 / S::kOther;
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
      const int k = (other * kEach + s) * 16;
      uint32_t xa[P::kIn][4];
#pragma unroll
      for (int p = 0; p < P::kIn; ++p)
        ldsm(xa[p], xs + ((p * kTile + row_warp * 16 + lane % 16) * S::kInPitch + k + lane / 16 * 8) * 2);
#pragma unroll
      for (int n = 0; n < kRank / 16; ++n)
#pragma unroll
        for (int j = 0; j < P::kIn; ++j) {
          uint32_t w[4];
          if constexpr (kBack)
            ldsm_t(w, ws + ((j * S::kStep + k + lane % 16) * S::kRankPitch + n * 16 + lane / 16 * 8) * 2);
          else
            ldsm(w, ws + ((j * kRank + n * 16 + lane % 8 + lane / 16 * 8) * S::kInPitch + k + lane / 8 % 2 * 8) * 2);
#pragma unroll
          for (int i = 0; i < P::kIn; ++i)
            if (P::takes(i, j)) {
              mma<kF16>(kShort ? chain[2 * n] : acc[2 * n], xa[i], w[0], w[1]);
              mma<kF16>(kShort ? chain[2 * n + 1] : acc[2 * n + 1], xa[i], w[2], w[3]);
            }
        }
    }
    if constexpr (kShort) {
#pragma unroll
      for (int n = 0; n < kRank / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += chain[n][i];
    }
    if (step + 1 < steps) store_stage((step + 1) & 1);
    __syncthreads();
  }
  const bool writes = col0 < col1;
  if (writes) load_second(col0);

  // ---- the warps' sums, then the blocks'
  {
    float* const to = sums + (other * kTile + row_warp * 16 + lane / 4) * kRank + lane % 4 * 2;
#pragma unroll
    for (int n = 0; n < kRank / 8; ++n) {
      *reinterpret_cast<float2*>(to + n * 8) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(to + 8 * kRank + n * 8) = make_float2(acc[n][2], acc[n][3]);
    }
  }
  __syncthreads();
  constexpr int kQuads = kTile * kRank / 4;
  for (int i = tid; i < kQuads; i += kThreads) {
    float4 v = reinterpret_cast<const float4*>(sums)[i];
#pragma unroll
    for (int o = 1; o < S::kOther; ++o) v = v + reinterpret_cast<const float4*>(sums)[o * kQuads + i];
    reinterpret_cast<float4*>(own)[i] = v;
  }
  const uint32_t used = static_cast<uint32_t>((a.in + a.part_in - 1) / a.part_in);  // parts with columns
  auto joined = [&](int i) {
    float4 v = remote_f32x4(smem_u32(own) + i * 16, 0);
    for (uint32_t p = 1; p < used; ++p) v = v + remote_f32x4(smem_u32(own) + i * 16, p);
    return v;
  };
  auto put = [&](int i, float4 v, bool keeps) {
    const int row = i * 4 / kRank, col = i * 4 % kRank;
    float e[4] = {v.x, v.y, v.z, v.w};
    if (kBack)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] *= scale;
    if (keeps && row < rows)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < static_cast<int>(a.rank)) a.hidden[(row0 + row) * a.rank + col + j] = e[j];
    if (!kBack)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] *= scale;
    uint32_t lo[P::kP], hi[P::kP];
    split_pair<P::kP>(e[0], e[1], lo);
    split_pair<P::kP>(e[2], e[3], hi);
#pragma unroll
    for (int p = 0; p < P::kP; ++p)
      *reinterpret_cast<uint2*>(planes + ((p * kTile + row) * S::kRankPitch + col) * 2) = make_uint2(lo[p], hi[p]);
  };
  const bool keeps = a.hidden && group == 0;
  constexpr int kPuts = (kQuads + kThreads - 1) / kThreads;
  if (a.parts == 1) {
    float4 v[kPuts];  // out of the planes' way
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPuts; ++j)
      if (kQuads % kThreads == 0 || tid + j * kThreads < kQuads) v[j] = reinterpret_cast<const float4*>(own)[tid + j * kThreads];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPuts; ++j)
      if (kQuads % kThreads == 0 || tid + j * kThreads < kQuads) put(tid + j * kThreads, v[j], keeps);
  } else if constexpr (S::kDirect) {
    cluster_meet();
    for (int i = tid; i < kQuads; i += kThreads) put(i, joined(i), keeps && part == 0);
    cluster_arrive();
  } else {
    cluster_meet();
    const int each = kQuads / a.parts;
    for (int i = tid; i < each; i += kThreads) reinterpret_cast<float4*>(share)[i] = joined(part * each + i);
    cluster_meet();
    for (int i = tid; i < kQuads; i += kThreads)
      put(i, remote_f32x4(smem_u32(share) + i % each * 16, i / each), keeps && part == static_cast<uint32_t>(i / each));
    cluster_arrive();
  }
  // (the work space has been read: the barriers above)
  // ---- the second product: this block's columns of y
  const int col_steps = writes ? static_cast<int>((col1 - col0 + S::kCols - 1) / S::kCols) : 0;
  if (col_steps) store_second(0);
  __syncthreads();
  constexpr int kSets = S::kCols / 32 / S::kOther;  // of 32 columns, to a warp
  const uint32_t quad = lane % 4;
  for (int step = 0; step < col_steps; ++step) {
    const uint64_t c0 = col0 + static_cast<uint64_t>(step) * S::kCols;
    Raw<T> base[kSets][2];
#pragma unroll
    for (int set = 0; set < kSets; ++set)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = row_warp * 16 + lane / 4 + half * 8;
        const uint64_t col = c0 + (other * kSets + set) * 32 + quad * 8;
        base[set][half].template load<true>(a.base + (row0 + row) * a.base_stride + col,
                                            a.base && row < rows ? static_cast<int64_t>(col1 - col) : 0, a.base_whole);
      }
    if (step + 1 < col_steps) load_second(c0 + S::kCols);
    const uint32_t ps = smem_u32(planes), ws = smem_u32(smem) + (step & 1) * S::kSecond;
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
      const int c = (other * kSets + set) * 32;
      float d[4][4] = {};
#pragma unroll
      for (int k = 0; k < kRank; k += 16) {
        uint32_t h[P::kP][4];
#pragma unroll
        for (int p = 0; p < P::kP; ++p)
          ldsm(h[p], ps + ((p * kTile + row_warp * 16 + lane % 16) * S::kRankPitch + k + lane / 16 * 8) * 2);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < P::kW; ++j) {
            uint32_t w[4];
            if constexpr (kBack)
              ldsm_t(w, ws + ((j * kRank + k + lane % 16) * S::kColPitch + c + n * 16 + lane / 16 * 8) * 2);
            else
              ldsm(w, ws + ((j * S::kCols + c + n * 16 + lane % 8 + lane / 16 * 8) * S::kRankPitch + k + lane / 8 % 2 * 8) * 2);
#pragma unroll
            for (int i = 0; i < P::kP; ++i)
              if (P::takes(i, j)) {
                mma<false>(d[2 * n], h[i], w[0], w[1]);
                mma<false>(d[2 * n + 1], h[i], w[2], w[3]);
              }
          }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = row_warp * 16 + lane / 4 + half * 8;
        const uint64_t col = c0 + c + quad * 8;
        const int64_t n = row < rows ? static_cast<int64_t>(col1 - col) : 0;
        Raw<T> r;
        T* const e = reinterpret_cast<T*>(r.v);
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = from_f32<T>(base[set][half].at(j) + d[j / 2][half * 2 + j % 2]);
        r.store(a.y + (row0 + row) * a.y_stride + col, n, a.y_whole);
      }
    }
    if (step + 1 < col_steps) store_second((step + 1) & 1);
    __syncthreads();
  }
  if (a.parts > 1) cluster_wait();  // the others have read this block's sums
}

// ---------------------------------------------------------------------------
// The adapters' gradients: sum over an adapter's rows of p_t m_t^T, with p = dh and
// m = x for D, and p = c h and m = dy for U (written transposed).  A block takes
// kCols columns of m for one adapter; the blocks of a cluster share its rows.
// ---------------------------------------------------------------------------
template <class T>
struct Grads {
  Requests q;
  uint32_t rank, parts;
  uint64_t blocks[2];   // of columns, of x and of dy
  uint64_t cols[2];     // k, n
  const T* m[2];        // x, dy
  uint64_t stride[2];
  const float* p[2];    // dh, h
  T* out[2];            // adapters x rank x k, adapters x n x rank
  bool whole[2];
};

template <class T, int kRank>
struct GradShape {
  using P = Planes<T>;
  static constexpr int kRows = 64, kCols = 128;
  static constexpr int kRankPitch = kRank + 8, kColPitch = kCols + 8;
  static constexpr int kM = P::kW * kRows * kColPitch * 2;
  static constexpr int kP = P::kP * kRows * kRankPitch * 2;
  static constexpr int kStage = kM + kP;
  static constexpr int kSums = kRank * kCols * 4;
  static constexpr int kBytes = 2 * kStage > kSums ? 2 * kStage : kSums;
};

template <class T, int kRank>
__global__ void __launch_bounds__(kAdapterThreads)
    grads_kernel(const __grid_constant__ Grads<T> a) {
  using S = GradShape<T, kRank>;
  using P = Planes<T>;
  constexpr int kThreads = kAdapterThreads;
  constexpr int kMLoads = S::kRows * S::kCols / 8 / kThreads;
  constexpr int kPQuads = S::kRows * kRank / 4, kPLoads = (kPQuads + kThreads - 1) / kThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t from[kThreads], to[kThreads];  // rows of the adapter's requests
  __shared__ uint32_t counts[kThreads / 32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const uint32_t part = blockIdx.x % a.parts;
  const uint64_t all = a.blocks[0] + a.blocks[1];
  const uint64_t adapter = blockIdx.x / a.parts / all;
  uint64_t block = blockIdx.x / a.parts % all;
  const int sel = block >= a.blocks[0];
  if (sel) block -= a.blocks[0];
  const uint64_t col0 = block * S::kCols, cols = a.cols[sel];
  const T* const m = a.m[sel];
  const float* const p = a.p[sel];
  const uint64_t stride = a.stride[sel];
  const bool whole = a.whole[sel];
  const float scale = sel && a.q.scales ? a.q.scales[adapter] : 1.f;

  float acc[kRank / 16][2][4] = {};
  Raw<T> m_raw[kMLoads];
  float4 p_raw[kPLoads];
  auto load_stage = [&](uint64_t row0, int rows) {
#pragma unroll
    for (int i = 0; i < kMLoads; ++i) {
      const int at = tid + i * kThreads, row = at / (S::kCols / 8);
      const uint64_t col = col0 + at % (S::kCols / 8) * 8;
      m_raw[i].load(m + (row0 + row) * stride + col, row < rows ? static_cast<int64_t>(cols - col) : 0, whole);
    }
#pragma unroll
    for (int i = 0; i < kPLoads; ++i) {
      const int at = tid + i * kThreads, row = at * 4 / kRank, col = at * 4 % kRank;
      float* const e = reinterpret_cast<float*>(&p_raw[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        e[j] = row < rows && col + j < static_cast<int>(a.rank) ? p[(row0 + row) * a.rank + col + j] * scale : 0.f;
    }
  };
  auto store_stage = [&](int buffer) {
    uint8_t* const b = smem + buffer * S::kStage;
#pragma unroll
    for (int i = 0; i < kMLoads; ++i) {
      const int at = tid + i * kThreads, row = at / (S::kCols / 8), col = at % (S::kCols / 8) * 8;
      uint4 v[P::kW];
      split<T, P::kW>(m_raw[i], v);
#pragma unroll
      for (int q = 0; q < P::kW; ++q)
        *reinterpret_cast<uint4*>(b + ((q * S::kRows + row) * S::kColPitch + col) * 2) = v[q];
    }
#pragma unroll
    for (int i = 0; i < kPLoads; ++i) {
      const int at = tid + i * kThreads, row = at * 4 / kRank, col = at * 4 % kRank;
      if (kPQuads % kThreads && at >= kPQuads) break;
      uint32_t lo[P::kP], hi[P::kP];
      split_pair<P::kP>(p_raw[i].x, p_raw[i].y, lo);
      split_pair<P::kP>(p_raw[i].z, p_raw[i].w, hi);
#pragma unroll
      for (int q = 0; q < P::kP; ++q)
        *reinterpret_cast<uint2*>(b + S::kM + ((q * S::kRows + row) * S::kRankPitch + col) * 2) = make_uint2(lo[q], hi[q]);
    }
  };
  auto multiply = [&](int buffer) {
    const uint32_t ms = smem_u32(smem) + buffer * S::kStage, ps = ms + S::kM;
    constexpr bool kShort = sizeof(T) == 4;
    float chain[kRank / 16][2][4] = {};
#pragma unroll
    for (int t = 0; t < S::kRows; t += 16) {
      uint32_t w[P::kW][4];
#pragma unroll
      for (int j = 0; j < P::kW; ++j)
        ldsm_t(w[j], ms + ((j * S::kRows + t + lane % 16) * S::kColPitch + warp * 16 + lane / 16 * 8) * 2);
#pragma unroll
      for (int r = 0; r < kRank / 16; ++r)
#pragma unroll
        for (int i = 0; i < P::kP; ++i) {
          // rows of the product are ranks: the planes lie the other way around
          uint32_t h[4];
          ldsm_t(h, ps + ((i * S::kRows + t + lane % 8 + lane / 16 * 8) * S::kRankPitch + r * 16 + lane / 8 % 2 * 8) * 2);
#pragma unroll
          for (int j = 0; j < P::kW; ++j)
            if (P::takes(i, j)) {
              mma<false>(kShort ? chain[r][0] : acc[r][0], h, w[j][0], w[j][1]);
              mma<false>(kShort ? chain[r][1] : acc[r][1], h, w[j][2], w[j][3]);
            }
        }
    }
    if constexpr (kShort) {
#pragma unroll
      for (int r = 0; r < kRank / 16; ++r)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][n][i] += chain[r][n][i];
    }
  };

  uint64_t tile = 0;  // of the adapter's, counted over its requests
  for (uint64_t s0 = 0; s0 < a.q.requests; s0 += kThreads) {
    // the requests of this adapter among the next ones, in their order
    const uint64_t s = s0 + tid;
    const bool mine = s < a.q.requests && a.q.adapter(s + 1) == static_cast<int64_t>(adapter);
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, mine);
    if (lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    uint32_t at = __popc(votes & ((1u << lane) - 1)), found = 0;
    for (uint32_t w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += counts[w];
      found += counts[w];
    }
    if (mine) {
      from[at] = a.q.start(s + 1);
      to[at] = a.q.start(s + 2);
    }
    __syncthreads();
    // this block's tiles of theirs, the next one's loads on the way
    uint32_t i = 0;
    uint64_t row = found ? from[0] : 0;
    auto next = [&](uint64_t& row0, int& rows) {  // false: none left
      while (i < found) {
        if (row >= to[i]) {
          if (++i < found) row = from[i];
          continue;
        }
        row0 = row;
        rows = static_cast<int>(min(to[i] - row, static_cast<uint64_t>(S::kRows)));
        row += S::kRows;
        if (tile++ % a.parts == part) return true;
      }
      return false;
    };
    uint64_t row0;
    int rows, buffer = 0;
    bool more = next(row0, rows);
    if (more) {
      load_stage(row0, rows);
      store_stage(0);
    }
    __syncthreads();
    while (more) {
      more = next(row0, rows);
      if (more) load_stage(row0, rows);
      multiply(buffer);
      buffer ^= 1;
      if (more) store_stage(buffer);
      __syncthreads();
    }
  }

  // the parts' sums in a fixed order, and the result
  float* const sums = reinterpret_cast<float*>(smem);  // [rank][cols]
#pragma unroll
  for (int r = 0; r < kRank / 16; ++r)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        *reinterpret_cast<float2*>(sums + (r * 16 + lane / 4 + half * 8) * S::kCols + warp * 16 + n * 8 + lane % 4 * 2) =
            make_float2(acc[r][n][half * 2], acc[r][n][half * 2 + 1]);
  if (a.parts > 1) cluster_meet();
  else __syncthreads();
  T* const out = a.out[sel];
  const int each = kRank * S::kCols / a.parts;
  for (int e = tid; e < each; e += kThreads) {
    // neighbouring threads write neighbouring elements of either layout
    const int at = part * each + e;
    const int r = sel ? at % kRank : at / S::kCols, c = sel ? at / kRank : at % S::kCols;
    if (r >= static_cast<int>(a.rank) || col0 + c >= cols) continue;
    float v = 0.f;
    if (a.parts == 1) v = sums[r * S::kCols + c];
    else
      for (uint32_t q = 0; q < a.parts; ++q) v += remote_f32(smem_u32(sums + r * S::kCols + c), q);
    const uint64_t to_at = sel ? (adapter * cols + col0 + c) * a.rank + r : (adapter * a.rank + r) * cols + col0 + c;
    out[to_at] = from_f32<T>(v);
  }
  if (a.parts > 1) cluster_meet();  // the others stay until their parts are read
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <class A>
cudaError_t launch_clusters(void (*kernel)(A), const A& args, uint64_t blocks, uint32_t parts, int smem,
                            cudaStream_t st) {
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  if (smem > 40 * 1024) {  // static shared memory counts too
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kAdapterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <class T, int kRank, int kTile, bool kBack>
cudaError_t launch_chain(Chain<T> a, cudaStream_t st) {
  using S = ChainShape<T, kRank, kTile, kBack>;
  const uint64_t slots = slots_of(a.q.tokens, a.q.requests, kTile);
  a.parts = 1;
  while (a.parts < kAdapterParts && a.in >= 2ull * a.parts * 128) a.parts *= 2;
  auto share = [](uint64_t n, uint64_t by, uint64_t unit) { return ((n + by - 1) / by + unit - 1) / unit * unit; };
  a.part_in = share(a.in, a.parts, 64);
  const uint64_t tiles = a.q.tokens / kTile + (a.q.requests < a.q.tokens ? a.q.requests : a.q.tokens) + 1;
  const uint64_t most = a.out / (static_cast<uint64_t>(a.parts) * S::kCols) + 1;
  uint64_t groups = (4ull * sm_count() + tiles * a.parts - 1) / (tiles * a.parts);
  if (groups > most) groups = most;
  a.groups = static_cast<uint32_t>(groups);
  a.part_out = share(a.out, groups * a.parts, 32);
  return launch_clusters(chain_kernel<T, kRank, kTile, kBack>, a, slots * groups * a.parts, a.parts, S::kBytes, st);
}

template <class T, bool kBack>
cudaError_t chain(const Chain<T>& a, cudaStream_t st) {
  const bool tall = a.q.tokens >= 32 * a.q.requests;
  if (a.rank <= 16) return tall ? launch_chain<T, 16, 64, kBack>(a, st) : launch_chain<T, 16, 16, kBack>(a, st);
  return tall ? launch_chain<T, 64, 64, kBack>(a, st) : launch_chain<T, 64, 16, kBack>(a, st);
}

template <class T, int kRank>
cudaError_t launch_grads(Grads<T> a, cudaStream_t st) {
  using S = GradShape<T, kRank>;
  a.blocks[0] = a.out[0] ? (a.cols[0] + S::kCols - 1) / S::kCols : 0;
  a.blocks[1] = a.out[1] ? (a.cols[1] + S::kCols - 1) / S::kCols : 0;
  const uint64_t blocks = a.q.adapters * (a.blocks[0] + a.blocks[1]);
  if (!blocks) return cudaSuccess;
  a.parts = 1;
  while (a.parts < kAdapterParts && blocks * a.parts < 4ull * sm_count() &&
         a.q.tokens >= 2ull * a.parts * S::kRows)
    a.parts *= 2;
  return launch_clusters(grads_kernel<T, kRank>, a, blocks * a.parts, a.parts, S::kBytes, st);
}
template <class T>
cudaError_t grads(const Grads<T>& a, cudaStream_t st) {
  return a.rank <= 16 ? launch_grads<T, 16>(a, st) : launch_grads<T, 64>(a, st);
}

// adapter_f32.cu, adapter_bf16.cu, adapter_f16.cu
template <class T>
cudaError_t run_chain(const Chain<T>& a, bool back, cudaStream_t st);
template <class T>
cudaError_t run_grads(const Grads<T>& a, cudaStream_t st);

}  // namespace hkv
