// adapter.cuh -- the kernels of hkv_adapter_matmul and its backward pass: low-rank
// adapters of many requests beside a shared projection.
//
// A request s is the rows offsets[s] .. offsets[s + 1] - 1 of the batch and has
// the adapter a = which[s], two thin matrices D (rank x k) and U (n x rank) and a
// scale c:
//   h = c D x,  y = base + U h            dh = c U^T dy,  dx = base + D^T dh
//   dD = sum_t dh_t x_t^T                 dU = sum_t dy_t h_t^T
// Long requests take two kernels: the first product (x or dy with the first factor,
// its columns shared by a cluster's blocks, whose sums meet in distributed shared
// memory in a fixed order) and the second (onto base; it starts while the first one
// ends and has its factor and base on their way by then).  Short requests and single
// tokens, whose time is that of a launch and of a few latencies, take both in one
// kernel.  A third has the adapters' gradients, in tiles of rows or, where adapters have
// few of them, in sums of a thread's own.
//
// The products are thin: 2 rank operations for each element that is read or
// written, 16 to 64 where the tensor cores could take 280 and more, so memory is
// the bound.  16-bit matrices whose rows start on 16-byte boundaries go through
// tcgen05 (adapter_tensor.cuh); here is what takes ragged rows, short requests,
// float16 where it meets h, and float32: mma.sync, whose operands may be split in
// registers.  It multiplies bfloat16 (float16 in the first product of float16
// matrices); what has more digits is split into two or three bfloat16 numbers
// (planes), whose products are added in float32:
//   float32 = three planes exactly, products of planes i + j <= 2 (what is left
//   out is at most 2^-21 of a term); float16 = two planes exactly; h and dh, sums in
//   float32, in two planes where matrices have 16 bits (below 2^-16 of it is left
//   out, where a result is rounded to 2^-8 or 2^-11), in three where they have 32.
// Two planes are 16 of a sum's 24 digits, for a third less to read, to hold and to multiply
// wherever h and dh are used.  (7935 rows by rank 64, 4096 to 4096, bfloat16: h is off by
// 5.3e-6 of itself against 64 bits, 4.9e-6 of it by the planes, a product in 32 bits by
// 2.0e-7.  One output in 600, and one number of the gradients in 200, is the neighbouring
// bfloat16 number of what h in 32 bits gives; against 64 bits both are off by 1.57e-3 and
// 1.66e-3, bfloat16's own.)  Single rows have h in 32 bits for y and dh for dx, and hand on
// the planes to the gradients.
// Tiles come by asynchronous copies as they lie in memory (rows that start anywhere
// by the 16-byte pieces around them, shifted), and are split on the way to the tensor
// core.  Times: adapter_launch.cuh.  What they were with fewer of these: both products
// of long requests in one kernel of register-staged tiles 205 us where the two take 67
// (7883 rows, 4096 to 8192, rank 32) and 124 where they take 56 (7935 rows, 4096 to 4096,
// rank 64); single tokens in tiles of 16 rows 38 us, two kernels for them 20, one 12;
// gradients by request 57 us, across requests 31 (4096 rows in requests of 8, 2048 to
// 2048, rank 16), of 128 adapters of one row 57 and by thread 13; ragged x element by
// element 218 us, shifted 118.
#pragma once

#include <atomic>
#include <type_traits>

#include "operators.cuh"

namespace hkv {

constexpr int kAdapterThreads = 256;
constexpr int kAdapterParts = 8;  // blocks of a cluster at most
constexpr int kGradParts = 16;    // and of one that shares an adapter's rows

// Planes of the first product's operands, of a matrix that meets h or dh, and of
// these.
template <class T>
struct Planes {
  static constexpr int kIn = sizeof(T) == 4 ? 3 : 1;
  static constexpr int kW = sizeof(T) == 4 ? 3 : std::is_same_v<T, __half> ? 2 : 1;
  static constexpr int kP = sizeof(T) == 4 ? 3 : 2;
};

// Blocks of an SM that shared memory has room for, so that registers do not fall
// short of them.
template <class T, int kRank>
__host__ __device__ constexpr int blocks_of() { return sizeof(T) == 4 ? (kRank == 16 ? 3 : 2) : kRank == 64 ? 3 : 4; }

// What the requests are, as the kernels take it.  (Read past L1: the second
// product's kernel reads before it has waited.)
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
    const int64_t v = __ldcg(reinterpret_cast<const long long*>(offsets) + (s - 1));
    return v <= 0 ? 0 : min(static_cast<uint64_t>(v), tokens);
  }
  __device__ __forceinline__ int64_t adapter(uint64_t s) const {
    if (s == 0 || s > requests) return -1;
    const int64_t a = __ldcg(reinterpret_cast<const long long*>(which) + (s - 1));
    return a >= 0 && static_cast<uint64_t>(a) < adapters ? a : -1;
  }
};

// The rows of a block's tile.  Segment s has the slots start(s) / kTile + s up to
// start(s + 1) / kTile + s + 1, at least as many as it has tiles of kTile rows, so
// that a block finds its rows by one search and no list of tiles has to be made.
// (Tiles of one row: as many slots as rows, which need no request's number.)
struct Tile {
  uint64_t row0;
  int rows;
  int64_t adapter;
  template <int kTile>
  static __device__ __forceinline__ uint64_t first_slot(uint64_t start, uint64_t seg) {
    return kTile == 1 ? start : start / kTile + seg;
  }
  // False where the slot has none.  All threads of a warp call it.
  template <int kTile>
  __device__ __forceinline__ static bool find(const Requests& q, uint64_t slot, Tile& t) {
    const uint32_t lane = threadIdx.x & 31;
    uint64_t lo = 0, hi = q.requests + 2;  // the segment is one of lo .. hi - 1
    while (hi - lo > 31) {  // every turn leaves a thirty-second part
      const uint64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const bool before = at < hi && first_slot<kTile>(q.start(at), at) <= slot;
      const uint64_t n = __popc(__ballot_sync(0xFFFFFFFFu, before));
      lo += n * step;
      hi = min(lo + step, hi);
    }
    // the last ones all at once, with the next one's start and their adapters
    const uint64_t at = lo + lane, start = at <= hi ? q.start(at) : 0;
    const int64_t mine = at < hi ? q.adapter(at) : -1;
    const uint32_t before = __ballot_sync(0xFFFFFFFFu, at < hi && first_slot<kTile>(start, at) <= slot);
    const int seg = max(__popc(before) - 1, 0);
    const uint64_t from = __shfl_sync(0xFFFFFFFFu, start, seg), to = __shfl_sync(0xFFFFFFFFu, start, seg + 1);
    t.adapter = __shfl_sync(0xFFFFFFFFu, mine, seg);
    const uint64_t ahead = slot - first_slot<kTile>(from, lo + seg);
    t.row0 = from + ahead * kTile;
    if (t.row0 < from || t.row0 >= to) return false;
    t.rows = static_cast<int>(min(to - t.row0, static_cast<uint64_t>(kTile)));
    return true;
  }
};
inline uint64_t slots_of(uint64_t tokens, uint64_t requests, int tile) {
  return tile == 1 ? tokens : tokens / tile + requests + 2;
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// Eight neighbouring elements into shared memory, the first n of them and zeros
// behind: asynchronous, from a boundary of 16 bytes on.
__device__ __forceinline__ void copy_16(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
template <class T>
__device__ __forceinline__ void copy_eight(T* to, const T* from, int n) {
  constexpr int kVecs = sizeof(T) / 2, kPer = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    copy_16(smem_u32(to + i * kPer), from + i * kPer,
            (kVecs == 1 ? n : min(max(n - i * kPer, 0), kPer)) * static_cast<int>(sizeof(T)));
}
// The same from anywhere: the 16-byte pieces that hold any of them, shifted.
template <class T>
struct Shifted {
  static constexpr int kVecs = sizeof(T) / 2;
  uint4 piece[kVecs + 1];
  __device__ __forceinline__ void load(const T* from, int n) {
    const uint32_t off = reinterpret_cast<uintptr_t>(from) & 15;
    const uint4* const at = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(from) - off);
    const uint32_t end = off + n * static_cast<uint32_t>(sizeof(T));
#pragma unroll
    for (uint32_t i = 0; i <= kVecs; ++i) piece[i] = n > 0 && 16 * i < end ? __ldcg(at + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(T* to, const T* from, int n) {
    uint32_t x[4 * kVecs + 4];
#pragma unroll
    for (int i = 0; i <= kVecs; ++i) *reinterpret_cast<uint4*>(x + 4 * i) = piece[i];
    shift_bytes(x, reinterpret_cast<uintptr_t>(from) & 15);
    if (n < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= n) {
          if constexpr (sizeof(T) == 4) x[i] = 0;
          else x[i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(to)[i] = *reinterpret_cast<uint4*>(x + 4 * i);
  }
};
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kRows x kCols elements into a tile of that pitch by all threads: row r of the
// matrix is at data + r * stride, `rows` rows and `cols` columns of it are there.
// Rows that start anywhere (not `whole`) are read at once and shifted.
template <class T, int kRows, int kCols, int kPitch>
__device__ __noinline__ void copy_tile_shifted(T* tile, const T* data, uint64_t stride, int64_t rows, int64_t cols) {
  constexpr int kLanes = kCols / 8, kPass = kAdapterThreads / kLanes, kPasses = (kRows + kPass - 1) / kPass;
  const int row = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 8;
  if (kRows < kPass && row >= kRows) return;
  const int there = static_cast<int>(min(rows, static_cast<int64_t>(kRows))) - row;
  const int n = static_cast<int>(max(min(cols - col, static_cast<int64_t>(8)), static_cast<int64_t>(0)));
  const T* const from = data + row * stride + col;
  Shifted<T> v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) v[i].load(from + i * kPass * stride, i * kPass < there ? n : 0);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    v[i].store(tile + (row + i * kPass) * kPitch + col, from + i * kPass * stride, i * kPass < there ? n : 0);
}
template <class T, int kRows, int kCols, int kPitch>
__device__ __forceinline__ void copy_tile(T* tile, const T* data, uint64_t stride, int64_t rows, int64_t cols,
                                          bool whole) {
  constexpr int kLanes = kCols / 8, kPass = kAdapterThreads / kLanes;  // threads to a row, rows at a time
  static_assert(kAdapterThreads % kLanes == 0 && (kRows % kPass == 0 || kRows < kPass));
  if (!whole) {
    copy_tile_shifted<T, kRows, kCols, kPitch>(tile, data, stride, rows, cols);
    return;
  }
  const int row = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 8;
  if (kRows < kPass && row >= kRows) return;
  if (rows >= kRows && cols >= kCols) {
    const T* p = data + row * stride + col;
    uint32_t at = smem_u32(tile + row * kPitch + col);
#pragma unroll
    for (int i = 0; i < (kRows + kPass - 1) / kPass; ++i, p += kPass * stride, at += kPass * kPitch * sizeof(T))
#pragma unroll
      for (int v = 0; v < static_cast<int>(sizeof(T)) / 2; ++v)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + v * 16), "l"(p + v * (16 / sizeof(T))) : "memory");
    return;
  }
  const int there = static_cast<int>(min(rows, static_cast<int64_t>(kRows))) - row;
  const int n = static_cast<int>(max(min(cols - col, static_cast<int64_t>(8)), static_cast<int64_t>(0)));
  const T* const from = data + row * stride + col;
  T* const to = tile + row * kPitch + col;
#pragma unroll
  for (int i = 0; i < (kRows + kPass - 1) / kPass; ++i) {
    const bool has = i * kPass < there && n > 0;
    copy_eight(to + i * kPass * kPitch, has ? from + i * kPass * stride : data, has ? n : 0);
  }
}

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

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
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

// The planes of a 16 x 16 piece of a tile as the tensor core's first operand: rows
// row .. row + 15, columns k .. k + 15.
template <class T, int kN, int kPitch>
__device__ __forceinline__ void rows_operand(uint32_t (&a)[kN][4], const T* tile, int row, int k) {
  const int lane = threadIdx.x & 31;
  if constexpr (sizeof(T) == 2) {
    static_assert(kN == 1);
    ldsm(a[0], smem_u32(tile + (row + lane % 16) * kPitch + k + lane / 16 * 8));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(tile + (row + lane / 4 + i % 2 * 8) * kPitch + k + lane % 4 * 2 + i / 2 * 8);
      uint32_t p[kN];
      split_pair<kN>(v.x, v.y, p);
#pragma unroll
      for (int j = 0; j < kN; ++j) a[j][i] = p[j];
    }
  }
}
// And as its second operand, for 16 columns n .. n + 15 of the product ([0], [1] for
// the first eight): the tile holds them as rows, or, with kT, as columns.
template <class T, int kN, int kPitch, bool kT>
__device__ __forceinline__ void cols_operand(uint32_t (&b)[kN][4], const T* tile, int n, int k) {
  const int lane = threadIdx.x & 31;
  if constexpr (sizeof(T) == 2) {
    uint32_t r[4];
    if constexpr (kT) ldsm_t(r, smem_u32(tile + (k + lane % 16) * kPitch + n + lane / 16 * 8));
    else ldsm(r, smem_u32(tile + (n + lane % 8 + lane / 16 * 8) * kPitch + k + lane / 8 % 2 * 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kN == 1) {
        b[0][i] = r[i];
      } else {  // float16 in two planes
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
        uint32_t p[kN];
        split_pair<kN>(v.x, v.y, p);
#pragma unroll
        for (int j = 0; j < kN; ++j) b[j][i] = p[j];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = n + i / 2 * 8 + lane / 4, row = k + i % 2 * 8 + lane % 4 * 2;
      float2 v;
      if constexpr (kT) v = make_float2(tile[row * kPitch + col], tile[(row + 1) * kPitch + col]);
      else v = *reinterpret_cast<const float2*>(tile + col * kPitch + row);
      uint32_t p[kN];
      split_pair<kN>(v.x, v.y, p);
#pragma unroll
      for (int j = 0; j < kN; ++j) b[j][i] = p[j];
    }
  }
}

// A 16 x 16 piece of a product, as two of eight columns.  The tensor core cuts what
// it adds up, so float32 matrices keep the large terms in short chains of their own
// (`high`), the products with lower planes, 2^-8 of them, in another, and join both
// by rounding additions.
template <class T>
struct Sum {
  static constexpr bool kTwo = sizeof(T) == 4;
  float high[2][4] = {}, low[2][4] = {};
  __device__ __forceinline__ float at(int half, int i) const {
    return kTwo ? high[half][i] + low[half][i] : high[half][i];
  }
};
// Adds one k16 step to kN pieces side by side; products that follow one another go to
// different sums.
template <class T, int kN, int kA, int kB, bool kF16 = false>
__device__ __forceinline__ void add(Sum<T> (&d)[kN], const uint32_t (&a)[kA][4], const uint32_t (&b)[kN][kB][4]) {
#pragma unroll
  for (int i = 0; i < kA; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      if (Sum<T>::kTwo && i + j > 2) continue;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          mma<kF16>(Sum<T>::kTwo && i + j > 0 ? d[n].low[half] : d[n].high[half], a[i], b[n][j][half * 2], b[n][j][half * 2 + 1]);
    }
}
// And to chains that go on from one stage to the next where they need not be short.
template <class T, int kN, int kA, int kB, bool kF16>
__device__ __forceinline__ void add_onto(float (&acc)[kN][2][4], const uint32_t (&a)[kA][4], const uint32_t (&b)[kN][kB][4]) {
  Sum<T> d[kN];
  if constexpr (!Sum<T>::kTwo) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) d[n].high[i / 4][i % 4] = acc[n][i / 4][i % 4];
  }
  add<T, kN, kA, kB, kF16>(d, a, b);
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& to = acc[n][i / 4][i % 4];
      to = Sum<T>::kTwo ? to + d[n].at(i / 4, i % 4) : d[n].high[i / 4][i % 4];
    }
}

// Two neighbouring elements in shared memory.
template <class T>
__device__ __forceinline__ float2 pair_at(const T* p) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  else if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(p));
  else return *reinterpret_cast<const float2*>(p);
}
template <class T>
__device__ __forceinline__ void put_pair(T* p, float a, float b) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
  else if constexpr (std::is_same_v<T, __half>) *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
  else *reinterpret_cast<float2*>(p) = make_float2(a, b);
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
// elements in.  whole: eight elements of a row may be taken by 16-byte copies.
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
  __nv_bfloat16* hidden;  // tokens x planes x kRank, c h or dh
  uint32_t parts;         // first product: blocks of a cluster
  uint64_t part_in;       //   and columns of x to each
  uint32_t groups;        // second product: blocks of a tile of rows
  uint64_t group_out;     //   and columns of y to each
  bool x_whole, base_whole, y_whole;
  bool follows;           // the second product comes after a first one
};

// Four numbers of a row's c h or dh, as planes.
template <class T, int kRank>
__device__ __forceinline__ void put_hidden(__nv_bfloat16* hidden, uint64_t row, int col, float4 v, float scale) {
  using P = Planes<T>;
  uint32_t lo[P::kP], hi[P::kP];
  split_pair<P::kP>(v.x * scale, v.y * scale, lo);
  split_pair<P::kP>(v.z * scale, v.w * scale, hi);
  __nv_bfloat16* const h = hidden + row * (P::kP * kRank) + col;
#pragma unroll
  for (int p = 0; p < P::kP; ++p) *reinterpret_cast<uint2*>(h + p * kRank) = make_uint2(lo[p], hi[p]);
}

// ---------------------------------------------------------------------------
// the first product
// ---------------------------------------------------------------------------
template <class T, int kRank, int kTile, bool kBack>
struct FirstShape {
  static constexpr int kRowWarps = kTile / 16, kOther = 8 / kRowWarps;  // warps along rows, along columns of x
  static constexpr int kStep = kTile == 64 ? (sizeof(T) == 4 ? 64 : 128) : 128;  // columns of x to a stage
  static constexpr int kStages = sizeof(T) == 4 || kTile == 64 ? 3 : 4;
  static constexpr int kPitch = kStep + 8, kFirstPitch = kBack ? kRank + 8 : kPitch;
  static constexpr int kX = kTile * kPitch, kFirst = (kBack ? kStep : kRank) * kFirstPitch;
  static constexpr int kStage = kX + kFirst;  // elements
  static constexpr int kSums = (kOther + 1) * kTile * kRank * 4;
  static constexpr int kBytes = kStages * kStage * static_cast<int>(sizeof(T)) > kSums
                                    ? kStages * kStage * static_cast<int>(sizeof(T)) : kSums;
};

// acc = columns in0 .. in1 - 1 of x's tile times the first factor's: a warp's rows
// by all ranks, from its share of the columns.  All warps are through with the stages
// when it returns.
template <class T, int kRank, int kTile, bool kBack>
__device__ __forceinline__ void first_product(float (&acc)[kRank / 16][2][4], T* stages, const Chain<T>& a,
                                              const Tile& t, uint64_t in0, uint64_t in1) {
  using S = FirstShape<T, kRank, kTile, kBack>;
  using P = Planes<T>;
  const uint32_t warp = threadIdx.x >> 5, row_warp = warp % S::kRowWarps, other = warp / S::kRowWarps;
  const T* const x = a.x + t.row0 * a.x_stride;
  const T* const first = a.first.data + t.adapter * a.first.step;
  const int steps = static_cast<int>((in1 - in0 + S::kStep - 1) / S::kStep);
  auto load = [&](int step) {
    if (step < steps) {
      T* const to = stages + step % S::kStages * S::kStage;
      const uint64_t k = in0 + static_cast<uint64_t>(step) * S::kStep;
      const int64_t left = in1 - k;
      copy_tile<T, kTile, S::kStep, S::kPitch>(to, x + k, a.x_stride, t.rows, left, a.x_whole);
      if constexpr (kBack)
        copy_tile<T, S::kStep, kRank, S::kFirstPitch>(to + S::kX, first + k * a.first.stride, a.first.stride, left, a.rank, a.first.whole);
      else
        copy_tile<T, kRank, S::kStep, S::kFirstPitch>(to + S::kX, first + k, a.first.stride, a.rank, left, a.first.whole);
    }
    copies_end();
  };
#pragma unroll
  for (int n = 0; n < kRank / 16; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[n][i / 4][i % 4] = 0.f;
#pragma unroll
  for (int s = 0; s + 1 < S::kStages; ++s) load(s);
  for (int step = 0; step < steps; ++step) {
    copies_wait<S::kStages - 2>();
    __syncthreads();
    load(step + S::kStages - 1);
    const T* const xs = stages + step % S::kStages * S::kStage;
    const T* const ws = xs + S::kX;
    constexpr int kEach = S::kStep / 16 / S::kOther;
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
      const int k = (other * kEach + s) * 16;
      uint32_t xa[P::kIn][4];
      rows_operand<T, P::kIn, S::kPitch>(xa, xs, row_warp * 16, k);
      constexpr int kN = sizeof(T) == 4 ? 1 : kRank / 16;
#pragma unroll
      for (int n = 0; n < kRank / 16; n += kN) {
        uint32_t w[kN][P::kIn][4];
#pragma unroll
        for (int i = 0; i < kN; ++i) cols_operand<T, P::kIn, S::kFirstPitch, kBack>(w[i], ws, (n + i) * 16, k);
        add_onto<T, kN, P::kIn, P::kIn, std::is_same_v<T, __half>>(reinterpret_cast<float(&)[kN][2][4]>(acc[n]), xa, w);
      }
    }
  }
  copies_wait<0>();
  __syncthreads();
}

// A warp's sums as sums[other][tile][rank].
template <int kRank, int kTile>
__device__ __forceinline__ void put_sums(float* sums, const float (&acc)[kRank / 16][2][4], int other, int row_warp) {
  const int lane = threadIdx.x & 31;
  float* const to = sums + (other * kTile + row_warp * 16 + lane / 4) * kRank + lane % 4 * 2;
#pragma unroll
  for (int n = 0; n < kRank / 8; ++n) {
    const float(&v)[4] = acc[n / 2][n % 2];
    *reinterpret_cast<float2*>(to + n * 8) = make_float2(v[0], v[1]);
    *reinterpret_cast<float2*>(to + 8 * kRank + n * 8) = make_float2(v[2], v[3]);
  }
}

template <class T, int kRank, int kTile, bool kBack>
__global__ void __launch_bounds__(kAdapterThreads)
    first_kernel(const __grid_constant__ Chain<T> a) {
  using S = FirstShape<T, kRank, kTile, kBack>;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t tid = threadIdx.x, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();  // what the second product reads before it waits is complete from here on
  const uint32_t part = blockIdx.x % a.parts;
  Tile t;
  if (!Tile::find<kTile>(a.q, blockIdx.x / a.parts, t) || t.adapter < 0) return;  // the whole cluster
  const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
  float acc[kRank / 16][2][4];
  first_product<T, kRank, kTile, kBack>(acc, reinterpret_cast<T*>(smem), a, t, in0, in1);

  // the warps' sums, then the blocks', each block a share of them
  float* const sums = reinterpret_cast<float*>(smem);  // [other][tile][rank]
  float* const own = sums + S::kOther * kTile * kRank;
  put_sums<kRank, kTile>(sums, acc, warp / S::kRowWarps, warp % S::kRowWarps);
  __syncthreads();
  constexpr int kQuads = kTile * kRank / 4;
  const float scale = a.q.scales ? a.q.scales[t.adapter] : 1.f;
  auto block_sum = [&](int i) {
    float4 v = reinterpret_cast<const float4*>(sums)[i];
#pragma unroll
    for (int o = 1; o < S::kOther; ++o) v = v + reinterpret_cast<const float4*>(sums)[o * kQuads + i];
    return v;
  };
  auto put = [&](int i, float4 v) {
    const int row = i * 4 / kRank, col = i * 4 % kRank;
    if (row >= t.rows) return;
    put_hidden<T, kRank>(a.hidden, t.row0 + row, col, v, scale);
  };
  if (a.parts == 1) {
    for (int i = tid; i < kQuads; i += kAdapterThreads) put(i, block_sum(i));
    return;
  }
  for (int i = tid; i < kQuads; i += kAdapterThreads) reinterpret_cast<float4*>(own)[i] = block_sum(i);
  cluster_meet();
  const uint32_t used = static_cast<uint32_t>((a.in + a.part_in - 1) / a.part_in);  // parts with columns
  const int each = kQuads / a.parts;
  for (int e = tid; e < each; e += kAdapterThreads) {
    const int i = part * each + e;
    float4 v = remote_f32x4(smem_u32(own) + i * 16, 0);
    for (uint32_t p = 1; p < used; ++p) v = v + remote_f32x4(smem_u32(own) + i * 16, p);
    put(i, v);
  }
  cluster_meet();  // the others stay until their sums are read
}

// ---------------------------------------------------------------------------
// the second product
// ---------------------------------------------------------------------------
template <class T, int kRank, int kTile, bool kBack>
struct SecondShape {
  static constexpr int kRowWarps = kTile / 16, kOther = 8 / kRowWarps;
  static constexpr int kWarpCols = kTile == 64 ? (sizeof(T) == 4 ? 32 : 64) : (sizeof(T) == 4 ? 16 : 32);
  static constexpr int kCols = kOther * kWarpCols;  // columns of y to a stage
  static constexpr int kStages = 2;
  static constexpr int kPitch = kCols + 8, kSecondPitch = kBack ? kPitch : kRank + 8, kHiddenPitch = kRank + 8;
  static constexpr int kBase = kTile * kPitch, kSecond = (kBack ? kRank : kCols) * kSecondPitch;
  static constexpr int kStage = kBase + kSecond;  // elements
  static constexpr int kHidden = Planes<T>::kP * kTile * kHiddenPitch * 2;
  // the hidden numbers come by way of the last stage, before it has a tile
  static constexpr int kHiddenAt = (kStages - 1) * kStage * static_cast<int>(sizeof(T));
  static constexpr int kLast = kStage * static_cast<int>(sizeof(T));
  static constexpr int kBytes = kHiddenAt + (kLast > kHidden ? kLast : kHidden);
};

// One stage of base, in shared memory, and its columns c0 .. of the second factor
// behind it: y's columns c0 .. col1 - 1 of the stage.
template <class T, int kRank, int kTile, bool kBack>
__device__ __forceinline__ void second_step(T* stage, const uint32_t (&h)[kRank / 16][Planes<T>::kP][4], bool adapts,
                                            int rows, T* y, uint64_t c0, uint64_t col1, uint64_t stride, bool whole) {
  using S = SecondShape<T, kRank, kTile, kBack>;
  using P = Planes<T>;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t row_warp = warp % S::kRowWarps, other = warp / S::kRowWarps;
  if (adapts) {
    constexpr int kN = sizeof(T) == 4 ? 1 : 2;
#pragma unroll
    for (int n = 0; n < S::kWarpCols; n += 16 * kN) {
      const int c = other * S::kWarpCols + n;
      T* const at = stage + (row_warp * 16 + lane / 4) * S::kPitch + c + lane % 4 * 2;
      auto place = [&](int i) { return at + i % 2 * 8 * S::kPitch + i / 2 * 8; };  // of 4 kN pairs of base
      Sum<T> d[kN];
      if constexpr (!Sum<T>::kTwo) {  // sums start with base
#pragma unroll
        for (int i = 0; i < 4 * kN; ++i) {
          const float2 v = pair_at(place(i));
          d[i / 4].high[i / 2 % 2][i % 2 * 2] = v.x;
          d[i / 4].high[i / 2 % 2][i % 2 * 2 + 1] = v.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kRank / 16; ++k) {
        uint32_t w[kN][P::kW][4];
#pragma unroll
        for (int i = 0; i < kN; ++i) cols_operand<T, P::kW, S::kSecondPitch, kBack>(w[i], stage + S::kBase, c + i * 16, k * 16);
        add(d, h[k], w);
      }
#pragma unroll
      for (int i = 0; i < 4 * kN; ++i) {
        float2 v = make_float2(0.f, 0.f);
        if constexpr (Sum<T>::kTwo) v = pair_at(place(i));
        put_pair(place(i), v.x + d[i / 4].at(i / 2 % 2, i % 2 * 2), v.y + d[i / 4].at(i / 2 % 2, i % 2 * 2 + 1));
      }
    }
    __syncwarp();
  }
  if (!whole) {  // rows of y that start anywhere: neighbouring elements by neighbouring lanes
    const uint64_t first = c0 + other * S::kWarpCols;
    const int cols = static_cast<int>(min(static_cast<int64_t>(col1 - first), static_cast<int64_t>(S::kWarpCols)));
    for (int r = 0; r < 16 && row_warp * 16 + r < rows; ++r) {
      const int row = row_warp * 16 + r;
      const T* const from = stage + row * S::kPitch + other * S::kWarpCols;
      T* const out = y + row * stride + first;
#pragma unroll
      for (int c = lane; c < S::kWarpCols; c += 32)
        if (c < cols) out[c] = from[c];
    }
    return;
  }
  // a warp's rows of kWarpCols columns, eight to a lane
  constexpr int kLanes = S::kWarpCols / 8;
  const uint64_t col = c0 + other * S::kWarpCols + lane % kLanes * 8;
#pragma unroll
  for (int r = lane / kLanes; r < 16; r += 32 / kLanes) {
    const int row = row_warp * 16 + r;
    if (row >= rows) break;
    const int64_t n = col1 - col;
    const T* const from = stage + row * S::kPitch + other * S::kWarpCols + lane % kLanes * 8;
    T* const out = y + row * stride + col;
    if (n >= 8) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        st_stream_v4(out + i * (16 / sizeof(T)), reinterpret_cast<const uint4*>(from)[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) out[i] = from[i];
    }
  }
}

template <class T, int kRank, int kTile, bool kBack>
__global__ void __launch_bounds__(kAdapterThreads, blocks_of<T, kRank>())
    second_kernel(const __grid_constant__ Chain<T> a) {
  using S = SecondShape<T, kRank, kTile, kBack>;
  using P = Planes<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  T* const stages = reinterpret_cast<T*>(smem);
  __nv_bfloat16* const hidden = reinterpret_cast<__nv_bfloat16*>(smem + S::kHiddenAt);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t row_warp = warp % S::kRowWarps;

  // before the first product's end: its kernel lets this one start when all that
  // came before is complete, and it writes `hidden` alone
  if (!a.follows) pdl_wait();
  const uint64_t col0 = static_cast<uint64_t>(blockIdx.x % a.groups) * a.group_out;
  const uint64_t col1 = min(col0 + a.group_out, a.out);
  Tile t;
  const bool any = Tile::find<kTile>(a.q, blockIdx.x / a.groups, t) && col0 < col1;
  const bool adapts = any && t.adapter >= 0;
  const bool copies = any && (adapts || a.y != a.base);
  const T* const base = a.base ? a.base + t.row0 * a.base_stride : nullptr;
  const T* const second = a.second.data + (adapts ? t.adapter * a.second.step : 0);
  const int steps = copies ? static_cast<int>((col1 - col0 + S::kCols - 1) / S::kCols) : 0;
  auto load = [&](int step) {
    if (step < steps) {
      T* const to = stages + step % S::kStages * S::kStage;
      const uint64_t c = col0 + static_cast<uint64_t>(step) * S::kCols;
      const int64_t left = col1 - c;
      copy_tile<T, kTile, S::kCols, S::kPitch>(to, base ? base + c : reinterpret_cast<const T*>(a.hidden), a.base_stride, base ? t.rows : 0, left, a.base_whole);
      if (adapts) {
        if constexpr (kBack)
          copy_tile<T, kRank, S::kCols, S::kSecondPitch>(to + S::kBase, second + c, a.second.stride, a.rank, left, a.second.whole);
        else
          copy_tile<T, S::kCols, kRank, S::kSecondPitch>(to + S::kBase, second + c * a.second.stride, a.second.stride, left, a.rank, a.second.whole);
      }
    }
    copies_end();
  };
#pragma unroll
  for (int s = 0; s + 1 < S::kStages; ++s) load(s);
  pdl_wait();
  pdl_trigger();
  if (!copies) {
    copies_wait<0>();
    return;
  }
  uint32_t h[kRank / 16][P::kP][4];
  if (adapts) {
    constexpr int kChunks = P::kP * kTile * kRank / 8;
    for (int i = tid; i < kChunks; i += kAdapterThreads) {
      const int row = i / (P::kP * kRank / 8), plane = i / (kRank / 8) % P::kP, col = i % (kRank / 8) * 8;
      const bool there = row < t.rows;
      copy_16(smem_u32(hidden + (plane * kTile + row) * S::kHiddenPitch + col),
              a.hidden + (t.row0 + (there ? row : 0)) * (P::kP * kRank) + plane * kRank + col, there ? 16 : 0);
    }
    copies_end();
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRank / 16; ++k)
#pragma unroll
      for (int p = 0; p < P::kP; ++p)
        ldsm(h[k][p], smem_u32(hidden + (p * kTile + row_warp * 16 + lane % 16) * S::kHiddenPitch + k * 16 + lane / 16 * 8));
  }
  T* const y = a.y + t.row0 * a.y_stride;
  for (int step = 0; step < steps; ++step) {
    copies_wait<S::kStages - 2>();
    __syncthreads();
    load(step + S::kStages - 1);
    second_step<T, kRank, kTile, kBack>(stages + step % S::kStages * S::kStage, h, adapts, t.rows, y,
                                        col0 + static_cast<uint64_t>(step) * S::kCols, col1, a.y_stride, a.y_whole);
  }
  copies_wait<0>();
}

// ---------------------------------------------------------------------------
// Short requests: both products of a tile of 16 rows in one kernel.  A cluster's
// blocks share the tile's columns of x, put the sums together in every one of them,
// and share its columns of y.
// ---------------------------------------------------------------------------
template <class T, int kRank, bool kBack>
struct ShortShape {
  using F = FirstShape<T, kRank, 16, kBack>;
  using S = SecondShape<T, kRank, 16, kBack>;
  static constexpr int kHidden = Planes<T>::kP * 16 * S::kHiddenPitch * 2;
  // sums, the block's own and the planes lie where the first product's stages were,
  // the second one's stages behind them
  static constexpr int kSecondAt = F::kSums + kHidden;
  static constexpr int kSecond = kSecondAt + S::kStages * S::kStage * static_cast<int>(sizeof(T));
  static constexpr int kFirst = F::kStages * F::kStage * static_cast<int>(sizeof(T));
  static constexpr int kBytes = kFirst > kSecond ? kFirst : kSecond;
};

template <class T, int kRank, bool kBack>
__global__ void __launch_bounds__(kAdapterThreads, blocks_of<T, kRank>())
    short_kernel(const __grid_constant__ Chain<T> a) {
  using Shape = ShortShape<T, kRank, kBack>;
  using F = typename Shape::F;
  using S = typename Shape::S;
  using P = Planes<T>;
  constexpr int kTile = 16;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const uint32_t part = blockIdx.x % a.parts, group = blockIdx.x / a.parts % a.groups;
  Tile t;
  if (!Tile::find<kTile>(a.q, blockIdx.x / a.parts / a.groups, t)) return;  // the whole cluster
  const uint64_t col0 = (static_cast<uint64_t>(group) * a.parts + part) * a.group_out;
  const uint64_t col1 = min(col0 + a.group_out, a.out);
  const bool adapts = t.adapter >= 0;
  if (!adapts && (a.y == a.base || col0 >= col1)) return;  // no block of the cluster meets another

  float* const sums = reinterpret_cast<float*>(smem);  // [warp][tile][rank]
  float* const own = sums + F::kOther * kTile * kRank;
  __nv_bfloat16* const hidden = reinterpret_cast<__nv_bfloat16*>(smem + F::kSums);
  T* const stages = reinterpret_cast<T*>(smem + Shape::kSecondAt);
  const T* const base = a.base ? a.base + t.row0 * a.base_stride : nullptr;
  const T* const second = a.second.data + (adapts ? t.adapter * a.second.step : 0);
  const int col_steps = col0 < col1 ? static_cast<int>((col1 - col0 + S::kCols - 1) / S::kCols) : 0;
  auto load_second = [&](int step) {
    if (step < col_steps) {
      T* const to = stages + step % S::kStages * S::kStage;
      const uint64_t c = col0 + static_cast<uint64_t>(step) * S::kCols;
      const int64_t left = col1 - c;
      copy_tile<T, kTile, S::kCols, S::kPitch>(to, base ? base + c : reinterpret_cast<const T*>(a.hidden), a.base_stride, base ? t.rows : 0, left, a.base_whole);
      if (adapts) {
        if constexpr (kBack)
          copy_tile<T, kRank, S::kCols, S::kSecondPitch>(to + S::kBase, second + c, a.second.stride, a.rank, left, a.second.whole);
        else
          copy_tile<T, S::kCols, kRank, S::kSecondPitch>(to + S::kBase, second + c * a.second.stride, a.second.stride, left, a.rank, a.second.whole);
      }
    }
    copies_end();
  };
  uint32_t h[kRank / 16][P::kP][4];
  if (adapts) {
    const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
    float acc[kRank / 16][2][4];
    first_product<T, kRank, kTile, kBack>(acc, reinterpret_cast<T*>(smem), a, t, in0, in1);
    // (all warps are through with the stages)
#pragma unroll
    for (int s = 0; s + 1 < S::kStages; ++s) load_second(s);  // on their way meanwhile
    put_sums<kRank, kTile>(sums, acc, warp, 0);
    __syncthreads();
    constexpr int kQuads = kTile * kRank / 4;
    static_assert(kQuads <= kAdapterThreads);
    const float scale = a.q.scales ? a.q.scales[t.adapter] : 1.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid < kQuads) {
      v = reinterpret_cast<const float4*>(sums)[tid];
#pragma unroll
      for (int o = 1; o < F::kOther; ++o) v = v + reinterpret_cast<const float4*>(sums)[o * kQuads + tid];
    }
    if (a.parts > 1) {
      if (tid < kQuads) reinterpret_cast<float4*>(own)[tid] = v;
      cluster_meet();
      const uint32_t used = static_cast<uint32_t>((a.in + a.part_in - 1) / a.part_in);  // parts with columns
      if (tid < kQuads) {
        v = remote_f32x4(smem_u32(own) + tid * 16, 0);
        for (uint32_t p = 1; p < used; ++p) v = v + remote_f32x4(smem_u32(own) + tid * 16, p);
      }
      cluster_arrive();
    }
    if (tid < kQuads) {
      const int row = tid * 4 / kRank, col = tid * 4 % kRank;
      uint32_t lo[P::kP], hi[P::kP];
      split_pair<P::kP>(v.x * scale, v.y * scale, lo);
      split_pair<P::kP>(v.z * scale, v.w * scale, hi);
#pragma unroll
      for (int p = 0; p < P::kP; ++p) {
        *reinterpret_cast<uint2*>(hidden + (p * kTile + row) * S::kHiddenPitch + col) = make_uint2(lo[p], hi[p]);
        if (group == 0 && part == 0 && row < t.rows)
          *reinterpret_cast<uint2*>(a.hidden + (t.row0 + row) * (P::kP * kRank) + p * kRank + col) = make_uint2(lo[p], hi[p]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRank / 16; ++k)
#pragma unroll
      for (int p = 0; p < P::kP; ++p)
        ldsm(h[k][p], smem_u32(hidden + (p * kTile + lane % 16) * S::kHiddenPitch + k * 16 + lane / 16 * 8));
  } else {
#pragma unroll
    for (int s = 0; s + 1 < S::kStages; ++s) load_second(s);
  }
  T* const y = a.y + t.row0 * a.y_stride;
  for (int step = 0; step < col_steps; ++step) {
    copies_wait<S::kStages - 2>();
    __syncthreads();
    load_second(step + S::kStages - 1);
    second_step<T, kRank, kTile, kBack>(stages + step % S::kStages * S::kStage, h, adapts, t.rows, y,
                                        col0 + static_cast<uint64_t>(step) * S::kCols, col1, a.y_stride, a.y_whole);
  }
  copies_wait<0>();
  if (adapts && a.parts > 1) cluster_wait();  // the others have read this block's sums
}

// ---------------------------------------------------------------------------
// Single tokens, and requests of few rows: one row to a cluster, whose products are sums
// over factors that are read once, past shared memory, wherever their rows start.  h = c D x: a warp takes two ranks at a time, its
// lanes the columns, eight each; where there are fewer pairs of ranks than warps, the
// others take other columns.  y = base + U h: a column to a thread at a time.
// ---------------------------------------------------------------------------
// kN neighbouring elements of a row, n of which there are: from a 16-byte boundary on, or
// (not kWhole) the 16-byte pieces that hold any of them, to be shifted once they are there.
template <class T, int kN, bool kWhole>
struct Run {
  static constexpr int kPieces = kN * static_cast<int>(sizeof(T)) / 16 + !kWhole;
  uint32_t w[4 * kPieces];
  __device__ __forceinline__ void load(const T* p, int n) {
    const uint32_t off = kWhole ? 0 : reinterpret_cast<uintptr_t>(p) & 15;
    const int end = n > 0 ? static_cast<int>(off) + n * static_cast<int>(sizeof(T)) : 0;
    const char* const at = reinterpret_cast<const char*>(p) - off;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      *reinterpret_cast<uint4*>(w + 4 * i) = 16 * i < end ? ld_nc_v4(at + 16 * i) : make_uint4(0, 0, 0, 0);
  }
  // Of the same p and n: zeros behind the n elements.
  __device__ __forceinline__ void settle(const T* p, int n) {
    if constexpr (!kWhole) {
      shift_bytes(w, reinterpret_cast<uintptr_t>(p) & 15);
      if (n >= kN) return;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i >= n) {
          if constexpr (sizeof(T) == 4) w[i] = 0;
          else w[i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
  }
  __device__ __forceinline__ float2 pair(int i) const { return pair_at(reinterpret_cast<const T*>(w) + 2 * i); }
};

// A row's c h or dh in `hidden`, from the sums of `slices` shares of a block's columns and
// of the cluster's blocks.
template <class T, int kRank>
__device__ __forceinline__ void thin_hidden(const Chain<T>& a, const Tile& t, uint32_t part, uint32_t group,
                                            float (*sums)[kRank], uint32_t slices, float* hidden) {
  using P = Planes<T>;
  const uint32_t tid = threadIdx.x;
  __syncthreads();
  float v = 0.f;
  if (tid < kRank)
    for (uint32_t s = 0; s < slices; ++s) v += sums[s][tid];
  if (a.parts > 1) {
    __syncthreads();
    if (tid < kRank) sums[0][tid] = v;
    cluster_meet();
    if (tid < kRank) {
      v = 0.f;
      for (uint32_t p = 0; p < a.parts; ++p) v += remote_f32(smem_u32(&sums[0][tid]), p);
    }
    cluster_arrive();
  }
  if (tid < kRank) {
    hidden[tid] = v *= a.q.scales ? a.q.scales[t.adapter] : 1.f;
    if (group == 0 && part == 0) {  // for the gradients
      uint32_t w[P::kP];
      split_pair<P::kP>(v, 0.f, w);
#pragma unroll
      for (int p = 0; p < P::kP; ++p)
        reinterpret_cast<uint16_t*>(a.hidden)[t.row0 * (P::kP * kRank) + p * kRank + tid] = static_cast<uint16_t>(w[p]);
    }
  }
  __syncthreads();
}

// Columns of y that a thread has on their way at a time.  (Of eight ranks one, two and four:
// 302 float16 requests of 3 rows, 1163 to 12920, 66, 52 and 49 us.)
template <class T, int kUsed>
__host__ __device__ constexpr int thin_columns() {
  return kUsed == 8 ? 4 : kUsed == 64 || (kUsed == 32 && sizeof(T) == 4) ? 1 : 2;
}

// (The adapters have kUsed ranks at most.)
template <class T, int kRank, int kUsed, bool kWhole>
__global__ void __launch_bounds__(kAdapterThreads, 2)
    thin_kernel(const __grid_constant__ Chain<T> a) {
  constexpr int kWarps = kAdapterThreads / 32;
  constexpr int kMost = kWhole ? 4 : sizeof(T) == 2 ? 2 : 1;  // loads of a rank in flight
  constexpr int kEach = thin_columns<T, kUsed>();
  __shared__ __align__(16) float sums[kWarps][kRank], hidden[kRank];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const uint32_t part = blockIdx.x % a.parts, group = blockIdx.x / a.parts % a.groups;
  Tile t;
  if (!Tile::find<1>(a.q, blockIdx.x / a.parts / a.groups, t)) return;  // the whole cluster
  const uint64_t col0 = (static_cast<uint64_t>(group) * a.parts + part) * a.group_out;
  const uint64_t col1 = min(col0 + a.group_out, a.out);
  const bool adapts = t.adapter >= 0;
  if (!adapts && a.y == a.base) return;
  const T* const second = a.second.data + (adapts ? t.adapter * a.second.step : 0);
  const T* const base = a.base + t.row0 * a.base_stride;
  Run<T, kUsed, kWhole> u[kEach];
  float onto[kEach];
  auto load_columns = [&](uint64_t c) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint64_t col = c + e * kAdapterThreads + tid;
      u[e].load(second + col * a.second.stride, adapts && col < col1 ? a.rank : 0);
      onto[e] = a.base && col < col1 ? to_f32(base[col]) : 0.f;
    }
  };
  load_columns(col0);  // on their way during the first product
  if (adapts) {
    const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
    const uint32_t pairs = (a.rank + 1) / 2;
    uint32_t slices = 1;  // of the columns
    while (slices * 2 * pairs <= kWarps) slices *= 2;
    const uint32_t slice = warp % slices;
    const T* const first = a.first.data + t.adapter * a.first.step;
    const T* const x = a.x + t.row0 * a.x_stride;
    for (uint32_t i = tid; i < kWarps * kRank; i += kAdapterThreads) (&sums[0][0])[i] = 0.f;
    __syncthreads();
    for (uint32_t pair = warp / slices; pair < pairs; pair += kWarps / slices) {
      const T* const d0 = first + 2 * pair * a.first.stride;
      const bool two = 2 * pair + 1 < a.rank;
      float acc[2] = {};
      for (uint64_t k = in0 + slice * 256 + lane * 8; k < in1; k += slices * 256 * kMost) {
        Run<T, 8, kWhole> d[2][kMost], e[kWhole ? 1 : kMost];
        auto there = [&](uint64_t at) {
          return kWhole ? (at < in1 ? 8 : 0) : static_cast<int>(min(in1 - min(at, in1), static_cast<uint64_t>(8)));
        };
#pragma unroll
        for (int m = 0; m < kMost; ++m) {
          const uint64_t at = k + m * slices * 256;
          d[0][m].load(d0 + at, there(at));
          d[1][m].load(d0 + a.first.stride + at, two ? there(at) : 0);
          if constexpr (!kWhole) e[m].load(x + at, there(at));
        }
#pragma unroll
        for (int m = 0; m < kMost; ++m) {
          const uint64_t at = k + m * slices * 256;
          if constexpr (kWhole) e[0].load(x + at, there(at));
          auto& v8 = e[kWhole ? 0 : m];
          v8.settle(x + at, there(at));
          d[0][m].settle(d0 + at, there(at));
          d[1][m].settle(d0 + a.first.stride + at, two ? there(at) : 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = v8.pair(i), p = d[0][m].pair(i), q = d[1][m].pair(i);
            acc[0] = fmaf(v.y, p.y, fmaf(v.x, p.x, acc[0]));
            acc[1] = fmaf(v.y, q.y, fmaf(v.x, q.x, acc[1]));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xFFFFFFFFu, acc[r], o);
        if (lane == 0 && (r == 0 || two)) sums[slice][2 * pair + r] = acc[r];
      }
    }
    thin_hidden<T, kRank>(a, t, part, group, sums, slices, hidden);
  }
  T* const y = a.y + t.row0 * a.y_stride;
  for (uint64_t c = col0; c < col1; c += kEach * kAdapterThreads) {
    if (c > col0) load_columns(c);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint64_t col = c + e * kAdapterThreads + tid;
      float w = 0.f;
      if (adapts) {
        u[e].settle(second + col * a.second.stride, a.rank);
#pragma unroll
        for (int i = 0; i < kUsed / 2; i += 2) {
          const float4 h = *reinterpret_cast<const float4*>(&hidden[2 * i]);
          const float2 p = u[e].pair(i), q = u[e].pair(i + 1);
          w = fmaf(h.w, q.y, fmaf(h.z, q.x, fmaf(h.y, p.y, fmaf(h.x, p.x, w))));
        }
      }
      if (col < col1) y[col] = from_f32<T>(onto[e] + w);
    }
  }
  if (adapts && a.parts > 1) cluster_wait();  // the others have read this block's sums
}

// The same of the backward pass.  dh = c U^T dy: a column of dy to a thread at a time, its
// row of U times it onto sums of up to 32 ranks, which a warp's lanes put together by halves.
// dx = base + D^T dh: columns of dx to a thread, whose elements of D are neighbours of the
// other threads'.
constexpr int kBackEach = 4;  // columns of dx to a thread at a time
template <class T, int kRank, int kUsed, bool kWhole>
__global__ void __launch_bounds__(kAdapterThreads, 2)
    thin_back_kernel(const __grid_constant__ Chain<T> a) {
  constexpr int kWarps = kAdapterThreads / 32, kMost = 2;
  constexpr int kChunk = kUsed < 32 ? kUsed : 32, kHalves = kUsed / kChunk, kLines = kWarps / kHalves;
  __shared__ __align__(16) float sums[kLines][kRank], hidden[kRank];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const uint32_t part = blockIdx.x % a.parts, group = blockIdx.x / a.parts % a.groups;
  Tile t;
  if (!Tile::find<1>(a.q, blockIdx.x / a.parts / a.groups, t)) return;  // the whole cluster
  const uint64_t col0 = (static_cast<uint64_t>(group) * a.parts + part) * a.group_out;
  const uint64_t col1 = min(col0 + a.group_out, a.out);
  const bool adapts = t.adapter >= 0;
  if (!adapts && a.y == a.base) return;
  if (adapts) {
    const uint64_t in0 = min(part * a.part_in, a.in), in1 = min(in0 + a.part_in, a.in);
    const uint32_t half = warp % kHalves, line = warp / kHalves;
    const int n = min(static_cast<int>(a.rank) - static_cast<int>(half) * kChunk, kChunk);  // ranks; may be below 0
    const T* const first = a.first.data + t.adapter * a.first.step + half * kChunk;
    const T* const x = a.x + t.row0 * a.x_stride;
    float acc[kChunk] = {};
    for (uint64_t c = in0 + line * 32 + lane; c < in1; c += kLines * 32 * kMost) {
      Run<T, kChunk, kWhole> u[kMost];
      float v[kMost];
#pragma unroll
      for (int m = 0; m < kMost; ++m) {
        const uint64_t at = c + m * kLines * 32;
        u[m].load(first + at * a.first.stride, at < in1 ? n : 0);
        v[m] = at < in1 ? to_f32(x[at]) : 0.f;
      }
#pragma unroll
      for (int m = 0; m < kMost; ++m) {
        u[m].settle(first + (c + m * kLines * 32) * a.first.stride, n);
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
          const float2 p = u[m].pair(i);
          acc[2 * i] = fmaf(v[m], p.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(v[m], p.y, acc[2 * i + 1]);
        }
      }
    }
    // every turn half as many sums, of twice as many lanes each
#pragma unroll
    for (int o = 16, left = kChunk; left > 1; o /= 2, left /= 2) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < left / 2; ++i) {
        const float keep = upper ? acc[i + left / 2] : acc[i], send = upper ? acc[i] : acc[i + left / 2];
        acc[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
      }
    }
    for (int o = 32 / kChunk / 2; o > 0; o /= 2) acc[0] += __shfl_xor_sync(0xFFFFFFFFu, acc[0], o);
    if (kUsed < kRank)
      for (uint32_t i = lane + kUsed; i < kRank; i += 32) sums[line][i] = 0.f;
    sums[line][half * kChunk + lane / (32 / kChunk)] = acc[0];
    thin_hidden<T, kRank>(a, t, part, group, sums, kLines, hidden);
  }
  const T* const second = a.second.data + (adapts ? t.adapter * a.second.step : 0);
  const T* const base = a.base + t.row0 * a.base_stride;
  T* const y = a.y + t.row0 * a.y_stride;
  for (uint64_t c = col0 + tid; c < col1; c += kBackEach * kAdapterThreads) {
    float w[kBackEach], onto[kBackEach];
#pragma unroll
    for (int e = 0; e < kBackEach; ++e) {
      const uint64_t col = c + e * kAdapterThreads;
      onto[e] = a.base && col < col1 ? to_f32(base[col]) : 0.f;
      w[e] = 0.f;
    }
    if (adapts) {
#pragma unroll 4
      for (uint32_t r = 0; r < a.rank; ++r) {
        const float h = hidden[r];
#pragma unroll
        for (int e = 0; e < kBackEach; ++e) {
          const uint64_t col = c + e * kAdapterThreads;
          if (col < col1) w[e] = fmaf(h, to_f32(second[r * a.second.stride + col]), w[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kBackEach; ++e) {
      const uint64_t col = c + e * kAdapterThreads;
      if (col < col1) y[col] = from_f32<T>(onto[e] + w[e]);
    }
  }
  if (adapts && a.parts > 1) cluster_wait();  // the others have read this block's sums
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
  const __nv_bfloat16* p[2];  // dh, c h: tokens x planes x kRank
  T* out[2];            // adapters x rank x k, adapters x n x rank
  bool whole[2];
  bool by_request;      // blocks are for the requests' adapters, where these are the fewer
};

// The adapter of a block's place, -1 where another place has it.  All threads call it.
__device__ __forceinline__ int64_t adapter_at(const Requests& q, bool by_request, uint64_t place) {
  if (!by_request) return static_cast<int64_t>(place);
  const int64_t a = q.adapter(place + 1);
  bool earlier = false;
  for (uint64_t s = threadIdx.x; s < place; s += blockDim.x) earlier |= q.adapter(s + 1) == a;
  return __syncthreads_or(earlier) ? -1 : a;
}
// Zeros for the adapters of no request: kFill elements to a block.
constexpr uint32_t kFill = 32768;
template <class T>
__global__ void __launch_bounds__(kAdapterThreads) idle_grads_kernel(const __grid_constant__ Grads<T> a) {
  pdl_trigger();
  pdl_wait();
  const uint64_t all = a.blocks[0] + a.blocks[1], adapter = blockIdx.x / all;
  uint64_t block = blockIdx.x % all;
  const int sel = block >= a.blocks[0];
  if (sel) block -= a.blocks[0];
  bool idle = true;
  for (uint64_t s = threadIdx.x; s < a.q.requests; s += kAdapterThreads)
    idle &= a.q.adapter(s + 1) != static_cast<int64_t>(adapter);
  if (!__syncthreads_and(idle)) return;
  const uint64_t count = a.rank * a.cols[sel];
  T* const out = a.out[sel] + adapter * count + block * kFill;
  const uint32_t n = static_cast<uint32_t>(min(count - block * kFill, static_cast<uint64_t>(kFill)));
  constexpr uint32_t kPer = 16 / sizeof(T);
  const uint32_t head = min(n, static_cast<uint32_t>(-reinterpret_cast<uintptr_t>(out) & 15) / static_cast<uint32_t>(sizeof(T)));
  const uint32_t vecs = (n - head) / kPer, tail = head + vecs * kPer;
  for (uint32_t i = threadIdx.x; i < vecs; i += kAdapterThreads)
    reinterpret_cast<uint4*>(out + head)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < head) out[threadIdx.x] = from_f32<T>(0.f);
  if (threadIdx.x < n - tail) out[tail + threadIdx.x] = from_f32<T>(0.f);
}

// Ranks r0 .. r0 + w - 1 of n columns of a gradient: neighbouring threads write neighbouring
// elements of either layout.
template <class T, int kThreads, class F>
__device__ __forceinline__ void put_grads(const Grads<T>& a, int sel, uint64_t adapter, uint64_t col0, uint32_t n,
                                          int r0, int w, const F& value) {
  if (w <= 0) return;
  const uint64_t cols = a.cols[sel];
  if (!sel) {
    T* const out = a.out[0] + (adapter * a.rank + r0) * cols + col0;
    for (uint32_t r = threadIdx.x / 32; r < static_cast<uint32_t>(w); r += kThreads / 32)
      for (uint32_t c = threadIdx.x % 32; c < n; c += 32) out[r * cols + c] = from_f32<T>(value(r, c));
    return;
  }
  T* const out = a.out[1] + (adapter * cols + col0) * a.rank + r0;
  uint32_t c = threadIdx.x / w, r = threadIdx.x % w;
  const uint32_t on_c = kThreads / w, on_r = kThreads % w;
  while (c < n) {
    out[c * a.rank + r] = from_f32<T>(value(r, c));
    c += on_c;
    r += on_r;
    if (r >= static_cast<uint32_t>(w)) {
      r -= w;
      ++c;
    }
  }
}

// The requests of an adapter among the kAdapterThreads from s0 on, in their order, as one
// list of rows: their first rows, and how many come before theirs.  Returns the rows; all
// threads call it.
__device__ __forceinline__ uint64_t list_rows(const Requests& q, int64_t adapter, uint64_t s0, uint64_t* from,
                                              uint64_t* before, uint64_t* sums_before, uint32_t* counts,
                                              uint32_t& found) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint64_t s = s0 + tid;
  const bool mine = s < q.requests && q.adapter(s + 1) == adapter;
  const uint64_t start = mine ? q.start(s + 1) : 0, end = mine ? q.start(s + 2) : 0;
  const uint64_t length = end > start ? end - start : 0;
  uint64_t upto = length;
  for (int o = 1; o < 32; o *= 2) {
    const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  const uint32_t votes = __ballot_sync(0xFFFFFFFFu, mine);
  if (lane == 31) {
    counts[warp] = __popc(votes);
    sums_before[warp] = upto;
  }
  __syncthreads();
  uint32_t at = __popc(votes & ((1u << lane) - 1));
  uint64_t left = 0, rows = 0;
  found = 0;
  for (uint32_t w = 0; w < kAdapterThreads / 32; ++w) {
    if (w < warp) {
      at += counts[w];
      left += sums_before[w];
    }
    found += counts[w];
    rows += sums_before[w];
  }
  if (mine) {
    from[at] = start;
    before[at] = left + upto - length;
  }
  __syncthreads();
  return rows;
}
// The batch's row of the list's: the last request with no more than `want` before it.
__device__ __forceinline__ uint64_t row_at(const uint64_t* from, const uint64_t* before, uint32_t found, uint64_t want) {
  uint32_t lo = 0, hi = found;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (before[mid] <= want) lo = mid;
    else hi = mid;
  }
  return from[lo] + (want - before[lo]);
}

template <class T, int kRank>
struct GradShape {
  using P = Planes<T>;
  static constexpr int kRows = sizeof(T) == 4 ? 32 : 64, kCols = 128;
  static constexpr int kStages = sizeof(T) == 4 ? 2 : 3;
  static constexpr int kBlocks = sizeof(T) == 4 && kRank == 16 ? 3 : 2;  // of an SM
  static constexpr int kRankWarps = kRank / 16, kColWarps = 8 / kRankWarps, kWarpCols = kCols / kColWarps;
  static constexpr int kRankPitch = kRank + 8, kPitch = kCols + 8;
  static constexpr int kM = kRows * kPitch * static_cast<int>(sizeof(T));
  static constexpr int kP = P::kP * kRows * kRankPitch * 2;
  static constexpr int kStage = kM + kP;
  static constexpr int kSumPitch = kCols + 4;  // threads go along either axis of the sums
  static constexpr int kSums = kRank * kSumPitch * 4;
  static constexpr int kBytes = kStages * kStage > 2 * kSums ? kStages * kStage : 2 * kSums;  // own and joined
};

template <class T, int kRank>
__global__ void __launch_bounds__(kAdapterThreads, GradShape<T, kRank>::kBlocks)
    grads_kernel(const __grid_constant__ Grads<T> a) {
  using S = GradShape<T, kRank>;
  using P = Planes<T>;
  constexpr int kThreads = kAdapterThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  // the adapter's requests: their first rows, and how many rows come before theirs
  __shared__ uint64_t from[kThreads], before[kThreads], sums_before[kThreads / 32];
  __shared__ uint64_t row_of[S::kStages][S::kRows];  // of the batch, for a tile's rows
  __shared__ uint32_t counts[kThreads / 32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank_warp = warp % S::kRankWarps, col_warp = warp / S::kRankWarps;
  pdl_trigger();
  pdl_wait();
  const uint32_t part = blockIdx.x % a.parts;
  const uint64_t all = a.blocks[0] + a.blocks[1];
  const int64_t adapter = adapter_at(a.q, a.by_request, blockIdx.x / a.parts / all);
  if (adapter < 0) return;  // the whole cluster
  uint64_t block = blockIdx.x / a.parts % all;
  const int sel = block >= a.blocks[0];
  if (sel) block -= a.blocks[0];
  const uint64_t col0 = block * S::kCols, cols = a.cols[sel], stride = a.stride[sel];
  const T* const m = a.m[sel] + col0;
  const __nv_bfloat16* const p = a.p[sel];
  const bool whole = a.whole[sel];

  auto load = [&](int stage, int rows) {
    uint8_t* const b = smem + stage * S::kStage;
    constexpr int kLanes = S::kCols / 8, kPass = kThreads / kLanes;
    const int first = tid / kLanes, col = tid % kLanes * 8;
    const int n = static_cast<int>(max(min(static_cast<int64_t>(cols - col0) - col, static_cast<int64_t>(8)), static_cast<int64_t>(0)));
    T* const tile = reinterpret_cast<T*>(b) + first * S::kPitch + col;
    constexpr int kPasses = S::kRows / kPass;
    if (whole) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = first + i * kPass;
        const bool has = row < rows && n > 0;
        copy_eight(tile + i * kPass * S::kPitch, has ? m + row_of[stage][row] * stride + col : m, has ? n : 0);
      }
    } else {
      Shifted<T> v[kPasses];
      const T* at[kPasses];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = first + i * kPass;
        at[i] = row < rows ? m + row_of[stage][row] * stride + col : m;
        v[i].load(at[i], row < rows ? n : 0);
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i) v[i].store(tile + i * kPass * S::kPitch, at[i], first + i * kPass < rows ? n : 0);
    }
    __nv_bfloat16* const planes = reinterpret_cast<__nv_bfloat16*>(b + S::kM);
    constexpr int kChunks = P::kP * S::kRows * kRank / 8;
#pragma unroll
    for (int i = 0; i < (kChunks + kThreads - 1) / kThreads; ++i) {
      const int at = tid + i * kThreads;
      if (kChunks % kThreads && at >= kChunks) break;
      const int row = at / (P::kP * kRank / 8), plane = at / (kRank / 8) % P::kP, c = at % (kRank / 8) * 8;
      const bool there = row < rows;
      copy_16(smem_u32(planes + (plane * S::kRows + row) * S::kRankPitch + c),
              p + (there ? row_of[stage][row] : 0) * (P::kP * kRank) + plane * kRank + c, there ? 16 : 0);
    }
  };
  float acc[S::kWarpCols / 16][2][4] = {};
  int in_stage[S::kStages] = {};  // rows of the tile there
  auto multiply = [&](int stage) {
    int rows = in_stage[0];
#pragma unroll
    for (int i = 1; i < S::kStages; ++i) rows = stage == i ? in_stage[i] : rows;
    const T* const ms = reinterpret_cast<const T*>(smem + stage * S::kStage);
    const __nv_bfloat16* const ps = reinterpret_cast<const __nv_bfloat16*>(smem + stage * S::kStage + S::kM);
#pragma unroll
    for (int t = 0; t < S::kRows; t += 16) {
      if (t >= rows) break;
      uint32_t h[P::kP][4];  // rows of the product are ranks
#pragma unroll
      for (int i = 0; i < P::kP; ++i)
        ldsm_t(h[i], smem_u32(ps + (i * S::kRows + t + lane % 8 + lane / 16 * 8) * S::kRankPitch + rank_warp * 16 + lane / 8 % 2 * 8));
      constexpr int kN = sizeof(T) == 4 ? 1 : S::kWarpCols / 16;
#pragma unroll
      for (int n = 0; n < S::kWarpCols / 16; n += kN) {
        uint32_t w[kN][P::kW][4];
#pragma unroll
        for (int i = 0; i < kN; ++i) cols_operand<T, P::kW, S::kPitch, true>(w[i], ms, col_warp * S::kWarpCols + (n + i) * 16, t);
        add_onto<T, kN, P::kP, P::kW, false>(reinterpret_cast<float(&)[kN][2][4]>(acc[n]), h, w);
      }
    }
  };

  uint64_t tile = 0;  // of the adapter's
  for (uint64_t s0 = 0; s0 < a.q.requests; s0 += kThreads) {
    // (tiles go across requests)
    uint32_t found;
    const uint64_t all_rows = list_rows(a.q, adapter, s0, from, before, sums_before, counts, found);
    // this block's tiles of theirs, the next ones' loads on the way
    uint64_t row = 0;
    auto next = [&](int stage) {  // loads one; false: none left
      while (row < all_rows) {
        const uint64_t row0 = row;
        row += S::kRows;
        if (tile++ % a.parts != part) continue;
        const int rows = static_cast<int>(min(all_rows - row0, static_cast<uint64_t>(S::kRows)));
        if (static_cast<int>(tid) < rows) row_of[stage][tid] = row_at(from, before, found, row0 + tid);
        __syncthreads();
        load(stage, rows);
#pragma unroll
        for (int j = 0; j < S::kStages; ++j) in_stage[j] = stage == j ? rows : in_stage[j];
        return true;
      }
      return false;
    };
    int ahead = 0;  // tiles loaded and not yet multiplied
#pragma unroll
    for (int st = 0; st + 1 < S::kStages; ++st) {
      ahead += next(st);
      copies_end();
    }
    for (int step = 0; ahead; ++step) {
      copies_wait<S::kStages - 2>();
      __syncthreads();
      ahead += next((step + S::kStages - 1) % S::kStages);
      copies_end();
      multiply(step % S::kStages);
      --ahead;
    }
    copies_wait<0>();
    __syncthreads();
  }

  // the parts' sums in a fixed order, and the result
  float* const sums = reinterpret_cast<float*>(smem);  // [rank][kSumPitch]
#pragma unroll
  for (int n = 0; n < S::kWarpCols / 8; ++n)
#pragma unroll
    for (int half = 0; half < 2; ++half)
      *reinterpret_cast<float2*>(sums + (rank_warp * 16 + lane / 4 + half * 8) * S::kSumPitch + col_warp * S::kWarpCols + n * 8 + lane % 4 * 2) =
          make_float2(acc[n / 2][n % 2][half * 2], acc[n / 2][n % 2][half * 2 + 1]);
  // a part's share are whole rows (ranks)
  const int each = kRank / a.parts, r0 = part * each;
  if (a.parts > 1) {
    cluster_meet();
    constexpr int kQuads = S::kCols / 4;
    for (int e = tid; e < each * kQuads; e += kThreads) {
      const uint32_t at = smem_u32(sums + (r0 + e / kQuads) * S::kSumPitch + e % kQuads * 4);
      float4 v = remote_f32x4(at, 0);
      for (uint32_t q = 1; q < a.parts; ++q) v = v + remote_f32x4(at, q);
      reinterpret_cast<float4*>(sums + S::kSums / 4 + e / kQuads * S::kSumPitch)[e % kQuads] = v;
    }
  }
  __syncthreads();
  const float* const total = a.parts > 1 ? sums + S::kSums / 4 : sums;
  put_grads<T, kThreads>(a, sel, adapter, col0, static_cast<uint32_t>(min(cols - col0, static_cast<uint64_t>(S::kCols))), r0,
                         min(each, static_cast<int>(a.rank) - r0),
                         [&](uint32_t r, uint32_t c) { return total[r * S::kSumPitch + c]; });
  if (a.parts > 1) cluster_meet();  // the others stay until their parts are read
}

// The same where adapters have few rows: a column of m to a thread, whose sums over the
// rows stay in its registers; a step takes kRows rows' p through shared memory.
template <class T, int kRank>
struct FewShape {
  static constexpr int kCols = kAdapterThreads, kRows = 16;
  static constexpr int kPitch = kRank + 4 / static_cast<int>(sizeof(T));  // no bank twice
  // columns whose results are put in order at a time
  static constexpr int kTurn = kCols * kPitch * sizeof(T) > 36 * 1024 ? kCols / 2 : kCols;
};
template <class T, int kRank>
__global__ void __launch_bounds__(kAdapterThreads, kRank == 64 ? 2 : kRank == 32 ? 3 : 4)
    few_grads_kernel(const __grid_constant__ Grads<T> a) {
  using S = FewShape<T, kRank>;
  using P = Planes<T>;
  constexpr int kThreads = kAdapterThreads, kRows = S::kRows;
  __shared__ __align__(16) float ps[kRows][kRank];
  __shared__ __align__(16) T results[S::kTurn][S::kPitch];
  __shared__ uint64_t from[kThreads], before[kThreads], sums_before[kThreads / 32], row_of[kRows];
  __shared__ uint32_t counts[kThreads / 32];
  const uint32_t tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const uint64_t all = a.blocks[0] + a.blocks[1];
  const int64_t adapter = adapter_at(a.q, a.by_request, blockIdx.x / all);
  if (adapter < 0) return;
  uint64_t block = blockIdx.x % all;
  const int sel = block >= a.blocks[0];
  if (sel) block -= a.blocks[0];
  const uint64_t col0 = block * S::kCols, cols = a.cols[sel], col = col0 + tid, stride = a.stride[sel];
  const T* const m = a.m[sel] + col;
  const __nv_bfloat16* const p = a.p[sel];
  float acc[kRank] = {};
  for (uint64_t s0 = 0; s0 < a.q.requests; s0 += kThreads) {
    uint32_t found;
    const uint64_t rows = list_rows(a.q, adapter, s0, from, before, sums_before, counts, found);
    for (uint64_t row0 = 0; row0 < rows; row0 += kRows) {
      const int there = static_cast<int>(min(rows - row0, static_cast<uint64_t>(kRows)));
      if (static_cast<int>(tid) < there) row_of[tid] = row_at(from, before, found, row0 + tid);
      __syncthreads();
      constexpr int kBatch = 8;  // rows of m in flight
      float v[kBatch];
      auto load = [&](int at) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = at + i < there && col < cols ? to_f32(m[row_of[at + i] * stride]) : 0.f;
      };
      load(0);
      for (int e = tid; e < there * kRank; e += kThreads) {
        const __nv_bfloat16* const at = p + row_of[e / kRank] * (P::kP * kRank) + e % kRank;
        float sum = 0.f;
#pragma unroll
        for (int i = P::kP - 1; i >= 0; --i) sum += to_f32(at[i * kRank]);
        ps[e / kRank][e % kRank] = sum;
      }
      __syncthreads();
      for (int at = 0; at < there; at += kBatch) {
        if (at) load(at);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (at + i >= there) break;
#pragma unroll
          for (int r = 0; r < kRank; r += 4) {
            const float4 h = *reinterpret_cast<const float4*>(&ps[at + i][r]);
            acc[r] = fmaf(h.x, v[i], acc[r]);
            acc[r + 1] = fmaf(h.y, v[i], acc[r + 1]);
            acc[r + 2] = fmaf(h.z, v[i], acc[r + 2]);
            acc[r + 3] = fmaf(h.w, v[i], acc[r + 3]);
          }
        }
      }
      __syncthreads();
    }
  }
  const int n = static_cast<int>(min(cols - col0, static_cast<uint64_t>(S::kCols)));
  if (!sel) {
    T* const out = a.out[0] + adapter * a.rank * cols + col;
#pragma unroll
    for (int r = 0; r < kRank; ++r)
      if (r < static_cast<int>(a.rank) && col < cols) out[r * cols] = from_f32<T>(acc[r]);
    return;
  }
  // the block's columns of the second gradient lie together
#pragma unroll
  for (int c0 = 0; c0 < S::kCols; c0 += S::kTurn) {
    if (c0) __syncthreads();
    const int mine = static_cast<int>(tid) - c0;
    if (mine >= 0 && mine < S::kTurn)
#pragma unroll
      for (int r = 0; r < kRank; ++r) results[mine][r] = from_f32<T>(acc[r]);
    __syncthreads();
    T* const out = a.out[1] + (adapter * cols + col0 + c0) * a.rank;
    auto put = [&](auto* to, uint32_t w) {  // w elements (or pairs) to a column
      using V = std::remove_reference_t<decltype(*to)>;
      uint32_t c = tid / w, r = tid % w;
      const uint32_t on_c = kThreads / w, on_r = kThreads % w, end = max(min(n - c0, S::kTurn), 0);
      for (uint32_t e = tid; c < end; e += kThreads) {
        to[e] = reinterpret_cast<const V*>(results[c])[r];
        c += on_c;
        r += on_r;
        if (r >= w) {
          r -= w;
          ++c;
        }
      }
    };
    if (sizeof(T) == 2 && a.rank % 2 == 0 && reinterpret_cast<uintptr_t>(out) % 4 == 0)
      put(reinterpret_cast<uint32_t*>(out), a.rank / 2);
    else
      put(out, a.rank);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <auto kKernel, class... A>
cudaError_t launch_clusters(uint64_t blocks, uint32_t parts, int threads, int smem, cudaStream_t st, const A&... args) {
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  if (smem > 40 * 1024) {  // static shared memory counts too; once for each device
    static std::atomic<uint64_t> allowed{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
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
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

// adapter_f32.cu, adapter_bf16.cu, adapter_f16.cu
template <class T>
cudaError_t run_chain(const Chain<T>& a, bool back, cudaStream_t st);
template <class T>
cudaError_t run_grads(const Grads<T>& a, cudaStream_t st);
// Bounded waits of theirs that ran out, of the types that have any.
template <class T>
cudaError_t adapter_wait_timeouts(uint64_t* count);

}  // namespace hkv
