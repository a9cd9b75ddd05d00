// adapter_launch.cuh -- which of the adapters' kernels a call takes, and their launches.
//
// Times of one call (GB300, bfloat16 unless said, CUDA graph replays; "base" and y in
// memory, adapters in L2):
//   one row, 4096 to 4096, rank 16                                4.2 us
//   256 requests of one row, 64 adapters                          12 us
//   7883 rows of 24 requests, 4096 to 8192, rank 32               67 us, 4.9 TB/s
//   1447 rows of 16 requests, 64 to 131072, rank 8               132 us, 6.0 TB/s
//   7935 rows of 32 requests, 4096 to 4096, rank 64               56 us, 3.5 TB/s
//     and its backward pass                                       90 us: dx 56, gradients 34
//   7935 rows as above, float16                                   88 and 203 us (mma.sync but
//     for the forward call's and the backward call's first product)
//   and float32                                                 227 and 435 us (six products)
//   3905 rows of 333 requests, 128 to 128, rank 8, float32        10 and 20 us
//
// The lengths and the requests' adapters are on the device, so that the rules know how many
// rows, requests and adapters there are, and no more: what they say of "rows to a request"
// and "to an adapter" is the mean, and their figures are of equal lengths.  Uneven batches come
// out as well, but slower (forward and backward; 2048 to 2048 by rank 16):
//   a prompt of 500 rows and 255 single rows, by row              23 and 140 us
//     the two alone                                               10 and 25, 10 and 20
//   of 8192 rows, 4096 to 4096, in tiles of 64                    70 and 160
//     the two alone                                               47 and 90, 14 and 33
//   300 requests of 13 rows by one of 256 adapters                34 and 796
//     spread over them, or by one of one                          34 and 89, 34 and 88
//   3800 rows of one of 256 adapters, one of each other           33 and 812
// Every block of the gradients reads all requests' adapters: an adapter each for 333, 1024,
// 8192 and 32768 requests of a row, 128 to 128 by rank 8, float32, takes 15, 37, 992 and
// 14085 us backward.
#pragma once

#include "adapter_tensor.cuh"

namespace hkv {

// Long requests: tiles of 64 rows, the two products one after the other.
template <class T, int kRank, bool kBack>
cudaError_t launch_long(Chain<T> a, cudaStream_t st) {
  constexpr int kTile = 64;
  using F = FirstShape<T, kRank, kTile, kBack>;
  using S = SecondShape<T, kRank, kTile, kBack>;
  const uint64_t slots = slots_of(a.q.tokens, a.q.requests, kTile);
  const uint64_t tiles = a.q.tokens / kTile + a.q.requests + 1;
  a.follows = a.q.requests > 0 && a.q.adapters > 0;  // else all rows are base's
  if (a.follows) {
    bool by_tensor = false;
    int bytes = F::kBytes;
    tensor::Maps maps{};
    if constexpr (sizeof(T) == 2) {
      by_tensor = tensor::make_maps<T, kRank, kBack>(&maps, a);
      if (by_tensor) bytes = tensor::Shape<kRank>::kBytes;
    }
    // Clusters share a tile's columns, 512 to a block at least, while all blocks are on
    // the SMs at once (estimated by shared memory, and from the tiles that the requests
    // can have).  Half and twice as many blocks: 7935 rows by rank 64 with the second
    // product 66 and 65 us against 61, 7883 rows by rank 32 73 and 74 against 70.  Float32,
    // whose products are most of the time, twice as many: by rank 64 227 us against 340.
    const uint64_t room = (sizeof(T) == 4 ? 2 : 1) * sm_count() * (227ull * 1024 / (bytes + 1024));
    a.parts = 1;
    while (a.parts < kAdapterParts && a.in >= 512ull * a.parts && 2 * tiles * a.parts <= room) a.parts *= 2;
    a.part_in = ((a.in + a.parts - 1) / a.parts + 63) / 64 * 64;
    cudaError_t e = cudaSuccess;
    if (!by_tensor)
      e = launch_clusters<first_kernel<T, kRank, kTile, kBack>>(slots * a.parts, a.parts, kAdapterThreads, bytes, st, a);
    else if constexpr (sizeof(T) == 2)
      e = launch_clusters<tensor::first_tensor_kernel<T, kRank, kBack>>(slots * a.parts, a.parts,
                                                                        tensor::Shape<kRank>::kThreads, bytes, st, maps, a);
    if (e != cudaSuccess) return e;
  }
  // Eight blocks for every SM, of up to 16 stages of columns.  Four and twelve: 7935 rows
  // by rank 64 59 and 62 us against 56.
  const uint64_t steps = (a.out + S::kCols - 1) / S::kCols, blocks = 8ull * sm_count();
  const uint64_t each = (tiles * steps + blocks - 1) / blocks > 16 ? 16 : (tiles * steps + blocks - 1) / blocks;
  a.groups = static_cast<uint32_t>((steps + each - 1) / each);
  a.group_out = each * S::kCols;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    tensor::SecondMaps maps{};
    if (a.follows && tensor::make_maps<kRank, kBack>(&maps, a))
      return launch_clusters<tensor::second_tensor_kernel<kRank, kBack>>(
          slots * a.groups, 1, tensor::SecondShape<kRank>::kThreads, tensor::SecondShape<kRank>::kBytes, st, maps, a);
  }
  return launch_clusters<second_kernel<T, kRank, kTile, kBack>>(slots * a.groups, 1, kAdapterThreads, S::kBytes, st, a);
}

// Few rows to a request: one kernel, clusters while there are no more than two blocks for
// an SM (256 rows of 4096 by rank 16: 12 us; four 25, eight 35), and several clusters to a
// tile where its columns of y are many: of single rows as many as are on the SMs at once (64
// rows of 4096 7 us and more of them 11, 128 of 512 to 8192 by rank 8 9 and 13), of tiles more
// than that (float32, 100 requests of 16 rows, 512 to 8192 by rank 16, 84 us and fewer 102).
template <auto kKernel, class T>
cudaError_t launch_few(Chain<T> a, uint64_t slots, uint64_t tiles, uint64_t cols, bool at_once, int smem,
                       cudaStream_t st) {
  const uint64_t room = 2ull * sm_count();
  a.parts = 1;
  while (a.parts < kAdapterParts && 2 * tiles * a.parts <= room && (a.in >= 256ull * a.parts || a.out > cols * a.parts))
    a.parts *= 2;
  a.part_in = ((a.in + a.parts - 1) / a.parts + 63) / 64 * 64;
  const uint64_t most = (a.out + cols * a.parts - 1) / (cols * a.parts);
  uint64_t groups = (room + (at_once ? 0 : tiles * a.parts - 1)) / (tiles * a.parts);
  if (groups == 0) groups = 1;
  // every group has the first product anew
  if (groups > 1 + a.out / a.in) groups = 1 + a.out / a.in;
  if (groups > most) groups = most;
  a.groups = static_cast<uint32_t>(groups);
  a.group_out = ((a.out + groups * a.parts - 1) / (groups * a.parts) + 31) / 32 * 32;
  return launch_clusters<kKernel>(slots * groups * a.parts, a.parts, kAdapterThreads, smem, st, a);
}

// (For eight ranks at most: 465 float32 requests of 2 rows, 29 to 19637 by rank 2, 90 us and
// with sixteen 136; 302 float16 ones of 3, 1163 to 12920, by rank 8 48 us and by rank 10 78.)
template <class T, int kRank, int kUsed, bool kBack>
cudaError_t launch_thin(const Chain<T>& a, cudaStream_t st) {
  const uint64_t tokens = a.q.tokens, slots = slots_of(tokens, a.q.requests, 1);
  if constexpr (kBack) {
    constexpr int kCols = kBackEach * kAdapterThreads;
    return a.first.whole && a.rank % 8 == 0
               ? launch_few<thin_back_kernel<T, kRank, kUsed, true>>(a, slots, tokens, kCols, true, 0, st)
               : launch_few<thin_back_kernel<T, kRank, kUsed, false>>(a, slots, tokens, kCols, true, 0, st);
  } else {
    constexpr int kCols = thin_columns<T, kUsed>() * kAdapterThreads;
    return a.x_whole && a.first.whole && a.second.whole && a.in % 8 == 0 && a.rank % 8 == 0
               ? launch_few<thin_kernel<T, kRank, kUsed, true>>(a, slots, tokens, kCols, true, 0, st)
               : launch_few<thin_kernel<T, kRank, kUsed, false>>(a, slots, tokens, kCols, true, 0, st);
  }
}

template <class T, int kRank, bool kBack>
cudaError_t chain_of(const Chain<T>& a, cudaStream_t st) {
  const uint64_t tokens = a.q.tokens, requests = a.q.requests;
  // Few rows to a request, by row: factors are read once for each, past shared memory.  With
  // rows alone and in tiles of 16, bfloat16, 2048 to 2048: 128 requests of 1 row by rank 16 8
  // and 17 us (backward 9 and 19), of 4 14 and 21 (14 and 24), of 8 23 and 22 (22 and 20), but
  // 512 requests of 2 rows 21 and 30 (19 and 35), of 4 39 and 30 (32 and 35), of 6 58 and 31;
  // by rank 64 128 of 1 row 25 and 40 (19 and 39), of 4 47 and 31, 512 of 2 81 and 78 (84 and
  // 76; float32 150 and 184).  Rows that start anywhere, 450 rows of 5437 to 2437 by rank 8: 23
  // and 93.  Up to eight ranks, whose tiles are half empty, 300 requests of 8 rows, 512 to 8192
  // 60 and 68 us (float32 81 and 132), of 12 120 and 71 (126 and 152), but 512 of 6 rows, 2048
  // to 2048, 43 and 33 (backward 35 and 39).
  const bool half_empty = a.rank <= 8 && (sizeof(T) == 4 || kBack || a.out >= 4 * a.in);
  const uint64_t most = kRank > 16 ? 2 : half_empty ? 8 : 4;
  if (tokens <= most * requests || (kRank * tokens <= 16384 && kRank * tokens <= 128 * requests)) {
    if constexpr (kRank == 16)
      if (a.rank <= 8) return launch_thin<T, kRank, 8, kBack>(a, st);
    return launch_thin<T, kRank, kRank, kBack>(a, st);
  }
  // Few rows: with tiles of 16 and of 64 rows, bfloat16, 2048 to 2048 by rank 16, forward:
  // 341 requests of 12 30.0 and 33.9 us, 256 of 16 29.7 and 32.3, 204 of 20 29.2 and 28.0, 128
  // of 32 29.4 and 27.2; 170 of 12, 1024 to 1024 by rank 64, 27.0 and 22.1.
  if (tokens < 20 * requests) {
    return launch_few<short_kernel<T, kRank, kBack>>(a, slots_of(tokens, requests, 16), tokens / 16 + requests + 1,
                                                     SecondShape<T, kRank, 16, kBack>::kCols, false,
                                                     ShortShape<T, kRank, kBack>::kBytes, st);
  }
  return launch_long<T, kRank, kBack>(a, st);
}
template <class T, bool kBack>
cudaError_t chain(const Chain<T>& a, cudaStream_t st) {
  return a.rank <= 16 ? chain_of<T, 16, kBack>(a, st)
         : a.rank <= 32 ? chain_of<T, 32, kBack>(a, st) : chain_of<T, 64, kBack>(a, st);
}

template <class T, int kRank>
cudaError_t launch_grads(Grads<T> a, cudaStream_t st) {
  using S = GradShape<T, kRank>;
  // More adapters than requests: blocks for the requests' ones, zeros for the others.
  a.by_request = a.q.requests < a.q.adapters;
  const uint64_t places = a.by_request ? a.q.requests : a.q.adapters;
  if (a.by_request) {
    for (int i = 0; i < 2; ++i) a.blocks[i] = a.out[i] ? (a.rank * a.cols[i] + kFill - 1) / kFill : 0;
    const uint64_t blocks = a.q.adapters * (a.blocks[0] + a.blocks[1]);
    if (blocks) {
      const cudaError_t e = launch_clusters<idle_grads_kernel<T>>(blocks, 1, kAdapterThreads, 0, st, a);
      if (e != cudaSuccess) return e;
    }
  }
  // Few rows to an adapter: 128 adapters, 2048 to 2048, bfloat16, of 1 row by rank 16 14 us
  // where tiles of 64 rows take 57, of 16 rows 27 and 58; 32 adapters of 16 rows 11 and 19, of
  // 64 rows 33 and 19.  (Adapters without rows: 191 of rank 5, 1599 to 1933, 9.5 and 48.)
  if (a.q.tokens <= 16 * places) {
    constexpr int kCols = FewShape<T, kRank>::kCols;
    for (int i = 0; i < 2; ++i) a.blocks[i] = a.out[i] ? (a.cols[i] + kCols - 1) / kCols : 0;
    const uint64_t blocks = places * (a.blocks[0] + a.blocks[1]);
    return blocks ? launch_clusters<few_grads_kernel<T, kRank>>(blocks, 1, kAdapterThreads, 0, st, a) : cudaSuccess;
  }
  a.blocks[0] = a.out[0] ? (a.cols[0] + S::kCols - 1) / S::kCols : 0;
  a.blocks[1] = a.out[1] ? (a.cols[1] + S::kCols - 1) / S::kCols : 0;
  const uint64_t blocks = places * (a.blocks[0] + a.blocks[1]);
  if (!blocks) return cudaSuccess;
  // Clusters share an adapter's rows, two tiles to a block at least, up to two blocks for
  // an SM (7935 rows, 4 adapters of rank 64 and 4096 to 4096: 33 us; one 45, four 46).  Of
  // sixteen blocks: 17000 rows of one adapter of rank 43, 480 to 721, 83 us and of eight 122.
  a.parts = 1;
  while (a.parts < kGradParts && blocks * a.parts < 2ull * sm_count() && a.q.tokens >= 128ull * a.parts) a.parts *= 2;
  // (TMA takes rows that follow one another: requests of 32 rows and more)
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    tensor::GradMaps maps{};
    if (a.q.tokens >= 32 * a.q.requests && a.q.requests && tensor::make_maps<kRank>(&maps, a)) {
      while (a.parts > kAdapterParts || a.parts > kRank / 4) a.parts /= 2;  // four ranks to a part at least
      return launch_clusters<tensor::grads_tensor_kernel<kRank>>(blocks * a.parts, a.parts, tensor::GradShape<kRank>::kThreads,
                                                                 tensor::GradShape<kRank>::kBytes, st, maps, a);
    }
  }
  return launch_clusters<grads_kernel<T, kRank>>(blocks * a.parts, a.parts, kAdapterThreads, S::kBytes, st, a);
}
template <class T>
cudaError_t grads(const Grads<T>& a, cudaStream_t st) {
  return a.rank <= 16 ? launch_grads<T, 16>(a, st) : a.rank <= 32 ? launch_grads<T, 32>(a, st) : launch_grads<T, 64>(a, st);
}

}  // namespace hkv
