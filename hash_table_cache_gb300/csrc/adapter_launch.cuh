// adapter_launch.cuh -- which of the adapters' kernels a call takes, and their launches.
#pragma once

#include "adapter_tensor.cuh"

#ifndef HKV_TENSOR3
#define HKV_TENSOR3 1
#endif
#ifndef HKV_GT
#define HKV_GT 1
#endif
#ifndef HKV_TENSOR2
#define HKV_TENSOR2 1
#endif
#ifndef HKV_TENSOR
#define HKV_TENSOR 1
#endif

namespace hkv {

template <class T, int kRank, int kTile, bool kBack>
cudaError_t launch_chain(Chain<T> a, cudaStream_t st) {
  using F = FirstShape<T, kRank, kTile, kBack>;
  using S = SecondShape<T, kRank, kTile, kBack>;
  const uint64_t slots = slots_of(a.q.tokens, a.q.requests, kTile);
  const uint64_t tiles = a.q.tokens / kTile + (a.q.requests < a.q.tokens ? a.q.requests : a.q.tokens) + 1;
  a.parts = 1;
  a.follows = a.q.requests > 0 && a.q.adapters > 0;
  bool by_tensor = false;
  int bytes = F::kBytes;
  tensor::Maps maps{};
  if constexpr (sizeof(T) == 2) {
    by_tensor = HKV_TENSOR && a.follows && tensor::make_maps<T, kRank, kBack>(&maps, a);
    if (by_tensor) bytes = tensor::Shape<kRank>::kBytes;
  }
  // all blocks at once on the SMs, each with four stages of 128 columns at least
  const uint64_t room = sm_count() * (HKV_PM * 227ull * 1024 / (bytes + 1024)) / 100;
  while (a.parts < kAdapterParts && a.in >= 512ull * a.parts && 2 * tiles * a.parts <= room) a.parts *= 2;
  a.part_in = ((a.in + a.parts - 1) / a.parts + 63) / 64 * 64;
  if (a.follows) {  // (else all rows are base's)
    cudaError_t e = cudaSuccess;
    if constexpr (sizeof(T) == 2) {
      if (by_tensor)
        e = launch_clusters<tensor::first_tensor_kernel<T, kRank, kBack>>(slots * a.parts, a.parts, tensor::Shape<kRank>::kThreads,
                                                                          bytes, st, maps, a);
    }
    if (!by_tensor) e = launch_clusters<first_kernel<T, kRank, kTile, kBack>>(slots * a.parts, a.parts, kAdapterThreads, F::kBytes, st, a);
    if (e != cudaSuccess) return e;
  }
  // blocks for every SM several times over, of up to eight stages
  uint64_t steps = (a.out + S::kCols - 1) / S::kCols, each = (tiles * steps + HKV_GM * 1ull * sm_count() - 1) / (HKV_GM * 1ull * sm_count());
  if (each > HKV_EM) each = HKV_EM;
  a.groups = static_cast<uint32_t>((steps + each - 1) / each);
  a.group_out = each * S::kCols;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    tensor::SecondMaps maps{};
    if (HKV_TENSOR2 && a.follows && tensor::make_maps<kRank, kBack>(&maps, a))
      return launch_clusters<tensor::second_tensor_kernel<kRank, kBack>>(
          slots * a.groups, 1, tensor::SecondShape<kRank>::kThreads, tensor::SecondShape<kRank>::kBytes, st, maps, a);
  }
  return launch_clusters<second_kernel<T, kRank, kTile, kBack>>(slots * a.groups, 1, kAdapterThreads, S::kBytes, st, a);
}

// Few rows: one kernel, clusters of as many blocks as fill the SMs, and several
// clusters to a tile where its columns of y are many.
template <auto kKernel, class T>
cudaError_t launch_few(Chain<T> a, uint64_t slots, uint64_t tiles, uint64_t cols, int smem, cudaStream_t st) {
  const uint64_t room = HKV_ROOM * sm_count();
  a.parts = 1;
  while (a.parts < kAdapterParts && 2 * tiles * a.parts <= room && (a.in >= 256ull * a.parts || a.out > cols * a.parts)) a.parts *= 2;
  a.part_in = ((a.in + a.parts - 1) / a.parts + 63) / 64 * 64;
  const uint64_t most = (a.out + cols * a.parts - 1) / (cols * a.parts);
  uint64_t groups = (room + tiles * a.parts - 1) / (tiles * a.parts);
  // every group has the first product anew
  if (groups > 1 + a.out / a.in) groups = 1 + a.out / a.in;
  if (groups > most) groups = most;
  a.groups = static_cast<uint32_t>(groups);
  a.group_out = ((a.out + groups * a.parts - 1) / (groups * a.parts) + 31) / 32 * 32;
  return launch_clusters<kKernel>(slots * groups * a.parts, a.parts, kAdapterThreads, smem, st, a);
}

template <class T, int kRank, bool kBack>
cudaError_t chain_of(const Chain<T>& a, cudaStream_t st) {
  const uint64_t tokens = a.q.tokens, requests = a.q.requests;
  if constexpr (!kBack)
    if (tokens <= requests && a.x_whole && a.first.whole && a.second.whole && a.in % 8 == 0 && a.rank % 8 == 0)
      return launch_few<thin_kernel<T, kRank>>(a, slots_of(tokens, requests, 1), tokens, thin_columns<T, kRank>() * kAdapterThreads, 0, st);
  if (tokens < 32 * requests)
    return launch_few<short_kernel<T, kRank, kBack>>(a, slots_of(tokens, requests, 16), tokens / 16 + (requests < tokens ? requests : tokens) + 1,
                                                     SecondShape<T, kRank, 16, kBack>::kCols, ShortShape<T, kRank, kBack>::kBytes, st);
  return launch_chain<T, kRank, 64, kBack>(a, st);
}
template <class T, bool kBack>
cudaError_t chain(const Chain<T>& a, cudaStream_t st) {
  return a.rank <= 16 ? chain_of<T, 16, kBack>(a, st) : a.rank <= 32 ? chain_of<T, 32, kBack>(a, st) : chain_of<T, 64, kBack>(a, st);
}

template <class T, int kRank>
cudaError_t launch_grads(Grads<T> a, cudaStream_t st) {
  using S = GradShape<T, kRank>;
  a.blocks[0] = a.out[0] ? (a.cols[0] + S::kCols - 1) / S::kCols : 0;
  a.blocks[1] = a.out[1] ? (a.cols[1] + S::kCols - 1) / S::kCols : 0;
  const uint64_t blocks = a.q.adapters * (a.blocks[0] + a.blocks[1]);
  if (!blocks) return cudaSuccess;
  a.parts = 1;
  while (a.parts < kAdapterParts && blocks * a.parts < HKV_GP * 1ull * sm_count() &&
         a.q.tokens >= 2ull * a.parts * S::kRows)
    a.parts *= 2;  // (kRank is a multiple of it)
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    tensor::GradMaps maps{};
    if (HKV_TENSOR3 && a.q.requests && a.q.tokens >= HKV_GT * a.q.requests && tensor::make_maps<kRank>(&maps, a)) {
      if (a.parts > kRank / 4) a.parts = kRank / 4;  // four ranks to a part at least
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
