// adapter_f32.cu -- the adapters' kernels on float matrices.
#include "adapter_launch.cuh"

namespace hkv {

template <>
cudaError_t run_chain<float>(const Chain<float>& a, bool back, cudaStream_t st) {
  return back ? chain<float, true>(a, st) : chain<float, false>(a, st);
}
template <>
cudaError_t run_grads<float>(const Grads<float>& a, cudaStream_t st) {
  return grads<float>(a, st);
}

template <>
cudaError_t adapter_wait_timeouts<float>(uint64_t* count) {
  return tensor::wait_timeouts(count);
}

}  // namespace hkv
