// adapter_f16.cu -- the adapters' kernels on __half matrices.
#include "adapter_launch.cuh"

namespace hkv {

template <>
cudaError_t run_chain<__half>(const Chain<__half>& a, bool back, cudaStream_t st) {
  return back ? chain<__half, true>(a, st) : chain<__half, false>(a, st);
}
template <>
cudaError_t run_grads<__half>(const Grads<__half>& a, cudaStream_t st) {
  return grads<__half>(a, st);
}

template <>
cudaError_t adapter_wait_timeouts<__half>(uint64_t* count) {
  return tensor::wait_timeouts(count);
}

}  // namespace hkv
