// adapter_bf16.cu -- the adapters' kernels on __nv_bfloat16 matrices.
#include "adapter_launch.cuh"

namespace hkv {

template <>
cudaError_t run_chain<__nv_bfloat16>(const Chain<__nv_bfloat16>& a, bool back, cudaStream_t st) {
  return back ? chain<__nv_bfloat16, true>(a, st) : chain<__nv_bfloat16, false>(a, st);
}
template <>
cudaError_t run_grads<__nv_bfloat16>(const Grads<__nv_bfloat16>& a, cudaStream_t st) {
  return grads<__nv_bfloat16>(a, st);
}

template <>
cudaError_t adapter_wait_timeouts<__nv_bfloat16>(uint64_t* count) {
  return tensor::wait_timeouts(count);
}

}  // namespace hkv
