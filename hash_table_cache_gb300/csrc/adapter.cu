// adapter.cu -- hkv_adapter_matmul and hkv_adapter_matmul_backward: arguments and
// launches (the kernels are in adapter.cuh).
#include "adapter.cuh"

namespace hkv {
namespace {

constexpr uint64_t kMaxStride = 1ull << 31, kMaxStep = 1ull << 40;  // byte offsets stay within 64 bits

bool matrix_ok(const Matrix& m) {
  return m.stride >= m.cols && m.stride <= kMaxStride && (m.rows == 0 || (m.p && aligned(m.p, m.size)));
}
bool whole(const Matrix& m) { return aligned(m.p, 16) && m.stride * m.size % 16 == 0; }
bool same(const Matrix& a, const Matrix& b) { return a.p == b.p && a.stride == b.stride; }
// What a call writes without gaps: h or dh of all rows, and the gradient of `rows` x `cols`
// matrices of all adapters (more than any memory where the bytes pass 64 bits).
Matrix hidden_run(const void* p, uint64_t tokens, uint32_t rank, int type) {
  return run_of(p, HKV_ADAPTER_HIDDEN_BYTES(tokens, rank, type));
}
Matrix grad_run(const void* p, const hkv_adapters& w, uint64_t cols, size_t size) {
  const uint64_t rows = p ? w.count * w.rank : 0, most = 1ull << 60;
  return run_of(p, rows && cols * size > most / rows ? most : rows * cols * size);
}
template <class... M>
bool run_meets_any(const Matrix& run, const M&... others) { return (run_meets(run, others) || ...); }

bool requests_ok(uint64_t tokens, uint64_t requests, const int64_t* offsets, const int64_t* which) {
  return tokens <= HKV_MAX_BATCH && requests <= HKV_MAX_BATCH &&
         (requests == 0 || (offsets && which)) && aligned(offsets, 8) && aligned(which, 8);
}

bool adapters_ok(const hkv_adapters* a, uint64_t k, uint64_t n, int type) {
  if (!a || a->count > HKV_MAX_BATCH || a->rank < 1 || a->rank > HKV_MAX_RANK) return false;
  if (a->down_stride < k || a->up_stride < a->rank) return false;
  if (a->down_stride > kMaxStride || a->up_stride > kMaxStride) return false;
  if (a->down_step > kMaxStep || a->up_step > kMaxStep) return false;
  if (a->count && (!a->down || !a->up)) return false;
  return aligned(a->down, type_size(type)) && aligned(a->up, type_size(type)) && aligned(a->scales, 4);
}

template <class T>
Factor<T> factor(const void* p, uint64_t step, uint64_t stride) {
  return {static_cast<const T*>(p), step, stride,
          aligned(p, 16) && step * sizeof(T) % 16 == 0 && stride * sizeof(T) % 16 == 0};
}

// y = base + c second (first x), or the same the other way through the adapters.
cudaError_t run(bool back, int type, const Requests& q, const hkv_adapters& w, const Matrix& x,
                const Matrix& base, const Matrix& y, void* hidden, cudaStream_t st) {
  return with_type(type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const Factor<T> down = factor<T>(w.down, w.down_step, w.down_stride);
    const Factor<T> up = factor<T>(w.up, w.up_step, w.up_stride);
    Chain<T> c{};
    c.q = q;
    c.in = x.cols;
    c.out = y.cols;
    c.rank = w.rank;
    c.x = static_cast<const T*>(x.p);
    c.x_stride = x.stride;
    c.first = back ? up : down;
    c.second = back ? down : up;
    c.base = static_cast<const T*>(base.p);
    c.base_stride = base.stride;
    c.y = static_cast<T*>(const_cast<void*>(y.p));
    c.y_stride = y.stride;
    c.hidden = static_cast<__nv_bfloat16*>(hidden);
    c.x_whole = whole(x);
    c.base_whole = whole(base);
    c.y_whole = whole(y);
    return run_chain(c, back, st);
  });
}

}  // namespace
}  // namespace hkv

extern "C" {

hkv_status hkv_adapter_matmul(uint64_t tokens, uint64_t k, uint64_t n, int type,
                              const hkv_adapters* adapters, uint64_t requests,
                              const int64_t* offsets, const int64_t* which, const void* x,
                              uint64_t x_stride, const void* base, uint64_t base_stride, void* y,
                              uint64_t y_stride, void* hidden, void* stream) {
  using namespace hkv;
  if (!type_ok(type) || k < 1 || n < 1 || k > HKV_MAX_BATCH || n > HKV_MAX_BATCH) return HKV_ERR_INVALID;
  if (!requests_ok(tokens, requests, offsets, which) || !adapters_ok(adapters, k, n, type))
    return HKV_ERR_INVALID;
  const size_t size = type_size(type);
  const Matrix mx{x, tokens, k, x_stride, size}, my{y, tokens, n, y_stride, size};
  const Matrix mb{base, base ? tokens : 0, n, base ? base_stride : n, size};
  if (!matrix_ok(mx) || !matrix_ok(my) || !matrix_ok(mb)) return HKV_ERR_INVALID;
  if ((tokens && !hidden) || !aligned(hidden, 16)) return HKV_ERR_INVALID;
  if (meet(my, mx) || (meet(my, mb) && !same(my, mb))) return HKV_ERR_INVALID;
  if (run_meets_any(hidden_run(hidden, tokens, adapters->rank, type), mx, mb, my)) return HKV_ERR_INVALID;
  if (tokens == 0) return HKV_OK;
  const Requests q{tokens, requests, adapters->count, offsets, which, adapters->scales};
  return op_status(run(false, type, q, *adapters, mx, mb, my, hidden, static_cast<cudaStream_t>(stream)));
}

hkv_status hkv_adapter_matmul_backward(uint64_t tokens, uint64_t k, uint64_t n, int type,
                                       const hkv_adapters* adapters, uint64_t requests,
                                       const int64_t* offsets, const int64_t* which, const void* x,
                                       uint64_t x_stride, const void* dy, uint64_t dy_stride,
                                       const void* hidden, const void* base, uint64_t base_stride,
                                       void* dx, uint64_t dx_stride, void* ddown, void* dup,
                                       void* dhidden, void* stream) {
  using namespace hkv;
  if (!type_ok(type) || k < 1 || n < 1 || k > HKV_MAX_BATCH || n > HKV_MAX_BATCH) return HKV_ERR_INVALID;
  if (!requests_ok(tokens, requests, offsets, which) || !adapters_ok(adapters, k, n, type))
    return HKV_ERR_INVALID;
  const size_t size = type_size(type);
  const Matrix mx{x, tokens, k, x_stride, size}, md{dy, tokens, n, dy_stride, size};
  const Matrix mdx{dx, tokens, k, dx_stride, size};
  const Matrix mb{base, base ? tokens : 0, k, base ? base_stride : k, size};
  if (!matrix_ok(mx) || !matrix_ok(md) || !matrix_ok(mdx) || !matrix_ok(mb)) return HKV_ERR_INVALID;
  if (tokens && (!hidden || !dhidden)) return HKV_ERR_INVALID;
  if (!aligned(hidden, 16) || !aligned(dhidden, 16) || !aligned(ddown, size) || !aligned(dup, size))
    return HKV_ERR_INVALID;
  if (meet(mdx, mx) || meet(mdx, md) || (meet(mdx, mb) && !same(mdx, mb))) return HKV_ERR_INVALID;
  const Matrix rh = hidden_run(hidden, tokens, adapters->rank, type), rdh = hidden_run(dhidden, tokens, adapters->rank, type);
  const Matrix rd = grad_run(ddown, *adapters, k, size), ru = grad_run(dup, *adapters, n, size);
  if (run_meets(rh, mdx) || run_meets_any(rdh, mx, md, mb, mdx, rh) || run_meets_any(rd, mx, md, mb, mdx, rh, rdh) ||
      run_meets_any(ru, mx, md, mb, mdx, rh, rdh, rd))
    return HKV_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Requests q{tokens, requests, adapters->count, offsets, which, adapters->scales};
  cudaError_t e = cudaSuccess;
  if (tokens) e = run(true, type, q, *adapters, md, mb, mdx, dhidden, st);
  if (e == cudaSuccess && adapters->count && (ddown || dup))
    e = with_type(type, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      Grads<T> g{};
      g.q = q;
      g.rank = adapters->rank;
      g.cols[0] = k;
      g.cols[1] = n;
      g.m[0] = static_cast<const T*>(x);
      g.m[1] = static_cast<const T*>(dy);
      g.stride[0] = x_stride;
      g.stride[1] = dy_stride;
      g.p[0] = static_cast<const __nv_bfloat16*>(dhidden);
      g.p[1] = static_cast<const __nv_bfloat16*>(hidden);
      g.out[0] = static_cast<T*>(ddown);
      g.out[1] = static_cast<T*>(dup);
      g.whole[0] = whole(mx);
      g.whole[1] = whole(md);
      return run_grads(g, st);
    });
  return op_status(e);
}

}  // extern "C"
