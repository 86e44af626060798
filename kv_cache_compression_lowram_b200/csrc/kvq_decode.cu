// Quantised KV cache: attention of the last tokens over whole sequences.
//
// Simple form: one CTA per (layer, sequence, query token, query head), one pass over the
// tokens with the running maximum and sum of the softmax.
#include "kvq.cuh"
#include "kvq_simple.cuh"

namespace lowram {
namespace kvq {
namespace {

template <typename T, int BITS, int D>
__global__ void __launch_bounds__(kSimpleThreads) decode_kernel(Args a, const T* __restrict__ q, const int32_t* __restrict__ lens,
                                                                T* __restrict__ out) {
  const unsigned x = blockIdx.x;   // ((layer * B + b) * n + i) * Hq + j
  const int j = x % a.Hq, i = x / a.Hq % a.n, b = x / a.Hq / a.n % a.B, layer = x / a.Hq / a.n / a.B;
  if (threadIdx.x == 0 && i == 0 && j == 0 && len_bad(a, lens, b)) flag(a, KVQ_ERR_RANGE);
  const int lim = len_of(a, lens, b) - a.n + 1 + i;
  SimpleAttend<T, BITS, D> s;
  s.begin(q + (size_t)x * D);
  for (int pg = 0; (pg << a.page_log2) < lim; ++pg)
    s.page(a, a.layer0 + layer, b, j / a.g, pg, min(a.page, lim - (pg << a.page_log2)));
  s.end(out + (size_t)x * D);
}

template <typename T, int BITS>
cudaError_t go(const Args& a, const void* q, const int32_t* lens, void* out, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.n_layers * a.B * a.n * a.Hq);
  const T* qt = static_cast<const T*>(q);
  T* ot = static_cast<T*>(out);
  if (a.d == 64) decode_kernel<T, BITS, 64><<<grid, kSimpleThreads, 0, s>>>(a, qt, lens, ot);
  else if (a.d == 128) decode_kernel<T, BITS, 128><<<grid, kSimpleThreads, 0, s>>>(a, qt, lens, ot);
  else decode_kernel<T, BITS, 256><<<grid, kSimpleThreads, 0, s>>>(a, qt, lens, ot);
  return cudaGetLastError();
}

}  // namespace

size_t decode_workspace_bytes(const Args&) { return 16; }

cudaError_t launch_decode(const Args& a, int dtype, const void* q, const int32_t* lens, void* out, void*, cudaStream_t s) {
  if (dtype == LOWRAM_F32) return a.bits == 4 ? go<float, 4>(a, q, lens, out, s) : go<float, 8>(a, q, lens, out, s);
  return a.bits == 4 ? go<__nv_bfloat16, 4>(a, q, lens, out, s) : go<__nv_bfloat16, 8>(a, q, lens, out, s);
}

}  // namespace kvq
}  // namespace lowram
