// Quantised KV cache: attention over the pages that their mean keys select for each query.
//
// Simple form: one CTA per (layer, sequence, query token, KV head) scores the pages in 64
// bits, takes the best one top_k - 1 times, and attends head by head.
#include "kvq.cuh"
#include "kvq_simple.cuh"

namespace lowram {
namespace kvq {
namespace {

template <typename T, int BITS, int D>
__global__ void __launch_bounds__(kSimpleThreads) sparse_kernel(Args a, int top_k, const T* __restrict__ q,
                                                                const int32_t* __restrict__ lens, T* __restrict__ out,
                                                                int32_t* __restrict__ sel) {
  extern __shared__ double score[];   // [max_pages], then the selected pages' marks
  uint8_t* mark = reinterpret_cast<uint8_t*>(score + a.max_pages);
  __shared__ double qs[D], best_s[kSimpleThreads];
  __shared__ int best_c[kSimpleThreads];
  const unsigned x = blockIdx.x;   // ((layer * B + b) * n + i) * Hkv + h
  const int h = x % a.Hkv, i = x / a.Hkv % a.n, b = x / a.Hkv / a.n % a.B, layer = x / a.Hkv / a.n / a.B, tid = threadIdx.x;
  if (tid == 0 && i == 0 && h == 0 && len_bad(a, lens, b)) flag(a, KVQ_ERR_RANGE);
  const int lim = len_of(a, lens, b) - a.n + 1 + i, last = lim > 0 ? (lim - 1) >> a.page_log2 : -1;
  const T* qu = q + (size_t)x * a.g * D;
  for (int c = tid; c < D; c += kSimpleThreads) {
    double s = 0.0;
    for (int j = 0; j < a.g; ++j) s += (double)to_f<T>(qu[(size_t)j * D + c]);
    qs[c] = s;
  }
  __syncthreads();
  for (int c = tid; c < last; c += kSimpleThreads) {
    const int pid = page_of(a, b, c);
    double s = -INFINITY;
    if (pid < 0) {
      flag(a, KVQ_ERR_PAGE);
    } else {
      const __nv_bfloat16* mean = a.k_mean + (row0_of(a, a.layer0 + layer, pid, h) >> a.page_log2) * D;
      s = 0.0;
      for (int k = 0; k < D; ++k) s = fma(qs[k], (double)__bfloat162float(mean[k]), s);
      if (s != s) s = -INFINITY;
    }
    score[c] = s;
    mark[c] = 0;
  }
  if (tid == 0 && last >= 0) mark[last] = 1;
  __syncthreads();
  for (int r = 0; r < top_k - 1 && r < last; ++r) {
    double s = -INFINITY;
    int w = 0x7fffffff;
    for (int c = tid; c < last; c += kSimpleThreads)
      if (!mark[c] && (score[c] > s || w == 0x7fffffff)) {
        s = score[c];
        w = c;
      }
    best_s[tid] = s;
    best_c[tid] = w;
    __syncthreads();
    if (tid == 0) {
      for (int t = 1; t < kSimpleThreads; ++t)
        if (best_c[t] != 0x7fffffff && (w == 0x7fffffff || best_s[t] > s || (best_s[t] == s && best_c[t] < w))) {
          s = best_s[t];
          w = best_c[t];
        }
      mark[w] = 1;
    }
    __syncthreads();
  }
  if (sel && tid == 0) {
    int k = 0;
    for (int c = 0; c <= last; ++c)
      if (mark[c]) sel[(size_t)x * top_k + k++] = c;
    for (; k < top_k; ++k) sel[(size_t)x * top_k + k] = -1;
  }
  for (int j = 0; j < a.g; ++j) {
    SimpleAttend<T, BITS, D> s;
    s.begin(qu + (size_t)j * D);
    for (int pg = 0; pg <= last; ++pg)
      if (mark[pg]) s.page(a, a.layer0 + layer, b, h, pg, min(a.page, lim - (pg << a.page_log2)));
    s.end(out + ((size_t)x * a.g + j) * D);
    __syncthreads();
  }
}

template <typename T, int BITS, int D>
cudaError_t go(const Args& a, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.n_layers * a.B * a.n * a.Hkv);
  const size_t smem = (size_t)a.max_pages * 9;
  cudaError_t e = cudaFuncSetAttribute(sparse_kernel<T, BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  sparse_kernel<T, BITS, D><<<grid, kSimpleThreads, smem, s>>>(a, top_k, static_cast<const T*>(q), lens, static_cast<T*>(out), sel);
  return cudaGetLastError();
}
template <typename T, int BITS>
cudaError_t by_d(const Args& a, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel, cudaStream_t s) {
  if (a.d == 64) return go<T, BITS, 64>(a, top_k, q, lens, out, sel, s);
  if (a.d == 128) return go<T, BITS, 128>(a, top_k, q, lens, out, sel, s);
  return go<T, BITS, 256>(a, top_k, q, lens, out, sel, s);
}

}  // namespace

cudaError_t launch_sparse(const Args& a, int dtype, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel,
                          cudaStream_t s) {
  if (dtype == LOWRAM_F32)
    return a.bits == 4 ? by_d<float, 4>(a, top_k, q, lens, out, sel, s) : by_d<float, 8>(a, top_k, q, lens, out, sel, s);
  return a.bits == 4 ? by_d<__nv_bfloat16, 4>(a, top_k, q, lens, out, sel, s)
                     : by_d<__nv_bfloat16, 8>(a, top_k, q, lens, out, sel, s);
}

}  // namespace kvq
}  // namespace lowram
