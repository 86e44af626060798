// One query over pages of the quantised cache, a page at a time: thread t scores tokens t,
// t + 128, ...; thread c then sums channels c, c + 128, ... of the values.
#pragma once

#include "kvq.cuh"

namespace lowram {
namespace kvq {

constexpr int kSimpleThreads = 128;

template <int BITS, int D>
__device__ __forceinline__ float simple_value(const uint8_t* code, const __half2* scale, int c) {
  const int cell = (c % 64) / 8 * (D / 64) + c / 64, i = c % 8;
  const uint8_t byte = code[cell * BITS + i * BITS / 8];
  const int n = BITS == 8 ? byte : (i & 1 ? byte >> 4 : byte & 15);
  const float2 m = __half22float2(scale[c / 64]);
  return fmaf(m.x, (float)n, m.y);
}

template <typename T, int BITS, int D> struct SimpleAttend {
  float m, l, acc[(D + kSimpleThreads - 1) / kSimpleThreads];
  static __device__ __forceinline__ float* smem() {
    __shared__ float sm[D + 256 + 8];
    return sm;
  }
  __device__ void begin(const T* q) {
    float* qs = smem();
    for (int c = threadIdx.x; c < D; c += kSimpleThreads) qs[c] = to_f<T>(q[c]) * (1.4426950408889634f / sqrtf((float)D));
    m = -INFINITY;
    l = 0.f;
    for (float& x : acc) x = 0.f;
    __syncthreads();
  }
  __device__ void page(const Args& a, int layer, int b, int h, int pg, int cnt) {
    float *qs = smem(), *p = qs + D, *red = p + 256;
    const int pid = page_of(a, b, pg);
    if (pid < 0) {
      if (threadIdx.x == 0) flag(a, KVQ_ERR_PAGE);
      return;
    }
    const size_t row = row0_of(a, layer, pid, h);
    float mx = -INFINITY;
    for (int t = threadIdx.x; t < cnt; t += kSimpleThreads) {
      float x = 0.f;
      for (int c = 0; c < D; ++c)
        x = fmaf(qs[c], simple_value<BITS, D>(a.k_code + (row + t) * (D * BITS / 8), a.k_scale + (row + t) * (D / 64), c), x);
      p[t] = x;
      mx = fmaxf(mx, x);
    }
    mx = warp_max(mx);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = exp2f(m - mn);
    m = mn;
    for (int t = threadIdx.x; t < cnt; t += kSimpleThreads) p[t] = exp2f(p[t] - mn);
    __syncthreads();
    l *= alpha;
    for (int t = 0; t < cnt; ++t) l += p[t];
    for (int k = 0, c = threadIdx.x; c < D; c += kSimpleThreads, ++k) {
      float x = acc[k] * alpha;
      for (int t = 0; t < cnt; ++t)
        x = fmaf(p[t], simple_value<BITS, D>(a.v_code + (row + t) * (D * BITS / 8), a.v_scale + (row + t) * (D / 64), c), x);
      acc[k] = x;
    }
    __syncthreads();
  }
  __device__ void end(T* out) {
    for (int k = 0, c = threadIdx.x; c < D; c += kSimpleThreads, ++k) out[c] = from_f<T>(l > 0.f ? acc[k] / l : 0.f);
  }
};

}  // namespace kvq
}  // namespace lowram
