// Quantised KV cache: geometry and launchers (kvq.cu checks arguments, kvq_store.cu writes and
// reads rows, kvq_decode.cu and kvq_sparse.cu attend).
#pragma once

#include "lowram_internal.cuh"

namespace lowram {
namespace kvq {

constexpr int kGroup = 64;           // channels of a quantisation group
constexpr int kMaxQ = 16;            // query tokens of a call
constexpr int kMaxPagesSeq = 16384;  // pages of a sequence
constexpr int kMaxTopK = 512;

enum : uint32_t { KVQ_ERR_PAGE = 1u << 0, KVQ_ERR_RANGE = 1u << 1 };

struct Args {
  int B, Hkv, Hq, g, page_log2, page, n_pages, max_pages, bits, d;
  int layer0, n_layers, n;   // n: new tokens, tokens to read, or query tokens
  uint8_t* k_code;
  uint8_t* v_code;
  __half2* k_scale;          // (s, lo)
  __half2* v_scale;
  __nv_bfloat16* k_mean;
  const int32_t* table;
  uint32_t* err;
};

__device__ __forceinline__ void flag(const Args& a, uint32_t bit) {
  if (a.err) atomicOr(a.err, bit);
}
// The pool page of sequence b's page i (0 <= i < max_pages), or -1 if the table is wrong.
__device__ __forceinline__ int page_of(const Args& a, int b, int i) {
  if (!a.table) return b * a.max_pages + i;
  const int p = __ldg(a.table + (size_t)b * a.max_pages + i);
  return p >= 0 && p < a.n_pages ? p : -1;
}
// Row index (token rows) of slot 0 of (layer, pool page, head).
__device__ __forceinline__ size_t row0_of(const Args& a, int layer, int pid, int h) {
  return (((size_t)layer * a.n_pages + pid) * a.Hkv + h) << a.page_log2;
}
// A sequence's length, clamped to what its table row can hold.
__device__ __forceinline__ int len_of(const Args& a, const int32_t* lens, int b) {
  const int len = __ldg(lens + b), cap = a.max_pages << a.page_log2;
  return len < 0 ? 0 : (len > cap ? cap : len);
}
__device__ __forceinline__ bool len_bad(const Args& a, const int32_t* lens, int b) {
  const int len = __ldg(lens + b);
  return len < 0 || len > (a.max_pages << a.page_log2);
}

// Two fp32 numbers in one 64-bit register, and Blackwell's operations on both at once.
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
  __device__ __forceinline__ float2 get() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

struct Rows {   // strided rows of a caller's tensor, strides in elements
  void* p;
  int64_t layer, seq, tok, head;
};

cudaError_t launch_write(const Args& a, int dtype, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count,
                         cudaStream_t s);
cudaError_t launch_read(const Args& a, int dtype, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count,
                        cudaStream_t s);
size_t decode_workspace_bytes(const Args& a);
bool decode_line_fits(const Args& a);
cudaError_t launch_decode(const Args& a, int dtype, const void* q, const int32_t* lens, void* out, void* ws, cudaStream_t s);
cudaError_t launch_sparse(const Args& a, int dtype, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel,
                          cudaStream_t s);

}  // namespace kvq
}  // namespace lowram
