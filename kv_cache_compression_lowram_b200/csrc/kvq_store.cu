// Quantised KV cache: writing rows (quantise) and reading them back (dequantise).
//
// Both are one pass over the caller's rows, bound by HBM: per K or V row of d channels,
// d * sizeof(dt) bytes on one side and d * bits / 8 + d / 16 on the other.  A CTA takes the
// part of one page that a call touches, for one (layer, sequence, KV head): the page's codes
// and scales are one contiguous block each, the caller's rows are d-long pieces that
// neighbouring CTAs (the next head) continue.  Half of its warps take K, half V; a lane
// holds 8 channels (16 bytes of bf16), so 8 lanes hold a group and its minimum and maximum
// are three shuffles.
#include "kvq.cuh"

namespace lowram {
namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;   // rows in flight per lane
constexpr unsigned kAll = 0xffffffffu;

// fp32 value of a small non-negative integer sits in the low mantissa bits of x + kMagic.
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
constexpr uint32_t kMagicBits = 0x4B400000u;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight consecutive channels as they lie in the caller's row.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p) { w = __ldcs(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, const float (&x)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    __stcs(static_cast<uint4*>(p), *reinterpret_cast<uint4*>(h));
  }
};
template <> struct Raw8<float> {
  float4 w0, w1;
  __device__ __forceinline__ void load(const void* p) {
    w0 = __ldcs(static_cast<const float4*>(p));
    w1 = __ldcs(static_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { w0 = w1 = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = w0.x; x[1] = w0.y; x[2] = w0.z; x[3] = w0.w;
    x[4] = w1.x; x[5] = w1.y; x[6] = w1.z; x[7] = w1.w;
  }
  static __device__ __forceinline__ void store(void* p, const float (&x)[8]) {
    __stcs(static_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(static_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
};

// The codes of 8 channels: one word (4 bits) or two (8 bits).
template <int BITS> struct Cell {
  uint32_t w[BITS / 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BITS == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x;
      w[1] = t.y;
    }
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ uint32_t code(int i) const {
    if constexpr (BITS == 4) return (w[0] >> (4 * i)) & 15u;
    else return (w[i / 4] >> (8 * (i % 4))) & 255u;
  }
};

// lo + s n: s n has at most 11 + 8 significant bits, so this is one rounding to fp32.
template <int BITS>
__device__ __forceinline__ void dequant(const Cell<BITS>& c, __half2 meta, float (&x)[8]) {
  const float s = __low2float(meta), lo = __high2float(meta);
#pragma unroll
  for (int i = 0; i < 8; ++i)   // the integer to fp32 by way of its place in 2^23's mantissa
    x[i] = fmaf(s, __uint_as_float(0x4B000000u | c.code(i)) - 8388608.0f, lo);
}

// Codes and (s, lo) of the group that this lane's 8 neighbours share.
template <typename T, int BITS>
__device__ __forceinline__ void quantise(const float (&x)[8], Cell<BITS>& c, __half2& meta) {
  constexpr float kQ = (float)((1 << BITS) - 1);
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = min_nan(mn, x[i]);
    mx = max_nan(mx, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    mn = min_nan(mn, __shfl_xor_sync(kAll, mn, o));
    mx = max_nan(mx, __shfl_xor_sync(kAll, mx, o));
  }
  // bf16 values differ exactly in fp32 unless one is below 2^-16 of the other
  float sf;
  if constexpr (sizeof(T) == 2) sf = __fdiv_rn(mx - mn, kQ);
  else sf = (float)(((double)mx - (double)mn) / (double)kQ);
  meta = __halves2half2(__float2half_rn(sf), __float2half_rn(mn));
  const float s = __low2float(meta), lo = __high2float(meta);
  const bool usable = s > 0.f && s < INFINITY && fabsf(lo) < INFINITY;
  const float inv = usable ? __frcp_rn(s) : 0.f, off = usable ? -lo * inv : 0.f;
  // Fast codes: f = x inv + off = (x - lo) / s up to (2 kQ + |off|) 2^-24 (inv, off and the
  // sum are each off by 2^-24 relative), rounded by adding kMagic.  A value nearer than twice
  // that to a half step, and a group whose rounded lo or s lets codes leave [0, 2^b - 1], take
  // the exact path below.
  const float tie = 0.5f - (2.f * kQ + fabsf(off)) * 1.1920929e-7f;
  float near = 0.f;
  uint32_t bits[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = fmaf(x[i], inv, off), r = f + kMagic;
    bits[i] = __float_as_uint(r);
    near = fmaxf(near, fabsf(f - (r - kMagic)));
  }
  const bool inside = fmaf(mn, inv, off) > -0.49f && fmaf(mx, inv, off) < kQ + 0.49f;
  if (usable && !(inside && near < tie)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double f = rint(((double)x[i] - (double)lo) / (double)s);
      f = f < 0.0 ? 0.0 : (f > (double)kQ ? (double)kQ : f);
      bits[i] = kMagicBits + (uint32_t)(int)f;
    }
  }
  // sum of code_i << (BITS * i), the magic bits taken off once (arithmetic modulo 2^32)
#pragma unroll
  for (int j = 0; j < BITS / 4; ++j) {
    constexpr int kPer = 32 / BITS;
    uint32_t w = 0, m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      w += bits[j * kPer + i] << (BITS * i);
      m += kMagicBits << (BITS * i);
    }
    c.w[j] = usable ? w - m : 0u;
  }
}

// What a CTA works on: slots [s0, s1) of one page.
struct Piece {
  int layer, b, h, page, s0, s1, tok0;   // token of slot t: tok0 + t
};
__device__ __forceinline__ bool piece_of(const Args& a, const int32_t* pos, const int32_t* count, int pieces, Piece* p) {
  unsigned x = blockIdx.x;
  p->h = x % a.Hkv;
  x /= a.Hkv;
  const int j = x % pieces;
  x /= pieces;
  p->b = x % a.B;
  p->layer = x / a.B;
  const long long p0 = __ldg(pos + p->b);
  int n = a.n;
  bool bad = false;
  if (count) {
    const int c = __ldg(count + p->b);
    bad = c < 0 || c > a.n;
    n = c < 0 ? 0 : min(c, a.n);
  }
  const long long cap = (long long)a.max_pages << a.page_log2;
  bad |= n > 0 && (p0 < 0 || p0 + n > cap);
  if (bad && threadIdx.x == 0 && j == 0) flag(a, KVQ_ERR_RANGE);
  const long long pg = (p0 >> a.page_log2) + j, base = pg * a.page;
  const long long t0 = p0 > base ? p0 : base, t1 = p0 + n < base + a.page ? p0 + n : base + a.page;
  if (t0 >= t1) return false;
  p->page = pg >= 0 && pg < a.max_pages ? (int)pg : -1;
  p->s0 = (int)(t0 - base);
  p->s1 = (int)(t1 - base);
  p->tok0 = (int)(base - p0);
  return true;
}

template <typename T, int BITS, int D>
__global__ void __launch_bounds__(kThreads) write_kernel(Args a, Rows k, Rows v, const int32_t* __restrict__ pos,
                                                         const int32_t* __restrict__ count, int pieces) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = 2 * RPW, G = D / kGroup, ROW = D * BITS / 8;
  __shared__ float sums[STEP][D];
  Piece p;
  if (!piece_of(a, pos, count, pieces, &p)) return;
  const int pid = p.page < 0 ? -1 : page_of(a, p.b, p.page);
  if (pid < 0) {
    if (p.page >= 0 && threadIdx.x == 0) flag(a, KVQ_ERR_PAGE);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_v = warp >= 2;
  const int rsub = (warp & 1) * RPW + lane / LPR, c8 = lane % LPR, grp = c8 / 8, cell = (c8 % 8) * G + grp;
  const Rows& src = is_v ? v : k;
  const char* in = static_cast<const char*>(src.p) +
                   sizeof(T) * (p.layer * src.layer + p.b * src.seq + p.h * src.head + c8 * 8);
  const size_t row0 = row0_of(a, a.layer0 + p.layer, pid, p.h);
  uint8_t* code = (is_v ? a.v_code : a.k_code) + row0 * ROW + cell * BITS;
  __half2* scale = (is_v ? a.v_scale : a.k_scale) + row0 * G + grp;
  const bool mean = p.s1 == a.page && a.k_mean != nullptr;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  // Rows of slot t belong to the lanes with rsub = t mod STEP, so a page's mean is summed in
  // one order however its tokens arrived.
  if (mean && !is_v)
    for (int t = rsub; t < p.s0; t += STEP) {
      Cell<BITS> c;
      float x[8];
      c.load(code + (size_t)t * ROW);
      dequant<BITS>(c, scale[(size_t)t * G], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += x[i];
    }
  for (int base = p.s0 & ~(STEP - 1); base < p.s1; base += STEP * kUnroll) {
    Raw8<T> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = base + u * STEP + rsub;
      if (t >= p.s0 && t < p.s1) raw[u].load(in + sizeof(T) * ((int64_t)(p.tok0 + t) * src.tok));
      else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = base + u * STEP + rsub;
      if (base + u * STEP >= p.s1) break;
      float x[8];
      Cell<BITS> c;
      __half2 meta;
      raw[u].get(x);
      quantise<T, BITS>(x, c, meta);
      if (t < p.s0 || t >= p.s1) continue;
      c.store(code + (size_t)t * ROW);
      if ((c8 & 7) == 0) scale[(size_t)t * G] = meta;
      if (mean && !is_v) {
        dequant<BITS>(c, meta, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += x[i];
      }
    }
  }
  if (!mean) return;   // the same for the whole CTA
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[rsub][c8 * 8 + i] = acc[i];
  }
  __syncthreads();
  __nv_bfloat16* out = a.k_mean + (row0 >> a.page_log2) * D;
  const float inv = 1.f / (float)a.page;   // a power of two
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < STEP; ++r) s += sums[r][c];
    out[c] = __float2bfloat16_rn(s * inv);
  }
}

template <typename T, int BITS, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Args a, Rows k, Rows v, const int32_t* __restrict__ pos,
                                                        const int32_t* __restrict__ count, int pieces) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = 2 * RPW, G = D / kGroup, ROW = D * BITS / 8;
  Piece p;
  if (!piece_of(a, pos, count, pieces, &p)) return;
  const int pid = p.page < 0 ? -1 : page_of(a, p.b, p.page);
  if (pid < 0 && p.page >= 0 && threadIdx.x == 0) flag(a, KVQ_ERR_PAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_v = warp >= 2;
  const int rsub = (warp & 1) * RPW + lane / LPR, c8 = lane % LPR, grp = c8 / 8, cell = (c8 % 8) * G + grp;
  const Rows& dst = is_v ? v : k;
  char* out = static_cast<char*>(dst.p) + sizeof(T) * (p.layer * dst.layer + p.b * dst.seq + p.h * dst.head + c8 * 8);
  const size_t row0 = pid < 0 ? 0 : row0_of(a, a.layer0 + p.layer, pid, p.h);
  const uint8_t* code = (is_v ? a.v_code : a.k_code) + row0 * ROW + cell * BITS;
  const __half2* scale = (is_v ? a.v_scale : a.k_scale) + row0 * G + grp;
  for (int base = p.s0; base < p.s1; base += STEP * kUnroll) {
    Cell<BITS> c[kUnroll];
    __half2 meta[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = base + u * STEP + rsub;
      meta[u] = __half2half2(__ushort_as_half(0));
      if (t < p.s1 && pid >= 0) {
        c[u].load(code + (size_t)t * ROW);
        meta[u] = scale[(size_t)t * G];
      } else {
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) c[u].w[i] = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = base + u * STEP + rsub;
      if (t >= p.s1) break;
      float x[8];
      dequant<BITS>(c[u], meta[u], x);
      Raw8<T>::store(out + sizeof(T) * ((int64_t)(p.tok0 + t) * dst.tok), x);
    }
  }
}

template <bool WRITE, typename T, int BITS>
cudaError_t go(const Args& a, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count, cudaStream_t s) {
  const int pieces = ((a.n - 1) >> a.page_log2) + 2;   // a run of n tokens touches at most this many pages
  const unsigned grid = (unsigned)((long long)pieces * a.n_layers * a.B * a.Hkv);
#define LOWRAM_KVQ_GO(D)                                                              \
  if constexpr (WRITE) write_kernel<T, BITS, D><<<grid, kThreads, 0, s>>>(a, k, v, pos, count, pieces); \
  else read_kernel<T, BITS, D><<<grid, kThreads, 0, s>>>(a, k, v, pos, count, pieces)
  switch (a.d) {
    case 64: LOWRAM_KVQ_GO(64); break;
    case 128: LOWRAM_KVQ_GO(128); break;
    default: LOWRAM_KVQ_GO(256); break;
  }
#undef LOWRAM_KVQ_GO
  return cudaGetLastError();
}

template <bool WRITE>
cudaError_t launch(const Args& a, int dtype, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count, cudaStream_t s) {
  if (dtype == LOWRAM_F32)
    return a.bits == 4 ? go<WRITE, float, 4>(a, k, v, pos, count, s) : go<WRITE, float, 8>(a, k, v, pos, count, s);
  return a.bits == 4 ? go<WRITE, __nv_bfloat16, 4>(a, k, v, pos, count, s)
                     : go<WRITE, __nv_bfloat16, 8>(a, k, v, pos, count, s);
}

}  // namespace

cudaError_t launch_write(const Args& a, int dtype, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count,
                         cudaStream_t s) {
  return launch<true>(a, dtype, k, v, pos, count, s);
}
cudaError_t launch_read(const Args& a, int dtype, const Rows& k, const Rows& v, const int32_t* pos, const int32_t* count,
                        cudaStream_t s) {
  return launch<false>(a, dtype, k, v, pos, count, s);
}

}  // namespace kvq
}  // namespace lowram
