// Quantised KV cache: writing rows (quantise) and reading them back (dequantise).
//
// Both are one pass over the caller's rows, bound by HBM: per K or V row of d channels,
// d * sizeof(dt) bytes on one side and d * bits / 8 + d / 16 on the other (8 x 8192 tokens, 8 heads of 128,
// bf16 and 4 bits, 344 MB: written in 91 us, 3.8 TB/s, read back in 65 us, 5.3 TB/s).  A CTA takes the
// part of one page that a call touches, for one (layer, sequence, KV head): the page's codes
// and scales are one contiguous block each, the caller's rows are d-long pieces that
// neighbouring CTAs (the next head) continue.  Half of its warps take K, half V (writing has one
// each: with two each, what a warp does once was a third of its instructions).
//
// Writing is limited by instructions as much as by memory, so numbers go two to a register (channels
// k and k + 4 of a cell) through the packed fp32 operations, a lane holds 16 channels (4 lanes a
// group: the minimum and maximum are two shuffles, of a packed pair for bf16, and what a group
// costs once is spread over 16 values: 266 instructions of a warp per 512 values, in 70 % of the issue
// slots), and a code is one FFMA and one rounding add, with the
// distance to the next half step watched beside it: only where a value is too near to one is the
// remainder computed exactly.
#include "kvq.cuh"

namespace lowram {
namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kWriteThreads = 64;   // a warp for K and one for V
constexpr int kUnroll = 4;   // rows that a lane of the reading kernel has in flight
constexpr unsigned kAll = 0xffffffffu;

// x + kMagic - kMagic is x rounded to an integer (half to even; |x| < 2^22), whose parity is the last
// bit of x + kMagic.
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// max(|a|, |b|, |c|), not NaN unless all are
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// min(|a|, |b|, |c|)
__device__ __forceinline__ float min_abs(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
  // channels k and k + 4
  __device__ __forceinline__ F2 pair(int k) const {
    const uint32_t a = k < 2 ? w.x : w.y, b = k < 2 ? w.z : w.w;
    return k & 1 ? F2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)) : F2(__uint_as_float(a << 16), __uint_as_float(b << 16));
  }
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
  __device__ __forceinline__ F2 pair(int k) const {
    return k == 0 ? F2(w0.x, w1.x) : (k == 1 ? F2(w0.y, w1.y) : (k == 2 ? F2(w0.z, w1.z) : F2(w0.w, w1.w)));
  }
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

// Smallest and largest of the group's 64 values, 16 of which this lane holds; NaN if any is.
__device__ __forceinline__ float2 group_range(const Raw8<float> (&raw)[2]) {
  float x[16];
  raw[0].get(*reinterpret_cast<float(*)[8]>(x));
  raw[1].get(*reinterpret_cast<float(*)[8]>(x + 8));
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    mn = min_nan(mn, x[i]);
    mx = max_nan(mx, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = min_nan(mn, __shfl_xor_sync(kAll, mn, o));
    mx = max_nan(mx, __shfl_xor_sync(kAll, mx, o));
  }
  return make_float2(mn, mx);
}
__device__ __forceinline__ float2 group_range(const Raw8<__nv_bfloat16> (&raw)[2]) {
  const uint32_t w[8] = {raw[0].w.x, raw[0].w.y, raw[0].w.z, raw[0].w.w, raw[1].w.x, raw[1].w.y, raw[1].w.z, raw[1].w.w};
  auto h2 = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
  __nv_bfloat162 mn = h2(w[0]), mx = mn;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = __hmin2_nan(mn, h2(w[i]));
    mx = __hmax2_nan(mx, h2(w[i]));
  }
  // one pair (min, -max), so that each further step is one minimum
  const __nv_bfloat162 ng = __hneg2(mx);
  __nv_bfloat162 m = __hmin2_nan(__lows2bfloat162(mn, ng), __highs2bfloat162(mn, ng));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t y = __shfl_xor_sync(kAll, *reinterpret_cast<uint32_t*>(&m), o);
    m = __hmin2_nan(m, h2(y));
  }
  return make_float2(__low2float(m), -__high2float(m));
}

// What t = x - y, rounded to fp32, has lost: x - y = t + lost(x, y, t) exactly (two-sum).
__device__ __forceinline__ float lost(float x, float y, float t) {
  const float z = t - x;
  return (x - (t - z)) + (-y - z);
}

// What the codes of a group are made with.
struct Scale {
  float s, lo, inv, off;
  bool usable, inside;   // not a constant group or one with non-finite values; codes cannot leave [0, 2^b - 1]
};
template <typename T, int BITS>
__device__ __forceinline__ Scale scale_of(float2 range, __half2& meta) {
  constexpr float kQ = (float)((1 << BITS) - 1), kInvQ = 1.f / kQ;
  const float mn = range.x, mx = range.y;
  float sf;
  if constexpr (sizeof(T) == 2) {
    // The range (exact in fp32 unless one end is below 2^-16 of the other; what is lost joins the
    // remainder) over the constant, correctly rounded: Markstein's correction of a quotient by its
    // remainder ("IA-64 and Elementary Functions", 2000), with the constant's rounded reciprocal.
    const float span = mx - mn, q = span * kInvQ;
    sf = fmaf(fmaf(-q, kQ, span) + lost(mx, mn, span), kInvQ, q);
  } else {
    sf = (float)(((double)mx - (double)mn) / (double)kQ);
  }
  meta = __floats2half2_rn(sf, mn);
  Scale g;
  g.s = __low2float(meta);
  g.lo = __high2float(meta);
  g.usable = g.s > 0.f && g.s < INFINITY && fabsf(g.lo) < INFINITY;
  const float inv = __fdividef(1.f, g.s);
  g.inv = g.usable ? fmaf(inv, fmaf(-g.s, inv, 1.f), inv) : 0.f;
  g.off = g.usable ? -g.lo * g.inv : 0.f;
  g.inside = fmaf(mn, g.inv, g.off) > -0.49f && fmaf(mx, g.inv, g.off) < kQ + 0.49f;
  return g;
}

// The codes of 8 channels, as a cell and as numbers (nf[k]: channels k and k + 4).
template <typename T, int BITS>
__device__ __forceinline__ void codes_of(const Raw8<T>& raw, const Scale& g, Cell<BITS>& c, F2 (&nf)[4]) {
  constexpr float kQ = (float)((1 << BITS) - 1);
  const F2 magic(kMagic), unmagic(-kMagic), inv(g.inv);
  float near = 0.f;
  bool exact = !g.inside;
  auto exactly = [&]() {   // all codes anew
    auto code = [&](float x) {
      // t + te = x - lo exactly; n the nearest code up to one; m = t - n s exactly (n s has 19 bits and
      // is within s of t); so the sign of 2 (m + te) -+ s is known
      const float t = x - g.lo, te = lost(x, g.lo, t);
      float n = fminf(fmaxf(t * g.inv, -1.f), kQ + 1.f);
      n = (n + kMagic) - kMagic;
      const float m = fmaf(-n, g.s, t), above = (2.f * m - g.s) + 2.f * te, below = (2.f * m + g.s) + 2.f * te;
      const bool odd = __float_as_uint(n + kMagic) & 1u;
      if (above > 0.f || (above == 0.f && odd)) n += 1.f;
      else if (below < 0.f || (below == 0.f && odd)) n -= 1.f;
      return fminf(fmaxf(n, 0.f), kQ);
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = raw.pair(k).get();
      nf[k] = F2(code(x.x), code(x.y));
    }
  };
  if constexpr (sizeof(T) == 2) {
    // t = x - lo is exact but for x below 2^-16 of lo, and so is the remainder e = t - n s: a code is
    // right where |e| < s / 2.  (Half steps are fp32 numbers, so a t that was rounded lies on the same
    // side of them as x - lo, or meets one: then the codes are made exactly.)  Values of 8 bits do meet
    // half steps: every 28th group of 64 normal values has one in 4 bits.
    const float hs = 0.5f * g.s;
    const F2 minus_lo(-g.lo), minus_s(-g.s);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const F2 t = add2(raw.pair(k), minus_lo);
      nf[k] = add2(fma2(t, inv, magic), unmagic);
      const float2 e = fma2(nf[k], minus_s, t).get();
      near = max_abs(near, e.x, e.y);
    }
    if (near >= hs && g.usable) {   // (a group without a scale has codes of 0)
      float least = INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = raw.pair(k).get(), e = fma2(nf[k], minus_s, add2(raw.pair(k), minus_lo)).get();
        least = min_abs(least, x.x, x.y);
        float2 n = nf[k].get();
        auto odd = [](float x) { return __float_as_uint(x + kMagic) & 1u; };
        if (fabsf(e.x) > hs || (fabsf(e.x) == hs && odd(n.x))) n.x += copysignf(1.f, e.x);
        if (fabsf(e.y) > hs || (fabsf(e.y) == hs && odd(n.y))) n.y += copysignf(1.f, e.y);
        nf[k] = F2(n.x, n.y);
      }
      if (least < 3.0517578e-5f * fabsf(g.lo)) exactly();   // 2^-15
    }
  } else {
    // f = x inv + off = (x - lo) / s up to (2 kQ + |off|) 2^-24 (inv, off and the sum are each off by
    // 2^-24 relative), rounded by adding kMagic.  A value nearer than twice that to a half step takes
    // the exact path below.
    const float tie = 0.5f - (2.f * kQ + fabsf(g.off)) * 1.1920929e-7f;
    const F2 off(g.off), minus(-1.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const F2 f = fma2(raw.pair(k), inv, off);
      nf[k] = add2(add2(f, magic), unmagic);
      const float2 e = fma2(nf[k], minus, f).get();
      near = max_abs(near, e.x, e.y);
    }
    exact |= !(near < tie);
  }
  if (exact && g.usable) exactly();
  // four codes (two of 8 bits) in one fp32 number, whose integer then lies in its low mantissa bits
  const F2 bias(8388608.f);
  auto words = [&](F2 x) { const float2 y = add2(x, bias).get(); return make_uint2(__float_as_uint(y.x), __float_as_uint(y.y)); };
  if constexpr (BITS == 4) {
    const uint2 y = words(fma2(nf[3], F2(4096.f), fma2(nf[2], F2(256.f), fma2(nf[1], F2(16.f), nf[0]))));
    c.w[0] = __byte_perm(y.x, y.y, 0x5410);
  } else {
    const uint2 a = words(fma2(nf[1], F2(256.f), nf[0])), b = words(fma2(nf[3], F2(256.f), nf[2]));
    c.w[0] = __byte_perm(a.x, b.x, 0x5410);
    c.w[1] = __byte_perm(a.y, b.y, 0x5410);
  }
}

// What a CTA works on: slots [s0, s1) of one page.
struct Piece {
  int layer, b, h, page, s0, s1, tok0;   // token of slot t: tok0 + t
};
__device__ __forceinline__ bool piece_of(const Args& a, const int32_t* pos, const int32_t* count, Piece* p) {
  const int j = blockIdx.x / a.Hkv;        // grid: (piece, head), sequence, layer
  p->h = blockIdx.x - j * a.Hkv;
  p->b = blockIdx.y;
  p->layer = blockIdx.z;
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
__global__ void __launch_bounds__(kWriteThreads, sizeof(T) == 2 ? 14 : 12) write_kernel(Args a, Rows k, Rows v, const int32_t* __restrict__ pos,
                                                         const int32_t* __restrict__ count) {
  constexpr int LPR = D / 16, STEP = 32 / LPR, G = D / kGroup, ROW = D * BITS / 8, FLY = 2;
  __shared__ float sums[STEP][D];
  Piece p;
  if (!piece_of(a, pos, count, &p)) return;
  const int pid = p.page < 0 ? -1 : page_of(a, p.b, p.page);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_v = warp == 1;
  const int rsub = lane / LPR, l16 = lane % LPR, grp = l16 / 4, cell = l16 % 4 * G + grp;
  const int ch = grp * 64 + l16 % 4 * 8;   // the lane's channels: 8 from here on, and 8 that lie 32 further (every access whole sectors)
  const Rows& src = is_v ? v : k;
  const char* in = static_cast<const char*>(src.p) +
                   sizeof(T) * (p.layer * src.layer + p.b * src.seq + p.h * src.head + ch);
  // FLY rows of a lane are on their way from here on (the table's answer is not needed for them)
  int ahead = (p.s0 & ~(STEP - 1)) + rsub;
  in += sizeof(T) * ((int64_t)(p.tok0 + ahead) * src.tok);
  const int64_t in_step = (int64_t)sizeof(T) * STEP * src.tok;
  Raw8<T> raw[FLY][2];
  auto fetch = [&](Raw8<T> (&r)[2]) {
    if (ahead >= p.s0 && ahead < p.s1) {
      r[0].load(in);
      r[1].load(in + 32 * sizeof(T));
    } else {
      r[0].zero();
      r[1].zero();
    }
    ahead += STEP;
    in += in_step;
  };
#pragma unroll
  for (int u = 0; u < FLY; ++u) fetch(raw[u]);
  if (pid < 0) {
    if (p.page >= 0 && threadIdx.x == 0) flag(a, KVQ_ERR_PAGE);
    return;
  }
  const size_t row0 = row0_of(a, a.layer0 + p.layer, pid, p.h);
  uint8_t* code = (is_v ? a.v_code : a.k_code) + row0 * ROW + cell * BITS;
  __half2* scale = (is_v ? a.v_scale : a.k_scale) + row0 * G + grp;
  const bool mean = p.s1 == a.page && a.k_mean != nullptr;
  // Rows of slot t belong to the lanes with rsub = t mod STEP, and a lane sums s n and lo of its rows
  // in their order, so a page's mean is one sum however its tokens arrived.
  F2 acc[2][4];
  float los = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i / 4][i % 4] = F2(0.f);
  if (mean && !is_v)
    for (int t = rsub; t < p.s0; t += STEP) {
      Cell<BITS> c[2];
      c[0].load(code + (size_t)t * ROW);
      c[1].load(code + (size_t)t * ROW + 4 * G * BITS);
      const __half2 meta = scale[(size_t)t * G];
      const F2 s(__low2float(meta));
      los += __high2float(meta);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[i / 4][i % 4] = fma2(s, F2((float)c[i / 4].code(i % 4), (float)c[i / 4].code(i % 4 + 4)), acc[i / 4][i % 4]);
    }
  int t = (p.s0 & ~(STEP - 1)) + rsub;
  code += (size_t)t * ROW;
  scale += (size_t)t * G;
  for (int base = p.s0 & ~(STEP - 1); base < p.s1;) {
#pragma unroll
    for (int u = 0; u < FLY; ++u) {
      if (base >= p.s1) break;             // the same for the whole CTA
      __half2 meta;
      const Scale sc = scale_of<T, BITS>(group_range(raw[u]), meta);
      if (t >= p.s0 && t < p.s1) {
        if ((l16 & 3) == 0) *scale = meta;
        los += sc.lo;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          F2 nf[4];
          Cell<BITS> c;
          codes_of<T, BITS>(raw[u][j], sc, c, nf);
          c.store(code + j * 4 * G * BITS);
          if (mean && !is_v) {
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][k] = fma2(F2(sc.s), nf[k], acc[j][k]);
          }
        }
      }
      fetch(raw[u]);
      base += STEP;
      t += STEP;
      code += STEP * ROW;
      scale += STEP * G;
    }
  }
  if (!mean) return;   // the same for the whole CTA
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = acc[i / 4][i % 4].get();
      sums[rsub][ch + i / 4 * 32 + i % 4] = y.x + los;
      sums[rsub][ch + i / 4 * 32 + i % 4 + 4] = y.y + los;
    }
  }
  __syncthreads();
  __nv_bfloat16* out = a.k_mean + (row0 >> a.page_log2) * D;
  const float inv = 1.f / (float)a.page;   // a power of two
  for (int c = threadIdx.x; c < D; c += kWriteThreads) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < STEP; ++r) s += sums[r][c];
    out[c] = __float2bfloat16_rn(s * inv);
  }
}

template <typename T, int BITS, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Args a, Rows k, Rows v, const int32_t* __restrict__ pos,
                                                        const int32_t* __restrict__ count) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = 2 * RPW, G = D / kGroup, ROW = D * BITS / 8;
  Piece p;
  if (!piece_of(a, pos, count, &p)) return;
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
  const dim3 grid((unsigned)pieces * a.Hkv, a.B, a.n_layers);
#define LOWRAM_KVQ_GO(D)                                                              \
  if constexpr (WRITE) write_kernel<T, BITS, D><<<grid, kWriteThreads, 0, s>>>(a, k, v, pos, count); \
  else read_kernel<T, BITS, D><<<grid, kThreads, 0, s>>>(a, k, v, pos, count)
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
