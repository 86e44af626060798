// The attention tile of the quantised KV cache: one warp, 16 tokens at a time, 4, 8 or 16 query
// rows (query heads of one KV head, and query tokens) against all of them.
//
// Both products run on mma.sync m16n8k16 (fp16 in, fp32 out) with the CODES as the A operand
// (16 tokens, or 16 channels, a tile) and the queries as the 8 columns of B, so that few query
// rows waste little of a tile.  A code needs no conversion: its bits, masked in place in a
// 16-bit lane, ARE an fp16 number -- code n in the low mantissa bits is the subnormal n 2^-24, four
// bits higher n 2^-20 -- and products with subnormals are exact.  Unpacking is one mask per two
// codes and one shift per four.  The tile is bound by its instructions (about 2.3 of a thread per code
// at d = 128 in 4 bits, all of them counted) and their latencies, close to the rate at which HBM
// delivers 4-bit codes; the tensor pipe is 22 % busy.  That is why the matrix instruction that takes
// A from registers is used: tcgen05 reads A from shared memory, where every code would first have
// to be stored as 16 bits.
//
// Scores.  x_t = sum_g s_tg (n_tg . q_g) + lo_tg sum(q_g): the scale and the offset of a group enter
// per accumulator, in fp32, so keys are never rounded.  (fp32 calls unpack to centred codes, and
// lose nothing to sums that cancel either.)  q is multiplied by a power of two per row so that its
// largest entry lies in [2^13, 2^14): bf16 values stay exact in fp16 down to 2^-27 of the largest
// (an fp32 q is split into two fp16 parts).
//
// Values.  o_c = sum_t (p_t s_tg) (n_tc - mid) + sum_t p_t (lo_tg + mid s_tg): w = p s 2^-E (times a
// constant) is rounded to fp16 once (fp32 calls: split in two parts), E following a group's value scales so
// that w stays within fp16's normal range; the offsets are summed in fp32 beside.  A step's products
// are summed on their own and added to the output in fp32 (the tensor core's sums are cut off, not
// rounded).  p = 2^(f (x - m)) with a running m that moves only when a score passes it by some factor --
// w then still fits -- so most tiles neither reduce a maximum across lanes nor rescale.
//
// Lane l holds r = l / 4, q = l % 4:
//   A of the scores:  tokens r, r + 8; the cells 2q, 2q + 1 of every group -- one contiguous piece
//                     of the row, whose order of groups inside cells is made for this load;
//   scores C:         tokens r, r + 8 x columns 2q, 2q + 1;
//   B of the values:  C's 8 x 8 halves transposed by movmatrix;
//   A of the values:  cell r of tokens 2q, 2q + 1, 2q + 8, 2q + 9 (two tokens' words are merged, then
//                     masked); code pair (2j, 2j + 1) gives rows r, r + 8 of product j;
//   outputs C:        channels 64 g + 8 r + 2j (+ 1) x columns 2q, 2q + 1.
// With at most 4 rows, row j is column 2j: a lane then holds one row instead of two, and everything
// that is done per score and per output is halved.  The odd columns take the second part of an
// fp32 q, and the weights of the next group of channels.
#pragma once

#include "kvq.cuh"

namespace lowram {
namespace kvq {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x = hi + lo with both in fp16 (lo holds the next 11 bits)
__device__ __forceinline__ void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_h2(a - __low2float(h), b - __high2float(h));
}
template <int BYTES> __device__ __forceinline__ void lds(uint32_t (&w)[BYTES / 4], const uint8_t* p) {
  if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    w[0] = t.x;
    w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 t = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = t.x;
      w[4 * i + 1] = t.y;
      w[4 * i + 2] = t.z;
      w[4 * i + 3] = t.w;
    }
  }
}

// Codes in 16-bit lanes as they are (n 2^-24, or n 2^-20 where HIGH), or centred for fp32 calls:
// n - (2^b - 1) / 2, or 16 times that, by way of 1024 + n in fp16 (all steps exact).
template <int BITS, bool CENTRE, bool HIGH> __device__ __forceinline__ uint32_t lanes(uint32_t x) {
  constexpr uint32_t kMask = BITS == 8 ? 0x00FF00FFu : (HIGH ? 0x00F000F0u : 0x000F000Fu);
  if constexpr (!CENTRE) {
    return x & kMask;
  } else {
    const uint32_t y = (x & kMask) | 0x64006400u, c = BITS == 4 && !HIGH ? 0x64086408u : 0x64806480u;
    const uint32_t half = BITS == 4 && HIGH ? 0x48004800u : 0x38003800u;   // 8 or 0.5
    const __half2 h = __hadd2(__hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&c)),
                              *reinterpret_cast<const __half2*>(&half));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// The two 16-bit lanes of half j (0, 1) of a cell: even codes in `a`, odd ones in `b` (4 bits: 16
// times too large, made up for in B or in the output).
template <int BITS, bool CENTRE>
__device__ __forceinline__ void half_cell(const uint32_t* w, int j, uint32_t& a, uint32_t& b) {
  const uint32_t x = BITS == 4 ? (j ? w[0] >> 8 : w[0]) : w[BITS == 4 ? 0 : j];
  a = lanes<BITS, CENTRE, false>(x);
  b = lanes<BITS, CENTRE, true>(BITS == 4 ? x : x >> 8);
}
// Codes 2j, 2j + 1 of a cell of two tokens (low lanes: the first token).
template <int BITS, bool CENTRE>
__device__ __forceinline__ void pair_cell(const uint32_t* w0, const uint32_t* w1, int j, uint32_t& a, uint32_t& b) {
  uint32_t x;
  if constexpr (BITS == 4) {
    x = __byte_perm(w0[0], w1[0], j < 2 ? 0x5410 : 0x7632);
    if (j & 1) x >>= 8;
  } else {
    x = __byte_perm(w0[j / 2], w1[j / 2], j & 1 ? 0x7632 : 0x5410);
  }
  a = lanes<BITS, CENTRE, false>(x);
  b = lanes<BITS, CENTRE, true>(BITS == 4 ? x : x >> 8);
}

template <int BITS_, int D_, int ROWS_, bool F32_> struct Tile {
  static constexpr int BITS = BITS_, D = D_, ROWS = ROWS_;
  static constexpr bool F32 = F32_;
  static constexpr int CP = ROWS == 4 ? 1 : 2;        // rows a lane holds of an 8-column tile
  static constexpr int NT = ROWS == 16 ? 2 : 1;       // 8-column tiles
  static constexpr int G = D / kGroup, ROW = D * BITS / 8;
  static constexpr int SP = F32 ? 2 : 1;              // fp16 parts of w
  static constexpr int SPQ = F32 && CP == 2 ? 2 : 1;  // and of q (CP = 1: the second part is in the odd column)
  static constexpr int STEPS = 4 * G;                 // products of a score tile
  static constexpr int CODE = 16 * ROW, META = 16 * G * 4;      // bytes of 16 tokens: codes, scales
  static constexpr int BLOCK = 2 * (CODE + META);
  static constexpr int QFRAG = STEPS * NT * SPQ * 32 * 8;       // bytes of the queries' B operands
  static constexpr int QMETA = ROWS * (1 + G) * 4;              // f'' and the group sums
  static constexpr bool QREG = STEPS * NT * SPQ * 2 <= 16;       // B operands kept in registers
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  // A score may pass the running maximum by a factor of 2^kSlack in its weight, a value scale leave
  // [2^E, 2^(E+1)) by a factor of kWide either way: w <= 2^(kSlack + 1) kWide kBias = 2^15, half of what
  // fp16 holds (the other factor of two is for roundings), and what fp16's smallest step (2^-24) loses
  // is 2^-30 (fp32: 2^-33) of a weight of one.
  static constexpr int kSlackLog2 = F32 ? 2 : 4;
  static constexpr float kSlack = kSlackLog2, kWide = F32 ? 8.f : 16.f, kBias = F32 ? 512.f : 64.f;
  static_assert((1 << kSlackLog2) * 2.f * kWide * kBias <= 32768.f, "weights must stay within fp16");

  // What a code is multiplied by to be a number: fp32 calls centre their codes and have the 1.
  static constexpr float kCode = F32 ? 1.f : 16777216.f;
  // Codes are summed as n - kMid, so that an average over many tokens is not a small difference of
  // two large sums; the offsets become lo + kMid s.  kMidLow, kMidHigh: -kMid as two fp16 lanes, in
  // the units of the codes of rows r and r + 8.
  static constexpr float kMid = (BITS == 4 ? 8.f : 128.f) - (F32 ? 0.5f : 0.f);
  static constexpr uint32_t kMidLow = BITS == 4 ? 0x80088008u : 0x80808080u, kMidHigh = 0x80808080u;

  // [..][i * CP + c]: A's row r + 8 i, the lane's c-th column
  float o[NT][G][4][2 * CP], ls[NT][G][CP], l[NT][CP], qs[NT][G][CP];
  float f[NT][CP], mx[NT][CP], thr[NT][CP];           // f'', the running maximum (0 before the first), when it moves
  float unit_inv[G];                                  // of a group of channels: kBias 2^-E, 0 before the first scale
  uint32_t top_s[(G + 1) / 2];                        // the largest scales that need no new unit (fp16 bits, two groups each)
  uint2 qr[QREG ? STEPS * NT * SPQ : 1];

  // The query row of this lane's column (t, c).
  static __device__ __forceinline__ int row_of(int t, int c) {
    const int q = threadIdx.x & 3;
    return CP == 1 ? q : t * 8 + 2 * q + c;
  }

  // ---------------------------------------------------------------- queries
  // Warp w of WARPS takes the rows w, w + WARPS, ... of the tile.  fetch() starts their loads
  // (rows behind `rows` are zeros), prepare() makes the B operands and meta: [ROWS] f'', then
  // [ROWS][G] sums.
  template <int WARPS> struct Queries {
    static constexpr int PER = D / 32;   // channels of a lane, consecutive (within a cell)
    static constexpr int MINE = (ROWS + WARPS - 1) / WARPS;
    __align__(16) T raw[MINE][PER];
    template <class QRow> __device__ __forceinline__ void fetch(int rows, int warp, QRow q_row) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        const int j = warp + k * WARPS;
#pragma unroll
        for (int i = 0; i < PER; ++i) raw[k][i] = from_f<T>(0.f);
        if (j < rows) {
          const T* src = q_row(j) + lane * PER;
          constexpr int BY = PER * (int)sizeof(T);
          if constexpr (BY == 4) *reinterpret_cast<uint32_t*>(raw[k]) = __ldcg(reinterpret_cast<const uint32_t*>(src));
          else if constexpr (BY == 8) *reinterpret_cast<uint2*>(raw[k]) = __ldcg(reinterpret_cast<const uint2*>(src));
          else
#pragma unroll
            for (int i = 0; i < BY / 16; ++i) reinterpret_cast<uint4*>(raw[k])[i] = __ldcg(reinterpret_cast<const uint4*>(src) + i);
        }
      }
    }
    __device__ __forceinline__ void prepare(uint8_t* frag, float* meta, int warp) const {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        const int j = warp + k * WARPS;
        if (j >= ROWS) break;
        float x[PER], mx = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          x[i] = to_f<T>(raw[k][i]);
          mx = fmaxf(mx, fabsf(x[i]));
        }
        mx = warp_max(mx);
        // a power of two: 2^13 <= mx sigma < 2^14 (1 for a row of zeros, or with an infinity)
        const int e = (int)(__float_as_uint(mx) >> 23) - 127;
        const float sigma = e > -127 && e < 128 ? __uint_as_float((unsigned)(min(13 - e, 100) + 127) << 23) : 1.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum = fmaf(x[i], sigma, sum);   // scaled first: a sum of entries may pass fp32's range
#pragma unroll
        for (int i = 16 / G; i > 0; i >>= 1) sum += __shfl_xor_sync(kFull, sum, i);   // 32 / G lanes hold a group
        // At most 2^100 (queries from 2^113 on): scores that differ, by 2^-72 or more with what fp16 holds of q,
        // are millions apart in log2 units there, and a smaller factor gives the same weights, 0 and 1.
        if (lane == 0) meta[j] = fminf(kLog2e * rsqrtf((float)D) * (kCode / sigma), 1.2676506e30f);
        if (lane % (32 / G) == 0) meta[ROWS + j * G + lane / (32 / G)] = sum * (1.f / kCode);
        const int col = CP == 1 ? 2 * j : j % 8, tile = CP == 1 ? 0 : j / 8;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int c = lane * PER + i, g = c / 64, w = c % 64 / 8, code = c % 8;
          const int half = BITS == 4 ? code % 4 / 2 : code / 4, hi = BITS == 4 ? code / 4 : code % 4 / 2, reg = code % 2;
          float y = x[i] * sigma;
          if (BITS == 4 && reg) y *= 0.0625f;
          const int step = (g * 2 + w % 2) * 2 + half;
          __half* at = reinterpret_cast<__half*>(frag) + ((((step * NT + tile) * SPQ) * 32 + col * 4 + w / 2) * 2 + reg) * 2 + hi;
          const __half h = __float2half_rn(y);
          at[0] = h;
          if constexpr (F32) at[CP == 1 ? 4 * 4 : 32 * 4] = __float2half_rn(y - __half2float(h));   // the next column, or the next operand
        }
      }
    }
  };
  __device__ __forceinline__ void begin(const uint8_t* frag, const float* meta) {
    const int lane = threadIdx.x & 31;
    if constexpr (QREG) {
#pragma unroll
      for (int i = 0; i < STEPS * NT * SPQ; ++i) qr[i] = reinterpret_cast<const uint2*>(frag)[i * 32 + lane];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const int j = row_of(t, c);
        f[t][c] = meta[j];
        mx[t][c] = 0.f;
        thr[t][c] = -INFINITY;
        l[t][c] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          qs[t][g][c] = meta[ROWS + j * G + g];
          ls[t][g][c] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][g][k][c] = o[t][g][k][CP + c] = 0.f;
        }
      }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      unit_inv[g] = 0.f;
      top_s[g / 2] = 0;
    }
  }
  __device__ __forceinline__ uint2 qop(const uint8_t* frag, int i) const {
    if constexpr (QREG) return qr[i];
    else return reinterpret_cast<const uint2*>(frag)[i * 32 + (threadIdx.x & 31)];
  }

  // ---------------------------------------------------------------- loading
  // A slot of shared memory holds TB blocks of 16 tokens: [TB] K codes, [TB] V codes, [TB] K scales,
  // [TB] V scales.
  // Starts the copies of N blocks whose tokens follow one another from row `row` on, into the slot's
  // blocks b0, b0 + 1, ...
  template <int TB, int N> static __device__ __forceinline__ void load(const Args& a, uint32_t slot, int b0, uint32_t row) {
    const int lane = threadIdx.x & 31;
    const uint64_t at = (uint64_t)row * ROW + lane * 16;
    const uint8_t *k = a.k_code + at, *v = a.v_code + at;
    const uint32_t dst = slot + b0 * CODE + lane * 16;
#pragma unroll
    for (int i = 0; i < N * CODE / 512; ++i) {
      cp16(dst + i * 512, k + i * 512);
      cp16(dst + TB * CODE + i * 512, v + i * 512);
    }
    // the scales of K and V, half of the lanes each
    constexpr int PIECES = N * META / 16;
#pragma unroll
    for (int i = 0; i < (2 * PIECES + 31) / 32; ++i) {
      const int p = i * 32 + lane, mine = p % PIECES;
      const bool is_v = p >= PIECES;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(is_v ? a.v_scale : a.k_scale) + (uint64_t)row * (G * 4) + mine * 16;
      if (2 * PIECES % 32 == 0 || p < 2 * PIECES) cp16(slot + TB * (2 * CODE + (is_v ? META : 0)) + b0 * META + mine * 16, src);
    }
  }

  // ---------------------------------------------------------------- 16 TB tokens
  // The slot's blocks b0 .. b0 + N - 1.  Token t of the first has place tok + t; column (t, c) sees the
  // places below lim[t][c].  EDGE: some place is masked; what such a place holds (anything, NaN too)
  // plays no part.
  template <int TB, int N, bool EDGE>
  __device__ __forceinline__ void step(const uint8_t* slot, int b0, const uint8_t* frag, int tok, const int (&lim)[NT][CP]) {
    const int lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
    constexpr int CW = BITS / 4;
    const uint8_t *kc = slot + b0 * CODE, *vc = kc + TB * CODE, *km = slot + TB * 2 * CODE + b0 * META, *vmeta = km + TB * META;
    float x[N][NT][2 * CP];
    // scores, in units of 1 / f''
#pragma unroll
    for (int b = 0; b < N; ++b) {
      uint32_t k0[2 * G * CW], k1[2 * G * CW];
      lds<2 * G * BITS>(k0, kc + b * CODE + r * ROW + q * 2 * G * BITS);
      lds<2 * G * BITS>(k1, kc + b * CODE + (r + 8) * ROW + q * 2 * G * BITS);
      uint32_t m0[G], m1[G];
      lds<4 * G>(m0, km + b * META + r * 4 * G);
      lds<4 * G>(m1, km + b * META + (r + 8) * 4 * G);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2 * CP; ++k) x[b][t][k] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[t][k] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            half_cell<BITS, F32>(k0 + (e * G + g) * CW, h, a0, a2);
            half_cell<BITS, F32>(k1 + (e * G + g) * CW, h, a1, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int s = 0; s < SPQ; ++s) mma_f16(acc[t], a0, a1, a2, a3, qop(frag, (((g * 2 + e) * 2 + h) * NT + t) * SPQ + s));
          }
        if constexpr (F32 && CP == 1) {   // the two parts of q
          acc[0][0] += acc[0][1];
          acc[0][2] += acc[0][3];
        }
        float2 u0 = __half22float2(*reinterpret_cast<const __half2*>(&m0[g]));
        float2 u1 = __half22float2(*reinterpret_cast<const __half2*>(&m1[g]));
        if constexpr (F32) {
          u0.y = fmaf(kMid, u0.x, u0.y);
          u1.y = fmaf(kMid, u1.x, u1.y);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < CP; ++c) {
              const float2 u = i ? u1 : u0;
              float& y = x[b][t][i * CP + c];
              y = fmaf(u.x, acc[t][2 * i + c], fmaf(u.y, qs[t][g][c], y));
            }
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2 * CP; ++k)
            if (tok + 16 * b + r + 8 * (k / CP) >= lim[t][k % CP]) x[b][t][k] = -INFINITY;
      }
    }
    // value scales and offsets of the tokens r, r + 8
    uint32_t vm[N][2][G], most_s[G];    // (s, lo) pairs; a group's largest s in the low half (s >= 0, so its bits are ordered)
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lds<4 * G>(vm[b][i], vmeta + b * META + (r + 8 * i) * 4 * G);
        if constexpr (EDGE) {
          int most = lim[0][0];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < CP; ++c) most = max(most, lim[t][c]);
          if (tok + 16 * b + r + 8 * i >= most)
#pragma unroll
            for (int g = 0; g < G; ++g) vm[b][i][g] = 0;
        }
      }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      most_s[g] = __vmaxu2(vm[0][0][g], vm[0][1][g]);
      if constexpr (N == 2) most_s[g] = __vimax3_u16x2(most_s[g], vm[N - 1][0][g], vm[N - 1][1][g]);
    }
    bool high = false;
#pragma unroll
    for (int g = 0; g < G; g += 2) {
      const uint32_t two = G > 1 ? __byte_perm(most_s[g], most_s[G > 1 ? g + 1 : g], 0x5410) : most_s[g] & 0xffffu;
      high |= __vmaxu2(two, top_s[g / 2]) != top_s[g / 2];
    }
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2 * CP; ++k) high |= x[b][t][k] > thr[t][k % CP];
    if (__any_sync(kFull, high)) move<N>(x, vm);
    // weights: p in x's place, the sum of the weights
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2 * CP; ++k) {
          // the difference first: a product rounded to fp32 is off by much more than one for scores above 2^25
          const float p = ex2((x[b][t][k] - mx[t][k % CP]) * f[t][k % CP]);
          x[b][t][k] = p;
          l[t][k % CP] += p;
        }
    uint32_t v[N][4][G * CW];   // cell r of the tokens 2q, 2q + 1, 2q + 8, 2q + 9
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) lds<G * BITS>(v[b][i], vc + b * CODE + (2 * q + (i & 1) + (i >> 1) * 8) * ROW + r * G * BITS);
    // The two columns e of a lane are its two rows (CP = 2), or its one row for two groups (CP = 1):
    // then one operand of weights serves both groups, each taking its own columns of the product.
    constexpr int SETS = CP == 2 ? G : (G + 1) / 2;
#pragma unroll
    for (int gs = 0; gs < SETS; ++gs) {
      uint2 w[N][NT][SP];
      float base[NT][4];   // -kMid sum_t w_t in every row: the products below then add w (n - kMid) (fp32: 0)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) base[t][k] = 0.f;
#pragma unroll
      for (int b = 0; b < N; ++b) {
        float2 u[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < (CP == 1 && G > 1 ? 2 : 1); ++e) {
            const float2 m = __half22float2(*reinterpret_cast<const __half2*>(&vm[b][i][CP == 2 ? gs : 2 * gs + e]));
            u[i][e] = make_float2(m.x * unit_inv[CP == 2 ? gs : 2 * gs + e], fmaf(kMid, m.x, m.y));
          }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float y[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = CP == 2 ? e : 0, g = CP == 2 ? gs : 2 * gs + e;
              if (g >= G) continue;
              const float2 ue = u[i][CP == 2 ? 0 : e];
              const float p = x[b][t][i * CP + c];
              y[i][e] = p * ue.x;
              if constexpr (EDGE) {   // a place this column does not see may hold anything
                const bool seen = tok + 16 * b + r + 8 * i < lim[t][c];
                y[i][e] = seen ? y[i][e] : 0.f;
                ls[t][g][c] += seen ? p * ue.y : 0.f;
              } else {
                ls[t][g][c] = fmaf(p, ue.y, ls[t][g][c]);
              }
            }
          if constexpr (F32) {
            uint32_t h0, h1, l0, l1;
            split_h2(y[0][0], y[0][1], h0, l0);
            split_h2(y[1][0], y[1][1], h1, l1);
            w[b][t][0] = make_uint2(trans8x8(h0), trans8x8(h1));
            w[b][t][SP - 1] = make_uint2(trans8x8(l0), trans8x8(l1));
          } else {
            w[b][t][0] = make_uint2(trans8x8(pack_h2(y[0][0], y[0][1])), trans8x8(pack_h2(y[1][0], y[1][1])));
          }
          if constexpr (!F32) mma_f16(base[t], kMidLow, kMidHigh, kMidLow, kMidHigh, w[b][t][0]);
        }
      }
#pragma unroll
      for (int ge = 0; ge < (CP == 1 ? 2 : 1); ++ge) {
        const int g = CP == 2 ? gs : 2 * gs + ge;
        if (g >= G) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float acc[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[t][k] = base[t][k];
#pragma unroll
          for (int b = 0; b < N; ++b) {
            uint32_t a0, a1, a2, a3;
            pair_cell<BITS, F32>(v[b][0] + g * CW, v[b][1] + g * CW, j, a0, a1);
            pair_cell<BITS, F32>(v[b][2] + g * CW, v[b][3] + g * CW, j, a2, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = SP - 1; i >= 0; --i) mma_f16(acc[t], a0, a1, a2, a3, w[b][t][i]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int c = 0; c < CP; ++c) o[t][g][j][i * CP + c] += acc[t][2 * i + (CP == 2 ? c : ge)];
        }
      }
    }
  }

  // A score passed the running maximum, or a value scale its unit's room: both anew.  A unit that
  // has become far too large is made smaller here as well: the scales it was made for have lost
  // their weight only if the maximum has moved.
  template <int TB> __device__ __forceinline__ void move(const float (&x)[TB][NT][2 * CP], const uint32_t (&vm)[TB][2][G]) {
    float scale[G];
    uint32_t sb[G];   // the largest finite scale (one that is not spoils the rows that see it, but not the unit)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sb[g] = 0;
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t s16 = vm[b][i][g] & 0xffffu;
          sb[g] = max(sb[g], s16 < 0x7c00u ? s16 : 0u);
        }
      sb[g] = __reduce_max_sync(kFull, sb[g]);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t top = g & 1 ? top_s[g / 2] >> 16 : top_s[g / 2] & 0xffffu;
      const float s = __half2float(__ushort_as_half((unsigned short)sb[g])), old = unit_inv[g];
      const bool anew = sb[g] && (old == 0.f || sb[g] > top || !(s * old > kBias / kWide));
      // powers of two, whose reciprocals are exponents: kBias <= s inv < 2 kBias
      const uint32_t two_e = __float_as_uint(s) & 0x7f800000u;
      const float inv = kBias * __uint_as_float((254u << 23) - two_e), over = old == 0.f ? 1.f : __uint_as_float((254u << 23) - __float_as_uint(old));
      const uint32_t room = __half_as_ushort(__float2half_rz(fminf(kWide * 2.f * __uint_as_float(two_e), 65504.f)));
      scale[g] = anew && old != 0.f ? inv * over : 1.f;
      unit_inv[g] = anew ? inv : old;
      if (anew) top_s[g / 2] = __byte_perm(top_s[g / 2], room, g & 1 ? 0x5410 : 0x3254);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        float most = -INFINITY;
#pragma unroll
        for (int b = 0; b < TB; ++b) most = fmaxf(most, fmaxf(x[b][t][c], x[b][t][CP + c]));
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, i));
        float alpha = 1.f;
        if (most > thr[t][c]) {
          alpha = thr[t][c] == -INFINITY ? 0.f : ex2((mx[t][c] - most) * f[t][c]);
          mx[t][c] = most;
          thr[t][c] = __fadd_rd(most, __fdividef(kSlack, f[t][c]));   // rounded down: no weight above 2^kSlack
          l[t][c] *= alpha;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float both = alpha * scale[g];
          ls[t][g][c] *= alpha;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[t][g][j][c] *= both;
            o[t][g][j][CP + c] *= both;
          }
        }
      }
  }

  // ---------------------------------------------------------------- end
  // Running maximum of column (t, c), -inf without a token; after reduce().  Where a score was NaN the
  // sum of the weights is, and counts against any other maximum: as +inf, whose factor is NaN.
  __device__ __forceinline__ float top(int t, int c) const {
    return l[t][c] != l[t][c] ? INFINITY : (thr[t][c] == -INFINITY ? -INFINITY : mx[t][c]);
  }
  // What sums with the running maximum m are multiplied by to be joined under the maximum `to`; f: the
  // row's f''.
  static __device__ __forceinline__ float factor(float m, float to, float f) { return m == -INFINITY ? 0.f : ex2((m - to) * f); }
  // Adds up what lanes hold apart: sums of the weights and of the offsets' part.
  __device__ __forceinline__ void reduce() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < CP; ++c)
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          l[t][c] += __shfl_xor_sync(kFull, l[t][c], i);
#pragma unroll
          for (int g = 0; g < G; ++g) ls[t][g][c] += __shfl_xor_sync(kFull, ls[t][g][c], i);
        }
  }
  // Leaves the maxima and the sums of the weights of this warp's rows (after reduce()).
  __device__ __forceinline__ void store_tops(float* tops, float* sums) const {
    if ((threadIdx.x & 31) < 4) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < CP; ++c) {
          tops[row_of(t, c)] = top(t, c);
          sums[row_of(t, c)] = l[t][c];
        }
    }
  }
  // The unnormalised outputs [ROWS][D], times weight(row) (0 leaves NaN of the values as it is).
  template <class Weight> __device__ __forceinline__ void store_out(float* to, Weight weight) const {
    const int r = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const int j = row_of(t, c);
        const float w = weight(j);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float u0 = unit_inv[g] == 0.f ? 0.f : kCode * __uint_as_float((254u << 23) - __float_as_uint(unit_inv[g])), u1 = BITS == 4 ? u0 * 0.0625f : u0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = make_float2(fmaf(o[t][g][k][c], u0, ls[t][g][c]), fmaf(o[t][g][k][CP + c], u1, ls[t][g][c]));
            *reinterpret_cast<float2*>(to + j * D + 64 * g + 8 * r + 2 * k) = make_float2(v.x * w, v.y * w);
          }
        }
      }
  }
};

}  // namespace kvq
}  // namespace lowram
