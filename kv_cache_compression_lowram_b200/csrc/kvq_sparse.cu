// Quantised KV cache: attention over the pages that their mean keys select for each query.
//
// One launch.  A unit -- (layer, sequence, query token, KV head) -- belongs to a cluster of 1 to 8
// CTAs, which do all of it together through each other's shared memory:
//   1. each CTA scores its share of the full pages (mean key . sum of the group's queries) into its
//      shared memory: 2 d bytes a page, the larger part of what a long context costs.  In fp32, with a
//      bound on how far that is from the score in 64 bits that selection goes by (16 sequences of up to
//      64K, a CTA's scoring: 12.6 us in fp64, 11.2 in fp32, 8.4 with the keys copied through a ring);
//   2. every CTA gathers all scores and finds the same top_k - 1 best pages: a histogram over the
//      range of the scores leaves a bin that holds the border (a bin of many pages is cut again);
//      pages further from it than twice the bound are decided, and the few others are scored once
//      more in fp64 and ranked by comparison;
//   3. the selected pages' 16-token blocks go round the warps of the cluster, as in the attention
//      over whole sequences; CTAs join their sums and the cluster joins the CTAs'.
// No workspace, no second launch, and nothing is written but the outputs.  (d = 128 in 4 bits, four rows: two
// CTAs an SM, 128 registers, and 48 bytes a thread stored to memory and 84 loaded.)  One 128K sequence, 32 of 2048
// pages of 64: 20 us, of which the histogram and the ranks take 5, the gathering of scores and the
// queries 2 each, scoring 3, attention 2.  16 sequences of up to 64K, 2 layers: 45 us for 109 MB,
// 2.4 TB/s: the longest sequence's steps in a row, half of it attention at the rate of whole sequences.
#include <cooperative_groups.h>
#include <limits.h>

#include <atomic>

#include "kvq.cuh"
#include "kvq_attend.cuh"

namespace cg = cooperative_groups;

namespace lowram {
namespace kvq {
namespace {

constexpr int kWarps = 8;     // (four: 63 us instead of 52 for the 16 sequences)
constexpr int kThreads = 32 * kWarps;
constexpr int kBins = 1024;
constexpr int kDeep = 4;      // stages of mean keys on their way
constexpr int kRank = 256;    // members of a border bin that are ranked by comparison

template <int BITS, int D, int ROWS, bool F32> struct Plan {
  using Tl = Tile<BITS, D, ROWS, F32>;
  static constexpr int TB = Tl::BLOCK <= 2304 ? 2 : 1;
  static constexpr int SLOT = TB * Tl::BLOCK;
  static constexpr int STAGES = 2;
  static constexpr int RING = kWarps * STAGES * SLOT;
  static constexpr int JOIN = kWarps * ROWS * D * 4;
  // what lives at once: the ring and the joined sums, or the scores and the histogram
  static constexpr int ATTEND = RING + JOIN + Tl::QFRAG;
  // scoring: a ring of mean keys per warp, kDeep stages of 4 x 512 bytes
  static constexpr int MEANS = kWarps * kDeep * 2048;
  static constexpr int SMALL = Tl::QMETA + kWarps * ROWS * 8 + 2 * ROWS * 4;
  static constexpr int MINB = ATTEND <= 100 * 1024 ? 2 : 1;
};

// Integers in the order of the numbers, and back.
__device__ __forceinline__ int key_of(float f) {
  const int b = __float_as_int(f);
  return b ^ (b < 0 ? 0x7fffffff : 0);
}
__device__ __forceinline__ float float_of(int k) { return __int_as_float(k ^ (k < 0 ? 0x7fffffff : 0)); }
// The same of a score, 0 the smallest; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ double plain_score(double s) { return s == s ? s + 0.0 : -INFINITY; }
__device__ __forceinline__ unsigned long long bits_of(double s) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(s);
  return b ^ (b >> 63 ? ~0ull : 1ull << 63);
}

struct Select {   // shared by the CTA while it selects
  unsigned hist[kBins];
  int wide[2][kWarps];
  unsigned sums[kWarps];
  int border, above, members, list[kRank];
  float bound[kWarps];   // of the norms of this CTA's means (read by the cluster)
  double score[kRank];
};

// x summed over the threads up to this one.  A barrier is inside; `sums` may be written anew after the next.
__device__ __forceinline__ unsigned scan_cta(unsigned x, unsigned* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += sums[w];
  return x;
}
__device__ __forceinline__ unsigned sum_cta(unsigned x, unsigned* sums) {
  x = __reduce_add_sync(kFull, x);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) x += sums[w];
  __syncthreads();
  return x;
}
__device__ __forceinline__ void range_cta(int& mn, int& mx, int (&wide)[2][kWarps]) {
  mx = __reduce_max_sync(kFull, mx);
  mn = __reduce_min_sync(kFull, mn);
  if ((threadIdx.x & 31) == 0) {
    wide[0][threadIdx.x >> 5] = mx;
    wide[1][threadIdx.x >> 5] = mn;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    mx = max(mx, wide[0][w]);
    mn = min(mn, wide[1][w]);
  }
}

// Marks (bits of `mark`, zeroed here) the `want` largest of n scores, 0 < want < n; equal ones from the
// lowest index on.  keys[i]: score i to within `off`, as key_of(); mn, mx: this thread's smallest and
// largest key; exact(members): makes s.score[j] score s.list[j] for all j.  False (and nothing marked)
// where more than kRank pages are too near to one another for that.  All threads of the CTA.
template <class Exact>
__device__ __forceinline__ bool select_largest(const int* keys, int n, int want, float off, int mn, int mx, unsigned* mark, Select& s, Exact exact) {
  const int tid = threadIdx.x;
  for (int i = tid; i < (n + 31) / 32; i += kThreads) mark[i] = 0;
  int lo = INT_MIN, hi = INT_MAX, left = want;   // the keys that may be the want-th, and its place among them
  bool linear = true;
  for (;;) {
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    if (tid == 0) s.members = 0;
    range_cta(mn, mx, s.wide);
    // bins: even in the scores at first (unless one is infinite), then even in the keys
    const float smin = float_of(mn), span = float_of(mx) - smin, scale = (kBins - 1) / span;
    linear = linear && span > 0.f && span < 1e38f && scale < 1e38f;
    const unsigned width = (unsigned)mx - (unsigned)mn;
    const int shift = max(0, 22 - __clz((int)width));
    auto bin_of = [&](int k) { return linear ? min((int)((float_of(k) - smin) * scale), kBins - 1) : (int)(((unsigned)k - (unsigned)mn) >> shift); };
#pragma unroll 2
    for (int i = tid; i < n; i += kThreads) {
      const int k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&s.hist[bin_of(k)], 1u);
    }
    __syncthreads();
    // the bin of the left-th largest: thread t sums bins from the top, kBins / kThreads each
    constexpr int PER = kBins / kThreads;
    unsigned sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += s.hist[kBins - 1 - tid * PER - i];
    const unsigned inc = scan_cta(sum, s.sums);
    unsigned before = inc - sum;
    if (before < (unsigned)left && inc >= (unsigned)left) {   // one thread
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = kBins - 1 - tid * PER - i;
        const unsigned h = s.hist[b];
        if (before < (unsigned)left && before + h >= (unsigned)left) {
          s.border = b;
          s.above = before;
        }
        before += h;
      }
    }
    __syncthreads();
    const int border = s.border;
    left -= s.above;
    const bool few = s.hist[border] <= kRank || mn == mx;
    int nlo = INT_MAX, nhi = INT_MIN;      // the border bin's keys
#pragma unroll 2
    for (int i = tid; i < n; i += kThreads) {
      const int k = keys[i];
      if (k >= lo && k <= hi && bin_of(k) == border) {
        nlo = min(nlo, k);
        nhi = max(nhi, k);
      }
    }
    __syncthreads();
    mn = nlo;
    mx = nhi;
    range_cta(nlo, nhi, s.wide);
    lo = nlo;
    hi = nhi;
    linear = false;
    __syncthreads();
    if (few) break;
  }
  // the want-th largest of the keys lies in [lo, hi]: that of the scores is within `off` of it
  const float over = float_of(hi) + 2.f * off, under = float_of(lo) - 2.f * off;
  unsigned in = 0;
#pragma unroll 2
  for (int i = tid; i < n; i += kThreads) {
    const float x = float_of(keys[i]);
    if (x > over) {
      atomicOr(&mark[i >> 5], 1u << (i & 31));
      ++in;
    } else if (!(x < under)) {
      const int at = atomicAdd(&s.members, 1);
      if (at < kRank) s.list[at] = i;
    }
  }
  want -= sum_cta(in, s.sums);
  const int members = s.members;
  if (members > kRank) return false;
  exact(members);
  __syncthreads();
  for (int j = tid; j < members; j += kThreads) {
    const int i = s.list[j];
    const double x = s.score[j];
    int r = 0;
    for (int t = 0; t < members; ++t) r += s.score[t] > x || (s.score[t] == x && s.list[t] < i);
    if (r < want) atomicOr(&mark[i >> 5], 1u << (i & 31));
  }
  __syncthreads();
  return true;
}

// The same without bounds, for scores too near to one another (mostly equal ones): the want-th largest
// bit by bit from the top of its 64-bit key, then equal ones from the lowest index on.
template <class Score> __device__ __noinline__ void select_exactly(int n, int want, unsigned* mark, Select& s, Score score) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < (n + 31) / 32; i += kThreads) mark[i] = 0;
  auto bits = [&](int i) { return bits_of(score(i)); };
  const unsigned long long one = bits(0);
  bool differ = false;
  for (int i = tid; i < n; i += kThreads) differ |= bits(i) != one;
  differ = __syncthreads_or(differ);
  unsigned long long top = differ ? 0 : one;   // the bits so far
  for (int bit = differ ? 63 : -1; bit >= 0; --bit) {
    const unsigned long long next = top | 1ull << bit;
    unsigned c = 0;
    for (int i = tid; i < n; i += kThreads) c += bits(i) >= next;
    if (sum_cta(c, s.sums) >= (unsigned)want) top = next;
  }
  unsigned over = 0;
  for (int i = tid; i < n; i += kThreads)
    if (bits(i) > top) {
      atomicOr(&mark[i >> 5], 1u << (i & 31));
      ++over;
    }
  want -= sum_cta(over, s.sums);
  if (warp == 0)
    for (int i = 0; i < n && want > 0; i += 32) {
      const bool is = i + lane < n && bits(i + lane) == top;
      const unsigned m = __ballot_sync(kFull, is);
      if (is && __popc(m & ((1u << lane) - 1)) < want) atomicOr(&mark[(i + lane) >> 5], 1u << lane);
      want -= __popc(m);
    }
  __syncthreads();
}

template <int BITS, int D, int ROWS, bool F32>
__global__ void __launch_bounds__(kThreads, Plan<BITS, D, ROWS, F32>::MINB)
sparse_kernel(Args a, int top_k, int share_room, int score_room, const void* qv, const int32_t* __restrict__ lens, void* outv,
              int32_t* __restrict__ sel) {
  using P = Plan<BITS, D, ROWS, F32>;
  using Tl = typename P::Tl;
  using T = typename Tl::T;
  constexpr int TB = P::TB;
  extern __shared__ __align__(128) uint8_t sm[];
  // attending: ring, joined sums, the queries' operands; selecting: this CTA's scores, everyone's keys
  uint8_t* frag = sm + P::RING + P::JOIN;
  float* join = reinterpret_cast<float*>(sm + P::RING);
  int* keys = reinterpret_cast<int*>(sm);                                           // [max_pages]
  uint8_t* scores = sm + (a.max_pages * 4 + 15) / 16 * 16;
  float* mine = reinterpret_cast<float*>(scores);                                   // [share], later as doubles
  const int body = max(P::ATTEND, score_room);
  unsigned* mark = reinterpret_cast<unsigned*>(sm + body);                          // [max_pages / 32]
  int* list = reinterpret_cast<int*>(mark + (a.max_pages + 31) / 32);               // [top_k] pages, ascending
  float* meta = reinterpret_cast<float*>(list + top_k);
  float* tops = meta + Tl::QMETA / 4;
  float* norm = tops + 2 * kWarps * ROWS;                                           // [ROWS] maxima, [ROWS] sums
  __shared__ Select s;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned unit = blockIdx.x / CS;   // ((layer * B + b) * n + i) * Hkv + h
  const int h = unit % a.Hkv, i = unit / a.Hkv % a.n, b = unit / a.Hkv / a.n % a.B, layer = unit / a.Hkv / a.n / a.B;
  if (rank == 0 && tid == 0 && i == 0 && h == 0 && layer == 0 && len_bad(a, lens, b)) flag(a, KVQ_ERR_RANGE);
  const int lim = len_of(a, lens, b) - a.n + 1 + i, last = lim > 0 ? (lim - 1) >> a.page_log2 : -1;
  const T* q = static_cast<const T*>(qv) + (size_t)unit * a.g * D;
  T* out = static_cast<T*>(outv) + (size_t)unit * a.g * D;
  if (last < 0) {                          // no token: the whole cluster leaves
    for (int e = rank * kThreads + tid; e < a.g * D; e += CS * kThreads) out[e] = from_f<T>(0.f);
    if (sel && rank == 0)
      for (int k = tid; k < top_k; k += kThreads) sel[(size_t)unit * top_k + k] = -1;
    return;
  }
  int cnt = last + 1;                      // pages attended
  if (top_k <= last) {
    // 1. scores of the full pages [c0, c1)
    const int share = (last + CS - 1) / CS, c0 = min(rank * share, last), c1 = min(c0 + share, last);
    constexpr int LPP = D / 8, PPW = 32 / LPP, FLY = 4, STEP = PPW * FLY;   // 16, 8 or 4 pages a stage
    const int c8 = lane % LPP;
    if (top_k > 1) {
      auto ask = [&](int base) {
        int pid = -2;
        if (lane < STEP && base + lane < c1) pid = page_of(a, b, base + lane);
        return pid;
      };
      int pid = ask(c0 + warp * STEP);
      double qs[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) qs[k] = 0.0;
#pragma unroll 1
      for (int j = 0; j < a.g; j += 4) {   // four rows on their way at once
        __align__(16) T x[4][8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint4* src = reinterpret_cast<const uint4*>(q + (size_t)min(j + r, a.g - 1) * D + c8 * 8);
#pragma unroll
          for (int k = 0; k < (int)sizeof(x[0]) / 16; ++k) reinterpret_cast<uint4*>(x[r])[k] = __ldcg(src + k);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j + r < a.g) {
#pragma unroll
            for (int k = 0; k < 8; ++k) qs[k] += (double)to_f<T>(x[r][k]);
          }
      }
      F2 q2[4];
      float qn = 0.f;                      // the squared norm of all channels
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q2[k] = F2((float)qs[2 * k], (float)qs[2 * k + 1]);
        const float2 y = q2[k].get();
        qn = fmaf(y.x, y.x, fmaf(y.y, y.y, qn));
      }
#pragma unroll
      for (int o = 1; o < LPP; o <<= 1) qn += __shfl_xor_sync(kFull, qn, o);
      const uint32_t row = (uint32_t)(row0_of(a, a.layer0 + layer, 0, h) >> a.page_log2);
      auto mean_at = [&](int p) { return reinterpret_cast<const uint4*>(a.k_mean + (size_t)(row + (uint32_t)p * a.Hkv) * D) + c8; };
      // kDeep - 1 stages are on their way; a lane reads only what it copied itself
      uint4* ring = reinterpret_cast<uint4*>(scores + (share_room * 4 + 15) / 16 * 16) + (warp * kDeep * FLY) * 32 + lane;
      int in = 0, rd = 0, next = c0 + (warp + kWarps) * STEP;
      auto issue = [&]() {
        if (pid == -1) flag(a, KVQ_ERR_PAGE);
        const int now = pid;
        pid = ask(next);
        next += kWarps * STEP;
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int p = __shfl_sync(kFull, now, f * PPW + lane / LPP);
          uint4* to = ring + (in * FLY + f) * 32;
          if (p >= 0) cp16(smem_u32(to), mean_at(p));
          else *to = make_uint4(0x7fc07fc0u, 0, 0, 0);   // a page that is not there scores NaN
        }
        cp_commit();
        in = in + 1 == kDeep ? 0 : in + 1;
      };
#pragma unroll 1
      for (int k = 0; k < kDeep - 1; ++k) issue();
      float mn2 = 0.f;                     // this lane's channels: the largest squared norm
      for (int base = c0 + warp * STEP; base < c1; base += kWarps * STEP) {
        cp_wait<kDeep - 2>();
        float x[FLY];
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const uint4 m4 = ring[(rd * FLY + f) * 32];
          const uint32_t v[4] = {m4.x, m4.y, m4.z, m4.w};
          F2 dot(0.f), norm(0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const F2 m(__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xffff0000u));
            dot = fma2(q2[k], m, dot);
            norm = fma2(m, m, norm);
          }
          const float2 d = dot.get(), nn = norm.get();
          x[f] = d.x + d.y;
          mn2 = fmaxf(mn2, nn.x + nn.y);   // (NaN, of a page that scores -infinity, plays no part)
        }
        rd = rd + 1 == kDeep ? 0 : rd + 1;
        issue();
        // sums over the LPP lanes of a page: lanes trade halves of their pages, and after two trades a lane
        // holds one page, whose bits its own low bits chose
        int have = FLY;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          have >>= 1;
          const int o = 1 << t;
          const bool up = lane & o;
#pragma unroll
          for (int f = 0; f < FLY / 2; ++f)
            if (f < have) {
              const float keep = up ? x[f + have] : x[f], give = up ? x[f] : x[f + have];
              x[f] = keep + __shfl_xor_sync(kFull, give, o);
            }
        }
#pragma unroll
        for (int o = 4; o < LPP; o <<= 1) x[0] += __shfl_xor_sync(kFull, x[0], o);
        const int f = (lane & 1) * 2 + (lane >> 1 & 1), c = base + f * PPW + lane / LPP;
        if (c8 < 4 && c < c1) mine[c - c0] = x[0] == x[0] ? x[0] : -INFINITY;
      }
      cp_wait<0>();
      // A score is the sum over LPP lanes of 4 packed products each, from a sum of queries rounded once: off
      // by at most 12 roundings of 2^-24 relative to sum |q m| <= |q| |m|, and the square roots' own.
#pragma unroll
      for (int o = 16; o >= LPP; o >>= 1) mn2 = fmaxf(mn2, __shfl_xor_sync(kFull, mn2, o));
#pragma unroll
      for (int o = 1; o < LPP; o <<= 1) mn2 += __shfl_xor_sync(kFull, mn2, o);
      if (lane == 0) s.bound[warp] = mn2;
      // 2. everyone's scores, and the best of them
      cluster.sync();
      float most_n = 0.f;
      for (int k = lane; k < CS * kWarps; k += 32) most_n = fmaxf(most_n, cluster.map_shared_rank(s.bound, k / kWarps)[k % kWarps]);
      most_n = warp_max(most_n);
      // 2^-20 of the norms; no bound where a square or a product may have underflowed
      const float off = qn > 1e-25f && most_n > 1e-25f ? 9.5367432e-7f * sqrtf(qn) * sqrtf(most_n) : INFINITY;
      int mn = INT_MAX, mx = INT_MIN;
#pragma unroll 8
      for (int c = tid; c < last; c += kThreads) {
        const int r = c / share, k = key_of(cluster.map_shared_rank(mine, r)[c - r * share]);
        keys[c] = k;
        mn = min(mn, k);
        mx = max(mx, k);
      }
      __syncthreads();
      // the score of page c in 64 bits, by LPP lanes together
      auto score64 = [&](int c) {
        const int p = page_of(a, b, c);
        double x = NAN;
        if (p >= 0) {
          const uint4 m = __ldg(mean_at(p));
          const uint32_t v[4] = {m.x, m.y, m.z, m.w};
          x = 0.0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x = fma(qs[2 * k], (double)__uint_as_float(v[k] << 16), x);
            x = fma(qs[2 * k + 1], (double)__uint_as_float(v[k] & 0xffff0000u), x);
          }
        }
#pragma unroll
        for (int o = LPP / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
        return plain_score(x);
      };
      const bool done = select_largest(keys, last, top_k - 1, off, mn, mx, mark, s, [&](int members) {
        for (int j0 = warp * PPW; j0 < members; j0 += kWarps * PPW) {
          const int j = min(j0 + lane / LPP, members - 1);
          const double x = score64(s.list[j]);
          if (c8 == 0) s.score[j] = x;
        }
      });
      cluster.sync();                      // `mine` may be overwritten from here on
      if (!done) {                         // the same in all CTAs: they have the same keys
        double* all = reinterpret_cast<double*>(scores);
        for (int c = c0 + warp * PPW; c < c1; c += kWarps * PPW) {
          const int cc = min(c + lane / LPP, c1 - 1);
          const double x = score64(cc);
          if (c8 == 0) all[cc - c0] = x;
        }
        cluster.sync();
        select_exactly(last, top_k - 1, mark, s, [&](int c) {
          const int r = c / share;
          return cluster.map_shared_rank(all, r)[c - r * share];
        });
        cluster.sync();
      }
    } else {
      for (int k = tid; k < (last + 31) / 32; k += kThreads) mark[k] = 0;
      __syncthreads();
    }
    // the selected pages in ascending order, the newest behind them
    const int words = (last + 31) / 32;
    int before = 0;
    for (int w0 = 0; w0 < words; w0 += kThreads) {
      const unsigned m = w0 + tid < words ? mark[w0 + tid] : 0;
      int at = before + scan_cta(__popc(m), s.sums) - __popc(m);
      for (unsigned left = m; left; left &= left - 1) list[at++] = (w0 + tid) * 32 + __ffs(left) - 1;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) before += s.sums[w];
      __syncthreads();
    }
    if (tid == 0) list[before] = last;
    cnt = before + 1;
  } else {
    for (int k = tid; k <= last; k += kThreads) list[k] = k;
  }
  __syncthreads();
  if (sel && rank == 0)
    for (int k = tid; k < top_k; k += kThreads) sel[(size_t)unit * top_k + k] = k < cnt ? list[k] : -1;

  // 3. the pages' blocks, TB to a step, steps round the cluster's warps
  const int per = a.page >> 4, blocks = (cnt - 1) * per + ((lim - (last << a.page_log2) + 15) >> 4);
  const int steps = (blocks + TB - 1) / TB, stride = CS * kWarps;
  uint8_t* ring = sm + warp * P::STAGES * P::SLOT;
  const uint32_t ring_u = smem_u32(ring), unit_row = (uint32_t)row0_of(a, a.layer0 + layer, 0, h);
  for (int row_base = 0; row_base < a.g; row_base += ROWS) {
    const int rows = min(ROWS, a.g - row_base);
    int in = 0, rd = 0, xa = rank * kWarps + warp;
    unsigned bad = 0;
    auto issue = [&](int place) {
      if (xa < steps) {
        const uint32_t dst = ring_u + in * P::SLOT;
        const int blk = xa * TB, slot = blk / per;
        if (per >= TB) {                   // the step lies in one page
          const int pid = page_of(a, b, list[slot]);
          if (pid >= 0) Tl::template load<TB, TB>(a, dst, 0, unit_row + ((uint32_t)(pid * a.Hkv) << a.page_log2) + (blk - slot * per) * 16);
          else bad |= ((1u << TB) - 1) << (place * TB);
          if (pid < 0 && lane == 0) flag(a, KVQ_ERR_PAGE);
        } else {
#pragma unroll
          for (int k = 0; k < TB; ++k) {
            const int pid = blk + k < blocks ? page_of(a, b, list[blk + k]) : -2;
            if (pid >= 0) Tl::template load<TB, 1>(a, dst, k, unit_row + ((uint32_t)(pid * a.Hkv) << a.page_log2));
            else bad |= 1u << (place * TB + k);
            if (pid == -1 && lane == 0) flag(a, KVQ_ERR_PAGE);
          }
        }
        in = in + 1 == P::STAGES ? 0 : in + 1;
        xa += stride;
      }
      cp_commit();
    };
    typename Tl::template Queries<kWarps> qr;
    qr.fetch(rows, warp, [&](int j) { return q + (size_t)(row_base + j) * D; });
#pragma unroll 1
    for (int k = 0; k < P::STAGES - 1; ++k) issue(k);
    qr.prepare(frag, meta, warp);
    __syncthreads();
    Tl tile;
    tile.begin(frag, meta);
    int lims[Tl::NT][Tl::CP];
#pragma unroll
    for (int t = 0; t < Tl::NT; ++t)
#pragma unroll
      for (int c = 0; c < Tl::CP; ++c) lims[t][c] = lim;
    for (int x = rank * kWarps + warp; x < steps; x += stride) {
      cp_wait<P::STAGES - 2>();
      __syncwarp();
      const unsigned gone = bad & ((1u << TB) - 1);
      bad >>= TB;
      const uint8_t* slot = ring + rd * P::SLOT;
      const int blk = x * TB;
      if (gone == 0 && (blk + TB) * 16 <= lim - ((last - (cnt - 1)) << a.page_log2)) {   // behind the newest page's tokens nothing follows
        tile.template step<TB, TB, false>(slot, 0, frag, 0, lims);
      } else {
#pragma unroll 1
        for (int k = 0; k < TB; ++k) {
          const int p = (blk + k) / per;
          if (!(gone >> k & 1) && blk + k < blocks)
            tile.template step<TB, 1, true>(slot, k, frag, (list[p] << a.page_log2) + (blk + k - p * per) * 16, lims);
        }
      }
      rd = rd + 1 == P::STAGES ? 0 : rd + 1;
      __syncwarp();
      issue(P::STAGES - 2);
    }
    cp_wait<0>();
    // the CTA's warps
    tile.reduce();
    tile.store_tops(tops + warp * ROWS, tops + (kWarps + warp) * ROWS);
    __syncthreads();
    auto most = [&](int j) {
      float m = tops[j];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, tops[w * ROWS + j]);
      return m;
    };
    tile.store_out(join + warp * ROWS * D, [&](int j) {
      return Tl::factor(tops[warp * ROWS + j], most(j), meta[j]);
    });
    if (tid < ROWS) {
      const float m = most(tid);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = tops[w * ROWS + tid];
        l = fmaf(tops[(kWarps + w) * ROWS + tid], Tl::factor(mw, m, meta[tid]), l);
      }
      norm[tid] = m;
      norm[ROWS + tid] = l;
    }
    __syncthreads();
    for (int e = tid; e < rows * D / 4; e += kThreads) {   // into warp 0's place
      float4 v = reinterpret_cast<const float4*>(join)[e];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 y = reinterpret_cast<const float4*>(join + w * ROWS * D)[e];
        v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
      }
      reinterpret_cast<float4*>(join)[e] = v;
    }
    // the cluster's CTAs, each joining a part of the outputs
    cluster.sync();
    // CS lanes to four channels, a CTA's part each
    const int src = tid & (CS - 1);
    for (int e0 = rank * (kThreads / CS); e0 < rows * D / 4; e0 += kThreads) {
      const int e = e0 + tid / CS;
      const bool in = e < rows * D / 4;
      const int j = in ? e / (D / 4) : 0;
      const float* nr = cluster.map_shared_rank(norm, src);
      const float mr = nr[j];
      float4 v = reinterpret_cast<const float4*>(cluster.map_shared_rank(join, src))[in ? e : 0];
      float l = nr[ROWS + j], m = mr;
      for (int o = 1; o < CS; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float w = Tl::factor(mr, m, meta[j]);
      l *= w;
      v = make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
      for (int o = 1; o < CS; o <<= 1) {
        l += __shfl_xor_sync(kFull, l, o);
        v.x += __shfl_xor_sync(kFull, v.x, o);
        v.y += __shfl_xor_sync(kFull, v.y, o);
        v.z += __shfl_xor_sync(kFull, v.z, o);
        v.w += __shfl_xor_sync(kFull, v.w, o);
      }
      if (!in || src) continue;
      const float inv = m == -INFINITY ? 0.f : 1.f / l;
      T* o = out + (size_t)row_base * D + 4 * e;
      v = m == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if constexpr (F32) {
        *reinterpret_cast<float4*>(o) = v;
      } else {
        __nv_bfloat162 hv[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(hv);
      }
    }
    cluster.sync();                        // no CTA leaves, or writes its sums anew, while another reads them
  }
}

template <int BITS, int D, int ROWS, bool F32>
cudaError_t go(const Args& a, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel, cudaStream_t s) {
  using P = Plan<BITS, D, ROWS, F32>;
  // per device: clusters of 1, 2, 4, 8 CTAs resident at once, where an SM holds one CTA and where it
  // holds as many as the registers allow
  struct Fits {
    std::atomic<bool> known{false};
    std::atomic<int> clusters[2][4] = {};
    std::atomic<int> per_sm{0}, beside{0};   // shared memory of an SM, and of a CTA beside its dynamic one
  };
  static Fits fits[64];
  auto kernel = sparse_kernel<BITS, D, ROWS, F32>;
  const unsigned units = (unsigned)a.n_layers * a.B * a.n * a.Hkv;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  cfg.blockDim = kThreads;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto share_room = [&](int cs) { return (a.max_pages + cs - 1) / cs; };
  auto score_room = [&](int cs) {   // all keys, then a share's scores in fp32 and the ring, or its scores in fp64
    const int fast = (share_room(cs) * 4 + 15) / 16 * 16 + P::MEANS, exact = share_room(cs) * 8;
    return (a.max_pages * 4 + 15) / 16 * 16 + (fast > exact ? fast : exact);
  };
  auto smem_of = [&](int cs) {
    return (score_room(cs) > P::ATTEND ? score_room(cs) : P::ATTEND) + (a.max_pages + 31) / 32 * 4 + top_k * 4 + P::SMALL + 16;
  };
  Fits now;
  Fits& fit = dev < 64 ? fits[dev] : now;
  if (!fit.known) {   // (threads that come here at once write the same numbers)
    int room = 0, per_sm = 0, reserved = 0;
    if ((e = cudaDeviceGetAttribute(&room, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev)) != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    room -= (int)fa.sharedSizeBytes;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room)) != cudaSuccess) return e;
    for (int many = 0; many < 2; ++many) {
      cfg.dynamicSmemBytes = many ? P::ATTEND + P::SMALL + 16 : room;
      for (int k = 0; k < 4; ++k) {
        cfg.gridDim = 1 << k;
        attr.val.clusterDim.x = 1 << k;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
        fit.clusters[many][k] = n;
      }
    }
    fit.per_sm = per_sm;
    fit.beside = (int)fa.sharedSizeBytes + reserved;
    fit.known = true;
  }
  // the largest cluster that leaves all units resident at once
  int k = 3;
  while (k > 0 && units > (unsigned)fit.clusters[P::MINB * (smem_of(1 << k) + fit.beside) <= fit.per_sm][k]) --k;
  const int cs = 1 << k;
  cfg.dynamicSmemBytes = smem_of(cs);
  cfg.gridDim = units * cs;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, top_k, share_room(cs), score_room(cs), q, lens, out, sel);
}

template <int BITS, bool F32>
cudaError_t by_shape(const Args& a, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel, cudaStream_t s) {
  const int r = a.g <= 4 ? 4 : (a.d <= 128 && a.g > 8 ? 16 : 8);
#define LOWRAM_KVQ_ROWS(D)                                                  \
  if (r == 4) return go<BITS, D, 4, F32>(a, top_k, q, lens, out, sel, s);   \
  if (r == 8) return go<BITS, D, 8, F32>(a, top_k, q, lens, out, sel, s)
  if (a.d == 64) {
    LOWRAM_KVQ_ROWS(64);
    return go<BITS, 64, 16, F32>(a, top_k, q, lens, out, sel, s);
  }
  if (a.d == 128) {
    LOWRAM_KVQ_ROWS(128);
    return go<BITS, 128, 16, F32>(a, top_k, q, lens, out, sel, s);
  }
  LOWRAM_KVQ_ROWS(256);
#undef LOWRAM_KVQ_ROWS
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_sparse(const Args& a, int dtype, int top_k, const void* q, const int32_t* lens, void* out, int32_t* sel,
                          cudaStream_t s) {
  if (dtype == LOWRAM_F32)
    return a.bits == 4 ? by_shape<4, true>(a, top_k, q, lens, out, sel, s) : by_shape<8, true>(a, top_k, q, lens, out, sel, s);
  return a.bits == 4 ? by_shape<4, false>(a, top_k, q, lens, out, sel, s) : by_shape<8, false>(a, top_k, q, lens, out, sel, s);
}

}  // namespace kvq
}  // namespace lowram
