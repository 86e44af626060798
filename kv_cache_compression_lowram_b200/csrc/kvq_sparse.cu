// Quantised KV cache: attention over the pages that their mean keys select for each query.
//
// One launch.  A unit -- (layer, sequence, query token, KV head) -- belongs to a cluster of 1 to 16
// CTAs, which do all of it together through each other's shared memory:
//   1. each CTA scores its share of the full pages (mean key . sum of the group's queries, in 64
//      bits) into its shared memory: 2 d bytes a page, the larger part of what a long context costs;
//   2. every CTA gathers all scores and finds the same top_k - 1 best pages: one histogram over the
//      range of the scores leaves a bin that holds the border, whose few members are ranked by
//      comparison (a bin too large for that is cut again by the bits of its scores);
//   3. the selected pages' 16-token blocks go round the warps of the cluster, as in the attention
//      over whole sequences; CTAs join their sums and the cluster joins the CTAs'.
// No workspace, no second launch, and nothing is written but the outputs.
#include <cooperative_groups.h>

#include "kvq.cuh"
#include "kvq_attend.cuh"

namespace cg = cooperative_groups;

namespace lowram {
namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBins = 1024;
constexpr int kRank = 256;    // members of a border bin that are ranked by comparison

template <int BITS, int D, int ROWS, bool F32> struct Plan {
  using Tl = Tile<BITS, D, ROWS, F32>;
  static constexpr int TB = Tl::BLOCK <= 2304 ? 2 : 1;
  static constexpr int SLOT = TB * Tl::BLOCK;
  static constexpr int STAGES = SLOT > 4608 ? 2 : 3;
  static constexpr int RING = kWarps * STAGES * SLOT;
  static constexpr int JOIN = kWarps * ROWS * D * 4;
  // what lives at once: the ring and the joined sums, or the scores and the histogram
  static constexpr int ATTEND = RING + JOIN + Tl::QFRAG;
  static constexpr int SMALL = Tl::QMETA + kWarps * ROWS * 8 + 2 * ROWS * 4;
  static constexpr int MINB = ATTEND <= 72 * 1024 ? 3 : (ATTEND <= 108 * 1024 ? 2 : 1);
};

// Scores as integers of the same order; NaN as -infinity.
__device__ __forceinline__ unsigned long long key_of(double s) {
  if (!(s == s)) s = -INFINITY;
  s += 0.0;   // -0 as 0
  const long long b = __double_as_longlong(s);
  return (unsigned long long)b ^ (b < 0 ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double score_of(unsigned long long k) {
  return __longlong_as_double((long long)(k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k));
}

__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(kFull, v, o);
    v = y > v ? y : v;
  }
  return v;
}

struct Select {   // shared by the CTA while it selects
  unsigned hist[kBins];
  unsigned long long wide[2][kWarps];
  unsigned sums[kWarps];
  int border, above, members, list[kRank];
};

// Marks (bits of `mark`, zeroed here) the `want` largest of keys[0, n), 0 < want < n; equal ones from the
// lowest index on.  All threads of the CTA.
__device__ void select_largest(const unsigned long long* keys, int n, int want, unsigned* mark, Select& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < (n + 31) / 32; i += kThreads) mark[i] = 0;
  unsigned long long lo = 0, hi = ~0ull;   // the keys still in question
  bool linear = true;
  for (;;) {
    // their range
    unsigned long long mx = 0, mn = 0;     // the largest key, and the largest complement
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = keys[i];
      if (k >= lo && k <= hi) {
        mx = k > mx ? k : mx;
        mn = ~k > mn ? ~k : mn;
      }
    }
    mx = warp_max_u64(mx);
    mn = warp_max_u64(mn);
    if (lane == 0) {
      s.wide[0][warp] = mx;
      s.wide[1][warp] = mn;
    }
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      mx = s.wide[0][w] > mx ? s.wide[0][w] : mx;
      mn = s.wide[1][w] > mn ? s.wide[1][w] : mn;
    }
    mn = ~mn;
    // bins: even in the scores at first (in the keys where a score is infinite), then even in the keys
    const double smin = score_of(mn), span = score_of(mx) - smin, scale = (kBins - 1) / span;
    linear = linear && span > 0.0 && span < 1e300 && scale < 1e300;
    const int shift = mx == mn ? 0 : max(0, 64 - __clzll((long long)(mx - mn)) - 10);
    auto bin_of = [&](unsigned long long k) { return linear ? (int)((score_of(k) - smin) * scale) : (int)((k - mn) >> shift); };
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&s.hist[bin_of(k)], 1u);
    }
    __syncthreads();
    // the bin of the want-th largest: thread t sums bins from the top, kBins / kThreads each
    constexpr int PER = kBins / kThreads;
    unsigned sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += s.hist[kBins - 1 - tid * PER - i];
    unsigned inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s.sums[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += s.sums[w];
    unsigned before = inc - sum;
    if (before < (unsigned)want && inc >= (unsigned)want) {   // one thread
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = kBins - 1 - tid * PER - i;
        const unsigned h = s.hist[b];
        if (before < (unsigned)want && before + h >= (unsigned)want) {
          s.border = b;
          s.above = before;
          s.members = h;
        }
        before += h;
      }
    }
    __syncthreads();
    const int border = s.border, members = s.members;
    want -= s.above;
    const bool rank = members <= kRank, equal = mx == mn;
    __syncthreads();
    if (tid == 0) s.members = 0;
    __syncthreads();
    unsigned long long nlo = ~0ull, nhi = 0;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = keys[i];
      if (!(k >= lo && k <= hi)) continue;
      const int b = bin_of(k);
      if (b > border) atomicOr(&mark[i >> 5], 1u << (i & 31));
      else if (b == border) {
        if (rank) s.list[atomicAdd(&s.members, 1)] = i;
        nlo = k < nlo ? k : nlo;
        nhi = k > nhi ? k : nhi;
      }
    }
    if (rank) {
      __syncthreads();
      for (int j = tid; j < members; j += kThreads) {
        const int i = s.list[j];
        const unsigned long long k = keys[i];
        int r = 0;
        for (int t = 0; t < members; ++t) {
          const int o = s.list[t];
          const unsigned long long ko = keys[o];
          r += ko > k || (ko == k && o < i);
        }
        if (r < want) atomicOr(&mark[i >> 5], 1u << (i & 31));
      }
      __syncthreads();
      return;
    }
    if (equal) {                                // a run of equal keys: the first `want` of them
      __syncthreads();
      if (warp == 0) {
        int left = want;
        for (int i = 0; i < n && left > 0; i += 32) {
          const bool is = i + lane < n && keys[i + lane] == mx;
          const unsigned m = __ballot_sync(kFull, is);
          if (is && __popc(m & ((1u << lane) - 1)) < left) atomicOr(&mark[(i + lane) >> 5], 1u << lane);
          left -= __popc(m);
        }
      }
      __syncthreads();
      return;
    }
    // the border bin alone, by its keys
    nhi = warp_max_u64(nhi);
    nlo = warp_max_u64(~nlo);
    if (lane == 0) {
      s.wide[0][warp] = nhi;
      s.wide[1][warp] = nlo;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      nhi = s.wide[0][w] > nhi ? s.wide[0][w] : nhi;
      nlo = s.wide[1][w] > nlo ? s.wide[1][w] : nlo;
    }
    lo = ~nlo;
    hi = nhi;
    linear = false;
    __syncthreads();
  }
}

template <int BITS, int D, int ROWS, bool F32>
__global__ void __launch_bounds__(kThreads, Plan<BITS, D, ROWS, F32>::MINB)
sparse_kernel(Args a, int top_k, int key_room, const void* __restrict__ qv, const int32_t* __restrict__ lens, void* __restrict__ outv,
              int32_t* __restrict__ sel) {
  using P = Plan<BITS, D, ROWS, F32>;
  using Tl = typename P::Tl;
  using T = typename Tl::T;
  constexpr int TB = P::TB;
  extern __shared__ __align__(128) uint8_t sm[];
  // attending: ring, joined sums, the queries' operands; selecting: all keys, marks
  uint8_t* frag = sm + P::RING + P::JOIN;
  float* join = reinterpret_cast<float*>(sm + P::RING);
  // (a CTA alone has one array for both: key_room = 0)
  unsigned long long* mine = reinterpret_cast<unsigned long long*>(sm);             // this CTA's scores: [key_room]
  unsigned long long* keys = mine + key_room;                                       // everyone's
  const int body = max(P::ATTEND, key_room * 8 + a.max_pages * 8);
  unsigned* mark = reinterpret_cast<unsigned*>(sm + body);                          // [max_pages / 32]
  int* list = reinterpret_cast<int*>(mark + (a.max_pages + 31) / 32);               // [top_k] pages, ascending
  float* meta = reinterpret_cast<float*>(list + top_k);
  float* tops = meta + Tl::QMETA / 4;
  float* norm = tops + 2 * kWarps * ROWS;                                           // [ROWS] maxima, [ROWS] sums
  __shared__ Select s;
  __shared__ int count;
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
    constexpr int LPP = D / 8, PPW = 32 / LPP, FLY = 8;
    const int c8 = lane % LPP;
    if (top_k > 1) {
      double qs[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) qs[k] = 0.0;
      for (int j = 0; j < a.g; ++j) {
        const T* src = q + (size_t)j * D + c8 * 8;
        __align__(16) T x[8];
#pragma unroll
        for (int k = 0; k < (int)sizeof(x) / 16; ++k) reinterpret_cast<uint4*>(x)[k] = __ldg(reinterpret_cast<const uint4*>(src) + k);
#pragma unroll
        for (int k = 0; k < 8; ++k) qs[k] += (double)to_f<T>(x[k]);
      }
      const uint32_t row = (uint32_t)(row0_of(a, a.layer0 + layer, 0, h) >> a.page_log2);
      for (int base = c0 + warp * PPW * FLY; base < c1; base += kWarps * PPW * FLY) {
        int pid = -1;
        if (lane < PPW * FLY && base + lane < c1) {
          pid = page_of(a, b, base + lane);
          if (pid < 0) flag(a, KVQ_ERR_PAGE);
        }
        uint4 w[FLY];
        bool there[FLY];
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int p = __shfl_sync(kFull, pid, f * PPW + lane / LPP);
          there[f] = p >= 0;
          w[f] = make_uint4(0, 0, 0, 0);
          if (p >= 0) w[f] = __ldg(reinterpret_cast<const uint4*>(a.k_mean + (size_t)(row + (uint32_t)p * a.Hkv) * D) + c8);
        }
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const uint32_t v[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
          double x = 0.0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x = fma(qs[2 * k], (double)__uint_as_float(v[k] << 16), x);
            x = fma(qs[2 * k + 1], (double)__uint_as_float(v[k] & 0xffff0000u), x);
          }
#pragma unroll
          for (int o = LPP / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
          const int c = base + f * PPW + lane / LPP;
          if (c8 == 0 && c < c1) mine[c - c0] = key_of(there[f] ? x : -INFINITY);
        }
      }
      // 2. everyone's scores, and the best of them
      if (CS > 1) {
        cluster.sync();
        for (int r = 0; r < CS; ++r) {
          const unsigned long long* from = cluster.map_shared_rank(mine, r);
          const int f0 = min(r * share, last), f1 = min(f0 + share, last);
          for (int c = f0 + tid; c < f1; c += kThreads) keys[c] = from[c - f0];
        }
        cluster.sync();                    // `mine` may be overwritten from here on
      } else {
        __syncthreads();
      }
      select_largest(keys, last, top_k - 1, mark, s);
    } else {
      for (int k = tid; k < (last + 31) / 32; k += kThreads) mark[k] = 0;
      __syncthreads();
    }
    // the selected pages in ascending order, the newest behind them
    const int words = (last + 31) / 32;
    int before = 0;
    for (int w0 = 0; w0 < words; w0 += kThreads) {
      const unsigned m = w0 + tid < words ? mark[w0 + tid] : 0;
      unsigned inc = __popc(m);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) s.sums[warp] = inc;
      __syncthreads();
      int at = before + inc - __popc(m);
      for (int w = 0; w < warp; ++w) at += s.sums[w];
      for (unsigned left = m; left; left &= left - 1) list[at++] = (w0 + tid) * 32 + __ffs(left) - 1;
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
      const float top = tops[warp * ROWS + j];
      return top == -INFINITY ? 0.f : ex2(top - most(j));
    });
    if (tid < ROWS) {
      const float m = most(tid);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = tops[w * ROWS + tid];
        if (mw != -INFINITY) l = fmaf(tops[(kWarps + w) * ROWS + tid], ex2(mw - m), l);
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
    for (int e = rank * kThreads + tid; e < rows * D / 4; e += CS * kThreads) {
      const int j = e / (D / 4);
      float m = -INFINITY, l = 0.f;
      for (int r = 0; r < CS; ++r) m = fmaxf(m, cluster.map_shared_rank(norm, r)[j]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < CS; ++r) {
        const float* nr = cluster.map_shared_rank(norm, r);
        const float mr = nr[j];
        if (mr == -INFINITY) continue;
        const float w = ex2(mr - m);
        l = fmaf(nr[ROWS + j], w, l);
        const float4 y = reinterpret_cast<const float4*>(cluster.map_shared_rank(join, r))[e];
        v = make_float4(fmaf(y.x, w, v.x), fmaf(y.y, w, v.y), fmaf(y.z, w, v.z), fmaf(y.w, w, v.w));
      }
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
  static int cap[64] = {0};   // per device: the largest cluster, once the attributes are set
  auto kernel = sparse_kernel<BITS, D, ROWS, F32>;
  const unsigned units = (unsigned)a.n_layers * a.B * a.n * a.Hkv;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = dev < 64 ? cap[dev] : 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  cfg.blockDim = kThreads;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto key_room = [&](int cs) { return cs > 1 ? (a.max_pages + cs - 1) / cs : 0; };
  auto smem_of = [&](int cs) {
    const int scores = (key_room(cs) + a.max_pages) * 8;
    return (scores > P::ATTEND ? scores : P::ATTEND) + (a.max_pages + 31) / 32 * 4 + top_k * 4 + P::SMALL + 16;
  };
  if (!most) {
    int room = 0;
    if ((e = cudaDeviceGetAttribute(&room, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
    room -= (int)sizeof(Select) + 1024;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    cfg.gridDim = 16;
    cfg.dynamicSmemBytes = room;
    attr.val.clusterDim.x = 16;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    int fit = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg)) != cudaSuccess) return e;
    most = fit > 0 ? 16 : 8;
    if (dev < 64) cap[dev] = most;
  }
  // as many CTAs of a unit as leave all units resident at once
  int cs = most;
  while (cs > 1 && units * cs > 296) cs >>= 1;
  cfg.dynamicSmemBytes = smem_of(cs);
  cfg.gridDim = units * cs;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, top_k, key_room(cs), q, lens, out, sel);
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
