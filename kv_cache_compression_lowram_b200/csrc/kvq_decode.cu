// Quantised KV cache: attention of the last tokens over whole sequences.
//
// Bound by HBM: 2 (d bits / 8 + d / 16) bytes per cached token and KV head, read once per 4, 8 or 16
// query rows (4 layers of 4 x 32K tokens, 8 heads of 128 in 4 bits: 604 MB in 129 us from a CUDA graph, 4.7 TB/s,
// 72 % of the measured copy rate, and 134 to 140 us a Python call, depending on the machine; one layer 42 us,
// a further one 29) -- and, nearly as much, by the instructions that unpack (49 % of the issue slots).
// All steps of all units -- a unit is (sequence, layer, KV head, tile of query rows), a step 16 or 32 of
// its tokens -- form one line that is shared out evenly among the CTAs (one wave of them), so ragged
// lengths and few long sequences load the SMs alike without the host knowing a length.
// A CTA's four warps take its steps in turn, each through a ring of its own in shared memory that
// cp.async fills ahead, across unit borders; at the end of a unit's part they join their sums.
// A unit that several CTAs share is joined by the one that finishes last, in the order of the
// pieces (the result does not depend on which that is).
#include <atomic>

#include "kvq.cuh"
#include "kvq_attend.cuh"

namespace lowram {
namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWorkers = 640;
// How the steps are shared out.  Units of at most kWhole steps are never split: joining parts through
// memory costs about 4 us, four steps of a warp about as much (one sequence of 301 tokens: 15 us in
// parts of 8 steps, 8 us whole).  A part has at least kLeast steps.  A unit's queries and its
// joining cost a CTA about as much as kOver steps: on the line every unit is so much longer.
// (16 ragged sequences, some of a few tokens: 128 us with 0, 68 with 6, 58 with 10 and with 16.)
// The steps of other shapes cost more or less than those, and the same numbers suit them: 64 ragged
// sequences of 128 in 4 bits take 40.7, 39.2 and 43.3 us with kOver 6, 12 and 24, 40 of 64 in fp32 22.3, 21.7
// and 24.7; with kWhole 8, 16 and 32, 250 tokens of 256 in 8 bits 15.5, 13.3 and 13.3, 700 of 128 in 4 bits
// 10.0, 10.0 and 11.3; with kSpare 4 and 12, 16 ragged sequences of 128 in 4 bits 26.2 and 28.4, of 64 22.8 and 21.9.
// (Equal parts are tried for up to 32 sequences: a lane each.)
constexpr unsigned kWhole = 16, kLeast = 8, kSpare = 12, kOver = 12;
constexpr size_t kPartBytes = (size_t)2 * kMaxWorkers * 16 * (128 + 2) * 4;   // two parts per CTA; 8 rows of 256 + 2 are fewer

template <int BITS, int D, int ROWS, bool F32> struct Plan {
  using Tl = Tile<BITS, D, ROWS, F32>;
  static constexpr int TB = Tl::BLOCK <= 2304 ? 2 : 1;      // 16-token blocks of a step: 32 tokens up to 4.6 KB
  static constexpr int SLOT = TB * Tl::BLOCK;
  static constexpr int STAGES = SLOT > 4608 ? 2 : 3;
  static constexpr int JOIN = kWarps * Tl::ROWS * D * 4;    // the warps' sums
  static constexpr int RING = kWarps * STAGES * SLOT;
  static constexpr int SMEM = RING + JOIN + Tl::QFRAG + Tl::QMETA + (kWarps + 1) * Tl::ROWS * 8 + 16;
  // Three CTAs an SM where the shared memory allows it (d = 128 in 4 bits, four rows: 12 warps of 168
  // registers, a few of which are kept in memory over a step -- 64 bytes stored, 52 loaded a thread, 192 and
  // 172 with eight rows; two CTAs of 255 took 21 % longer, four of 128 11 %, and steps of 16 tokens 17 %).
  static constexpr int MINB = SMEM <= 74 * 1024 ? 3 : (SMEM <= 112 * 1024 ? 2 : 1);
};

struct Walk {   // a place on the line of steps
  int b, u, st, n;   // sequence, unit inside it, step inside the unit, steps of its units
};

// `total` steps cut into `parts` pieces (parts <= total), the first total % parts one longer.
struct Cut {
  unsigned each, longer;
  __device__ Cut(unsigned total, unsigned parts) : each(total / parts), longer(total % parts) {}
  __device__ __forceinline__ unsigned begin(unsigned c) const { return c * each + min(c, longer); }
  __device__ __forceinline__ int piece_of(unsigned x) const {
    const unsigned turn = longer * (each + 1);
    return x < turn ? x / (each + 1) : longer + (x - turn) / each;
  }
};

template <class P> struct Line {
  const Args& a;
  const int32_t* lens;
  int U;   // units of a sequence
  static constexpr int TOK = 16 * P::TB;
  __device__ __forceinline__ int steps(int b) const { return max(1, (len_of(a, lens, b) + TOK - 1) / TOK); }
  static __device__ __forceinline__ unsigned running_sum(unsigned x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  // Place x (below the sum of count(b) over all sequences): its sequence and the rest of x.
  template <class Count> __device__ __forceinline__ int find(unsigned& x, Count count) const {
    const int lane = threadIdx.x & 31;
    for (int b0 = 0;; b0 += 32) {
      const unsigned n = b0 + lane < a.B ? count(b0 + lane) : 0, inc = running_sum(n);
      const unsigned past = __ballot_sync(kFull, inc > x);
      if (past) {
        const int w = __ffs(past) - 1;
        x -= __shfl_sync(kFull, inc - n, w);
        return b0 + w;
      }
      x -= __shfl_sync(kFull, inc, 31);
    }
  }
  __device__ __forceinline__ void next_unit(Walk& w) const {
    w.st = 0;
    if (++w.u == U) {
      w.u = 0;
      if (++w.b < a.B) w.n = steps(w.b);
    }
  }
  __device__ __forceinline__ void forward(Walk& w, int k) const {
    w.st += k;
    while (w.b < a.B && w.st >= w.n) {
      const int rest = w.st - w.n;
      next_unit(w);
      w.st = rest;
    }
  }
};

// The parts of a unit (CTAs c_first .. c_last), joined in their order.  A warp per row finds the
// weights of a chunk of parts, then each thread sums four channels over them with its loads in
// flight together.  wt: [kChunk][ROWS] floats; f: the rows' f''; norm: [ROWS] maxima, then [ROWS] sums.
template <class P, class Store>
__device__ __forceinline__ void join_parts(const float* part, int c_first, int c_last, int rows, float* wt, const float* f, float* norm, Store store) {
  constexpr int ROWS = P::Tl::ROWS, D = P::Tl::D, REC = ROWS * (D + 2), kChunk = P::JOIN / 4 / ROWS, FLY = 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = c_last - c_first + 1;
  auto at = [&](int i) { return part + (size_t)(2 * (c_first + i) + (i == 0 ? 1 : 0)) * REC; };
  constexpr int QUADS = ROWS * D / 4, MINE = (QUADS + kThreads - 1) / kThreads;
  float4 v[MINE];
#pragma unroll
  for (int k = 0; k < MINE; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kChunk) {
    const int nc = min(kChunk, n - i0);
    if (i0) __syncthreads();
    for (int j = warp; j < rows; j += kWarps) {
      // up to 64 parts at once, in registers
      float m = -INFINITY, l = 0.f, mp[2], lp[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool in = lane + 32 * k < nc;
        const float* p = at(i0 + (in ? lane + 32 * k : 0)) + ROWS * D + j;
        mp[k] = in ? __ldcg(p) : -INFINITY;
        lp[k] = __ldcg(p + ROWS);
      }
      if (i0 == 0) {
        m = fmaxf(mp[0], mp[1]);
        for (int i = lane + 64; i < n; i += 32) m = fmaxf(m, __ldcg(at(i) + ROWS * D + j));
        m = warp_max(m);
        if (lane == 0) norm[j] = m;
      } else {
        m = norm[j];
      }
      for (int i = lane, k = 0; i < nc; i += 32, ++k) {
        const float* p = at(i0 + i) + ROWS * D + j;
        const float mi = k == 0 ? mp[0] : (k == 1 ? mp[1] : __ldcg(p)), li = k == 0 ? lp[0] : (k == 1 ? lp[1] : __ldcg(p + ROWS));
        const float w = P::Tl::factor(mi, m, f[j]);
        wt[i * ROWS + j] = w;
        l = fmaf(w, li, l);
      }
      l = warp_sum(l);
      if (lane == 0) norm[ROWS + j] = i0 ? norm[ROWS + j] + l : l;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int e = tid + k * kThreads, j = e / (D / 4);
      if (j >= rows) continue;
      for (int i = 0; i < nc; i += FLY) {
        float4 x[FLY];
#pragma unroll
        for (int f = 0; f < FLY; ++f) x[f] = __ldcg(reinterpret_cast<const float4*>(at(i0 + min(i + f, nc - 1))) + e);
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const float w = i + f < nc ? wt[(i + f) * ROWS + j] : 0.f;
          v[k].x = fmaf(w, x[f].x, v[k].x);
          v[k].y = fmaf(w, x[f].y, v[k].y);
          v[k].z = fmaf(w, x[f].z, v[k].z);
          v[k].w = fmaf(w, x[f].w, v[k].w);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int e = tid + k * kThreads, j = e / (D / 4);
    if (j < rows) store(j, e % (D / 4) * 4, v[k], norm[j], norm[ROWS + j]);
  }
}

template <int BITS, int D, int ROWS, bool F32>
__global__ void __launch_bounds__(kThreads, Plan<BITS, D, ROWS, F32>::MINB)
decode_kernel(Args a, int row_tiles, const void* qv, const int32_t* __restrict__ lens, void* outv,
              unsigned* __restrict__ arrived, float* __restrict__ part) {
  using P = Plan<BITS, D, ROWS, F32>;
  using Tl = typename P::Tl;
  using T = typename Tl::T;
  constexpr int TB = P::TB;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* frag = sm + P::RING;
  float* join = reinterpret_cast<float*>(frag + Tl::QFRAG);
  float* meta = join + P::JOIN / 4;
  float* tops = meta + Tl::QMETA / 4;          // [warp][row] running maxima, then the sums of the weights
  float* norm = tops + 2 * kWarps * ROWS;      // [ROWS] maxima, [ROWS] sums of the CTA
  int* shared_int = reinterpret_cast<int*>(norm + 2 * ROWS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* q = static_cast<const T*>(qv);
  T* out = static_cast<T*>(outv);
  const int rows_all = a.n * a.g;
  const Line<P> line{a, lens, a.n_layers * a.Hkv * row_tiles};
  const int me = blockIdx.x;
  // This CTA's share: `left` steps from `cur` on.  A part of a unit belongs to the CTAs c_first ..
  // c_last; where a share is cut anywhere on the line these follow from `cut`.
  unsigned total = 0, longest = 0, left = 0, base = 0;   // base: the current unit's place on the line
  for (int b = lane; b < a.B; b += 32) {
    const unsigned n = line.steps(b);
    total += n;
    longest = max(longest, n);
  }
  total = (__reduce_add_sync(kFull, total) + a.B * kOver) * line.U;
  longest = __reduce_max_sync(kFull, longest);
  Walk cur;
  int c_first = -1, c_last = 0;
  Cut cut(1, 1);
  if (longest <= kWhole) {                      // whole units
    const unsigned units = a.B * line.U, workers = min(units, gridDim.x);
    if (me >= workers) return;
    const Cut c(units, workers);
    const unsigned u0 = c.begin(me);
    unsigned n = c.begin(me + 1) - u0;
    cur.b = u0 / line.U;
    cur.u = u0 - cur.b * line.U;
    cur.st = 0;
    cur.n = line.steps(cur.b);
    unsigned in_b = min(n, line.U - cur.u);
    left = in_b * cur.n;
    for (int b = cur.b + 1; n -= in_b; ++b) {
      in_b = min(n, (unsigned)line.U);
      left += in_b * line.steps(b);
    }
  } else {
    // Each unit cut into equal parts of about `piece` steps, one part per CTA, if that takes no more
    // than kSpare steps more than an even share; else the line cut evenly, across units.
    const unsigned even = max(kLeast, (total - a.B * line.U * kOver + gridDim.x - 1) / gridDim.x);
    unsigned piece = even, parts = ~0u;
    auto parts_of = [&](int b) { return ((unsigned)line.steps(b) + piece - 1) / piece; };
    if (a.B <= 32)
      for (; piece <= even + kSpare; piece += 1 + piece / 8) {
        parts = __reduce_add_sync(kFull, lane < a.B ? parts_of(lane) : 0) * line.U;
        if (parts <= gridDim.x) break;
      }
    if (parts <= gridDim.x) {
      if (me >= parts) return;
      unsigned x = me;
      cur.b = line.find(x, [&](int b) { return parts_of(b) * line.U; });
      cur.n = line.steps(cur.b);
      const unsigned k = ((unsigned)cur.n + piece - 1) / piece;
      cur.u = x / k;
      const unsigned i = x - cur.u * k;
      const Cut c(cur.n, k);
      cur.st = c.begin(i);
      left = c.begin(i + 1) - cur.st;
      c_first = me - i;
      c_last = c_first + k - 1;
    } else {
      const unsigned workers = min(gridDim.x, (total + kLeast - 1) / kLeast);
      if (me >= workers) return;
      cut = Cut(total, workers);
      auto place = [&](unsigned x) {
        Walk w;
        w.b = line.find(x, [&](int b) { return (line.steps(b) + kOver) * line.U; });
        w.n = line.steps(w.b);
        w.u = x / (w.n + kOver);
        w.st = x - w.u * (w.n + kOver);
        return w;
      };
      const unsigned s0 = cut.begin(me);
      cur = place(s0);
      base = s0 - cur.st;
      if (cur.st >= cur.n) {                    // in the room behind a unit's steps
        base += cur.n + kOver;
        line.next_unit(cur);
      }
      const Walk last = place(cut.begin(me + 1) - 1);
      const int to = min(last.st + 1, last.n);
      int mine = 0;
      if (cur.b == last.b) {
        mine = (last.u - cur.u) * cur.n + to - cur.st;
      } else if (cur.b < last.b) {
        mine = (line.U - cur.u) * cur.n - cur.st + last.u * last.n + to;
        for (int b = cur.b + 1; b < last.b; ++b) mine += line.U * line.steps(b);
      }
      if (mine <= 0) return;
      left = mine;
    }
  }
  if (me == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (len_bad(a, lens, b)) flag(a, KVQ_ERR_RANGE);
  Walk ahead = cur;
  line.forward(ahead, warp);
  unsigned xa = warp;                           // the next step to load
  uint8_t* ring = sm + warp * P::STAGES * P::SLOT;
  const uint32_t ring_u = smem_u32(ring);
  unsigned bad = 0;                             // TB bits per step under way: blocks that are not there
  int in = 0, rd = 0;
  // lookup() asks the table for the pages of the next step, issue() starts the copies of the step
  // looked up before and looks up the one after it.  Rows of the pool are counted in 32 bits (the
  // host checks; 2^32 rows of 64 channels in 4 bits, K and V, would be 309 GB).
  int seen_b = -1, seen_u = -1, len_a = 0, tok_a = -1, pid_a[TB];
  uint32_t unit_row = 0, row_a = 0;             // rows in front of (layer, page 0, head)
  auto lookup = [&]() {
    tok_a = -1;
    if (xa >= left) return;
    if (ahead.b != seen_b || ahead.u != seen_u) {   // another unit
      seen_b = ahead.b;
      seen_u = ahead.u;
      const int lh = ahead.u / row_tiles, layer = lh / a.Hkv;
      len_a = len_of(a, lens, ahead.b);
      unit_row = (uint32_t)row0_of(a, a.layer0 + layer, 0, lh - layer * a.Hkv);
    }
    row_a = unit_row;
    tok_a = ahead.st * Line<P>::TOK;
#pragma unroll
    for (int i = 0; i < TB; ++i) pid_a[i] = -2;
    if (tok_a < len_a) pid_a[0] = page_of(a, ahead.b, tok_a >> a.page_log2);
    if (TB == 2 && a.page == 16 && tok_a + 16 < len_a) pid_a[TB - 1] = page_of(a, ahead.b, (tok_a >> 4) + 1);
    xa += kWarps;
    if (ahead.st + kWarps < ahead.n) ahead.st += kWarps;
    else line.forward(ahead, kWarps);
  };
  // `place`: how many steps are under way
  auto issue = [&](int place) {
    const int tok = tok_a;
    if (tok >= 0) {
      int pid[TB];
#pragma unroll
      for (int i = 0; i < TB; ++i) pid[i] = pid_a[i];
      const uint32_t row = row_a + (tok & (a.page - 1)), dst = ring_u + in * P::SLOT;
      lookup();
      if (a.page >= 16 * TB) {                  // one run (its second block may lie behind the last token)
        if (pid[0] >= 0) Tl::template load<TB, TB>(a, dst, 0, row + ((uint32_t)(pid[0] * a.Hkv) << a.page_log2));
        else bad |= ((1u << TB) - 1) << (place * TB);
      } else {
#pragma unroll
        for (int i = 0; i < TB; ++i) {
          if (pid[i] >= 0) Tl::template load<TB, 1>(a, dst, i, row + ((uint32_t)(pid[i] * a.Hkv) << a.page_log2));
          else bad |= 1u << (place * TB + i);
        }
      }
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < TB; ++i)
          if (pid[i] == -1) flag(a, KVQ_ERR_PAGE);
      }
      in = in + 1 == P::STAGES ? 0 : in + 1;
    }
    cp_commit();
  };
  lookup();

  Tl tile;
  bool first = true;
  for (unsigned x = 0; x < left;) {             // a unit's part at a time
    const unsigned part_n = min(left - x, (unsigned)(cur.n - cur.st));
    const int rt = cur.u % row_tiles, lh = cur.u / row_tiles, layer = lh / a.Hkv, h = lh - layer * a.Hkv;
    const int row_base = rt * ROWS, rows = min(ROWS, rows_all - row_base), len = len_of(a, lens, cur.b);
    // row j of the tile: query token (row_base + j) / g, head (row_base + j) % g of the KV head
    const size_t qbase = ((size_t)layer * a.B + cur.b) * a.n;
    auto row_at = [&](int j) {
      const int i = (row_base + j) / a.g, jj = (row_base + j) % a.g;
      return ((qbase + i) * a.Hq + (size_t)h * a.g + jj) * D;
    };
    {
      typename Tl::template Queries<kWarps> qr;
      qr.fetch(rows, warp, [&](int j) { return q + row_at(j); });
      if (first) {
#pragma unroll 1
        for (int i = 0; i < P::STAGES - 1; ++i) issue(i);
        first = false;
      }
      qr.prepare(frag, meta, warp);
    }
    __syncthreads();
    tile.begin(frag, meta);
    int lim[Tl::NT][Tl::CP];
#pragma unroll
    for (int t = 0; t < Tl::NT; ++t)
#pragma unroll
      for (int c = 0; c < Tl::CP; ++c) lim[t][c] = len - a.n + 1 + (row_base + min(Tl::row_of(t, c), rows - 1)) / a.g;
    const int least = len - a.n + 1 + row_base / a.g;
    // this warp's steps of the part: those that are `warp` modulo kWarps in the share
    int st = cur.st + (warp - x % kWarps + kWarps) % kWarps;
    const int st1 = cur.st + part_n;
    for (; st < st1; st += kWarps) {
      cp_wait<P::STAGES - 2>();
      __syncwarp();
      const unsigned gone = bad & ((1u << TB) - 1);
      bad >>= TB;
      const uint8_t* slot = ring + rd * P::SLOT;
      const int tok = st * Line<P>::TOK;
      if (gone == 0 && tok + Line<P>::TOK <= least) {
        tile.template step<TB, TB, false>(slot, 0, frag, tok, lim);
      } else {
#pragma unroll 1
        for (int i = 0; i < TB; ++i)            // nothing to see in a block that is not there
          if (!(gone >> i & 1) && tok + 16 * i < len) tile.template step<TB, 1, true>(slot, i, frag, tok + 16 * i, lim);
      }
      rd = rd + 1 == P::STAGES ? 0 : rd + 1;
      __syncwarp();
      issue(P::STAGES - 2);
    }
    // join the warps: common maximum, scaled sums, channels added in the warps' order
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
    const bool whole = cur.st == 0 && part_n == cur.n;
    constexpr int REC = ROWS * (D + 2);         // floats of a part: [ROWS][D], maxima, sums of the weights
    float* rec = part + (size_t)(2 * me + (cur.st == 0 ? 1 : 0)) * REC;
    auto finish = [&](int j, int c, float4 v, float m, float l) {
      T* o = out + row_at(j) + c;
      const float inv = 1.f / l;
      v = m == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if constexpr (F32) {
        *reinterpret_cast<float4*>(o) = v;
      } else {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(h);
      }
    };
    for (int e = tid; e < rows * D / 4; e += kThreads) {
      const int j = e / (D / 4), c = e % (D / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(join + (w * ROWS + j) * D + c);
        v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
      }
      if (whole) finish(j, c, v, norm[j], norm[ROWS + j]);
      else *reinterpret_cast<float4*>(rec + 4 * e) = v;
    }
    if (!whole) {
      if (tid < 2 * ROWS) rec[ROWS * D + tid] = norm[tid];
      // the last CTA of the unit to come joins all parts, in their order
      int c0 = c_first, c1 = c_last;
      if (c0 < 0) {
        c0 = cut.piece_of(base);
        c1 = cut.piece_of(base + cur.n - 1);
      }
      __syncthreads();
      if (tid == 0) {
        unsigned* cnt = arrived + (size_t)cur.b * line.U + cur.u;
        __threadfence();                        // the CTA's writes (seen through the barrier) before the count
        const int last = atomicAdd(cnt, 1u) == (unsigned)(c1 - c0);
        if (last) *cnt = 0;                     // ready for the next call
        __threadfence();
        *shared_int = last;
      }
      __syncthreads();
      if (*shared_int) join_parts<P>(part, c0, c1, rows, join, meta, norm, finish);
    }
    __syncthreads();                            // the queries' operands and the sums may be written anew
    x += part_n;
    cur.st += part_n;
    if (cur.st >= cur.n) {
      base += cur.n + kOver;
      line.next_unit(cur);
    }
  }
  cp_wait<0>();
}

// Query rows of a tile: the fewest of 4, 8 and 16 that hold all, 16 only where the sums fit the
// registers (d <= 128).
int rows_tile(const Args& a) {
  const int rows = a.n * a.g;
  return rows <= 4 ? 4 : (a.d <= 128 && rows > 8 ? 16 : 8);
}

template <int BITS, int D, int ROWS, bool F32>
cudaError_t go(const Args& a, const void* q, const int32_t* lens, void* out, void* ws, cudaStream_t s) {
  using P = Plan<BITS, D, ROWS, F32>;
  // per device: the kernel's attribute and the CTAs that are resident at once
  static std::atomic<int> workers[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int w = dev < 64 ? workers[dev].load() : 0;
  if (!w) {
    int sm = 0, per = 0;
    if ((e = cudaFuncSetAttribute(decode_kernel<BITS, D, ROWS, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, decode_kernel<BITS, D, ROWS, F32>, kThreads, P::SMEM)) != cudaSuccess) return e;
    w = sm * (per < 1 ? 1 : per);
    if (w > kMaxWorkers) w = kMaxWorkers;
    if (dev < 64) workers[dev] = w;
  }
  static_assert((size_t)2 * kMaxWorkers * ROWS * (D + 2) * 4 <= kPartBytes, "parts");
  // the parts first: the counters of every kind of call start at one place and stay zero between calls
  float* part = static_cast<float*>(ws);
  unsigned* arrived = reinterpret_cast<unsigned*>(static_cast<char*>(ws) + kPartBytes);
  const int tiles = (a.n * a.g + ROWS - 1) / ROWS;
  decode_kernel<BITS, D, ROWS, F32><<<w, kThreads, P::SMEM, s>>>(a, tiles, q, lens, out, arrived, part);
  return cudaGetLastError();
}

template <int BITS, bool F32>
cudaError_t by_shape(const Args& a, const void* q, const int32_t* lens, void* out, void* ws, cudaStream_t s) {
  const int r = rows_tile(a);
#define LOWRAM_KVQ_ROWS(D)                                         \
  if (r == 4) return go<BITS, D, 4, F32>(a, q, lens, out, ws, s);  \
  if (r == 8) return go<BITS, D, 8, F32>(a, q, lens, out, ws, s)
  if (a.d == 64) {
    LOWRAM_KVQ_ROWS(64);
    return go<BITS, 64, 16, F32>(a, q, lens, out, ws, s);
  }
  if (a.d == 128) {
    LOWRAM_KVQ_ROWS(128);
    return go<BITS, 128, 16, F32>(a, q, lens, out, ws, s);
  }
  LOWRAM_KVQ_ROWS(256);
#undef LOWRAM_KVQ_ROWS
  return cudaErrorInvalidValue;
}

}  // namespace

// The line of steps (of at least 16 tokens) is counted in 32 bits.
bool decode_line_fits(const Args& a) {
  const int rt = rows_tile(a), tiles = (a.n * a.g + rt - 1) / rt;
  return (double)a.n_layers * a.B * a.Hkv * tiles * ((double)a.max_pages * a.page / 16 + 1 + kOver) < 2147483648.0;
}

size_t decode_workspace_bytes(const Args& a) {
  const int rt = rows_tile(a), tiles = (a.n * a.g + rt - 1) / rt;
  return kPartBytes + (size_t)a.B * a.n_layers * a.Hkv * tiles * 4;
}

cudaError_t launch_decode(const Args& a, int dtype, const void* q, const int32_t* lens, void* out, void* ws, cudaStream_t s) {
  if (dtype == LOWRAM_F32)
    return a.bits == 4 ? by_shape<4, true>(a, q, lens, out, ws, s) : by_shape<8, true>(a, q, lens, out, ws, s);
  return a.bits == 4 ? by_shape<4, false>(a, q, lens, out, ws, s) : by_shape<8, false>(a, q, lens, out, ws, s);
}

}  // namespace kvq
}  // namespace lowram
