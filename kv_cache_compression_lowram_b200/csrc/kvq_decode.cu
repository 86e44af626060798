// Quantised KV cache: attention of the last tokens over whole sequences.
//
// Bound by HBM: 2 (d bits / 8 + d / 16) bytes per cached token and KV head, read once per 8 or 16
// query rows.  All steps of all units -- a unit is (sequence, layer, KV head, tile of query rows), a
// step 16 or 32 of its tokens -- form one line that is cut into equal pieces, one per CTA, so
// ragged lengths and few long sequences load the SMs evenly without the host knowing a length.
// A CTA's four warps take its steps in turn, each through a ring of its own in shared memory that
// cp.async fills ahead, across unit borders; at the end of a unit's part they join their sums.
// A unit that several CTAs share is joined by the one that finishes last, in the order of the
// pieces (the result does not depend on which that is).
#include "kvq.cuh"
#include "kvq_attend.cuh"

namespace lowram {
namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWorkers = 640;
#ifndef KVQ_LEAST
#define KVQ_LEAST 8
#endif
constexpr unsigned kLeast = KVQ_LEAST;
constexpr size_t kPartBytes = (size_t)2 * kMaxWorkers * 16 * (128 + 2) * 4;   // two parts per CTA; 8 rows of 256 + 2 are fewer

template <int BITS, int D, int ROWS, bool F32> struct Plan {
  using Tl = Tile<BITS, D, ROWS, F32>;
  #ifdef KVQ_TB
  static constexpr int TB = KVQ_TB;
#else
  static constexpr int TB = Tl::BLOCK <= 2304 ? 2 : 1;
#endif      // 16-token blocks of a step
  static constexpr int SLOT = TB * Tl::BLOCK;
  #ifdef KVQ_STAGES
  static constexpr int STAGES = KVQ_STAGES;
#else
  static constexpr int STAGES = SLOT > 4608 ? 2 : 3;
#endif
  static constexpr int JOIN = kWarps * Tl::ROWS * D * 4;    // the warps' sums
  static constexpr int RING = kWarps * STAGES * SLOT;
  static constexpr int SMEM = RING + JOIN + Tl::QFRAG + Tl::QMETA + kWarps * Tl::ROWS * 8 + 16;
  #ifdef KVQ_MINB
  static constexpr int MINB = KVQ_MINB;
#else
  static constexpr int MINB = SMEM <= 74 * 1024 ? 3 : (SMEM <= 112 * 1024 ? 2 : 1);
#endif
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
  // The steps of all units (the same on every lane; below 2^31, the host checks).  Where there are at
  // most 32 sequences, `scan` is what at() needs: a lane's steps and their running sum.
  __device__ __forceinline__ unsigned total(uint2& scan) const {
    const int lane = threadIdx.x & 31;
    unsigned t = 0;
    for (int b = lane; b < a.B; b += 32) t += steps(b) * U;
    unsigned inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    scan = make_uint2(t, inc);
    return __shfl_sync(kFull, inc, 31);
  }
  __device__ __forceinline__ Walk at(unsigned x, uint2 scan) const {   // 0 <= x < total
    const int lane = threadIdx.x & 31;
    unsigned before = 0, n = scan.x, inc = scan.y;
    for (int b0 = 0;; b0 += 32) {
      if (a.B > 32) {
        n = b0 + lane < a.B ? steps(b0 + lane) * U : 0;
        inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(kFull, inc, o);
          if (lane >= o) inc += y;
        }
      }
      const unsigned past = __ballot_sync(kFull, before + inc > x);
      if (past) {
        const int w = __ffs(past) - 1;
        const unsigned in = x - (before + __shfl_sync(kFull, inc - n, w)), nn = __shfl_sync(kFull, n, w) / U, u = in / nn;
        return Walk{b0 + w, (int)u, (int)(in - u * nn), (int)nn};
      }
      before += __shfl_sync(kFull, inc, 31);
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

// The parts of a unit (CTAs c_first .. c_last), joined in their order.  The weights of a chunk of
// parts are computed side by side, then each thread sums four channels over them with its loads in
// flight together.  wt: [2][kChunk][ROWS] floats; norm: [ROWS] maxima, then [ROWS] sums.
template <class P, class Store>
__device__ __forceinline__ void join_parts(const float* part, int c_first, int c_last, int rows, float* wt, float* norm, Store store) {
  constexpr int ROWS = P::Tl::ROWS, D = P::Tl::D, REC = ROWS * (D + 2), kChunk = P::JOIN / 8 / ROWS;
  static_assert(2 * ROWS <= kThreads, "rows");
  const int tid = threadIdx.x, n = c_last - c_first + 1;
  auto at = [&](int i) { return part + (size_t)(2 * (c_first + i) + (i == 0 ? 1 : 0)) * REC; };
  // the maxima of all parts: kThreads / ROWS threads a row
  constexpr int PER = kThreads / ROWS;
  const int jr = tid % ROWS, pr = tid / ROWS;
  float m = -INFINITY;
#pragma unroll 4
  for (int i = pr; i < n; i += PER) m = fmaxf(m, __ldcg(at(i) + ROWS * D + jr));
  __syncthreads();
  wt[pr * ROWS + jr] = m;
  __syncthreads();
  if (tid < ROWS) {
    for (int i = 1; i < PER; ++i) m = fmaxf(m, wt[i * ROWS + tid]);
    norm[tid] = m;
    norm[ROWS + tid] = 0.f;
  }
  constexpr int QUADS = ROWS * D / 4, MINE = (QUADS + kThreads - 1) / kThreads;
  float4 v[MINE];
#pragma unroll
  for (int k = 0; k < MINE; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kChunk) {
    const int nc = min(kChunk, n - i0);
    __syncthreads();
    float* wl = wt + kChunk * ROWS;
#pragma unroll 4
    for (int e = tid; e < nc * ROWS; e += kThreads) {
      const float* p = at(i0 + e / ROWS) + ROWS * D + e % ROWS;
      const float mj = norm[e % ROWS], mp = __ldcg(p), lp = __ldcg(p + ROWS);
      wt[e] = mp == -INFINITY ? 0.f : ex2(mp - mj);
      wl[e] = mp == -INFINITY ? 0.f : lp * wt[e];
    }
    __syncthreads();
    if (tid < ROWS) {
      float l = norm[ROWS + tid];
      for (int i = 0; i < nc; ++i) l += wl[i * ROWS + tid];
      norm[ROWS + tid] = l;
    }
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int e = tid + k * kThreads, j = e / (D / 4);
      if (j >= rows) continue;
#pragma unroll 8
      for (int i = 0; i < nc; ++i) {
        const float4 p = __ldcg(reinterpret_cast<const float4*>(at(i0 + i)) + e);
        const float w = wt[i * ROWS + j];
        if (w != 0.f) {
          v[k].x = fmaf(w, p.x, v[k].x);
          v[k].y = fmaf(w, p.y, v[k].y);
          v[k].z = fmaf(w, p.z, v[k].z);
          v[k].w = fmaf(w, p.w, v[k].w);
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int e = tid + k * kThreads, j = e / (D / 4);
    if (j >= rows) continue;
    const float inv = norm[j] == -INFINITY ? 0.f : 1.f / norm[ROWS + j];
    store(j, e % (D / 4) * 4, norm[j] == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                  : make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv));
  }
}

template <int BITS, int D, int ROWS, bool F32>
__global__ void __launch_bounds__(kThreads, Plan<BITS, D, ROWS, F32>::MINB)
decode_kernel(Args a, int row_tiles, const void* __restrict__ qv, const int32_t* __restrict__ lens, void* __restrict__ outv,
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
  int* shared_int = reinterpret_cast<int*>(tops + 2 * kWarps * ROWS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* q = static_cast<const T*>(qv);
  T* out = static_cast<T*>(outv);
  const int rows_all = a.n * a.g;
  const Line<P> line{a, lens, a.n_layers * a.Hkv * row_tiles};
  uint2 scan;
  const unsigned total = line.total(scan);
  // a piece of fewer steps than kLeast would be gone before the joining of its parts
  const unsigned want = (total + kLeast - 1) / kLeast;
  const int workers = want < gridDim.x ? (int)want : gridDim.x, me = blockIdx.x;
  if (me >= workers) return;
  if (me == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (len_bad(a, lens, b)) flag(a, KVQ_ERR_RANGE);
  const Cut cut(total, workers);
  const unsigned s0 = cut.begin(me), s1 = cut.begin(me + 1);
  Walk cur = line.at(s0, scan), ahead = cur;
  line.forward(ahead, warp);
  unsigned xa = s0 + warp;                      // the next step to load
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
    if (xa >= s1) return;
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
  for (unsigned x = s0; x < s1;) {              // a unit's part at a time
    const unsigned x1 = min(s1, x + (cur.n - cur.st));
    const int unit0 = (int)x - cur.st;          // its first step
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
    // this warp's steps of the part: x = s0 + warp modulo kWarps
    int st = cur.st + (int)((warp - (x - s0) % kWarps + kWarps) % kWarps);
    const int st1 = cur.st + (int)(x1 - x);
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
    // join the warps: common maximum, scaled sums, channels added warp by warp
    tile.reduce();
    tile.store_tops(tops + warp * ROWS, tops + (kWarps + warp) * ROWS);
    __syncthreads();
    tile.store_out(join + warp * ROWS * D, [&](int j) {
      float m = tops[j];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, tops[w * ROWS + j]);
      const float mine = tops[warp * ROWS + j];
      return mine == -INFINITY ? 0.f : ex2(mine - m);
    });
    __syncthreads();
    const bool starts = unit0 >= (int)s0, whole = starts && unit0 + cur.n <= (int)s1;
    constexpr int REC = ROWS * (D + 2);         // floats of a part: [ROWS][D], maxima, sums of the weights
    float* rec = part + (size_t)(2 * me + (starts ? 1 : 0)) * REC;
    for (int e = tid; e < rows * D; e += kThreads) {
      const int j = e / D, c = e % D;
      float m = tops[j], lsum = 0.f, v = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, tops[w * ROWS + j]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = tops[w * ROWS + j];
        if (mw != -INFINITY) lsum = fmaf(tops[(kWarps + w) * ROWS + j], ex2(mw - m), lsum);
        v += join[(size_t)(w * ROWS + j) * D + c];
      }
      if (whole) {
        out[row_at(j) + c] = from_f<T>(m == -INFINITY ? 0.f : v / lsum);
      } else {
        rec[e] = v;
        if (c == 0) {
          rec[ROWS * D + j] = m;
          rec[ROWS * D + ROWS + j] = lsum;
        }
      }
    }
    if (!whole) {
      // the last CTA of the unit to come joins all parts, in their order
      const int c_first = cut.piece_of(unit0), c_last = cut.piece_of(unit0 + cur.n - 1);
      __threadfence();
      __syncthreads();
      unsigned* cnt = arrived + (size_t)cur.b * line.U + cur.u;
      if (tid == 0) {
        const int last = atomicAdd(cnt, 1u) == (unsigned)(c_last - c_first);
        if (last) *cnt = 0;                     // ready for the next call
        *shared_int = last;
      }
      __syncthreads();
      if (*shared_int) {
        __threadfence();
        join_parts<P>(part, c_first, c_last, rows, join, tops, [&](int j, int c, float4 v) {
          T* o = out + row_at(j) + c;
          if constexpr (F32) {
            *reinterpret_cast<float4*>(o) = v;
          } else {
            __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
            *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(h);
          }
        });
      }
    }
    __syncthreads();                            // the queries' operands and the sums may be written anew
    x = x1;
    cur.st += (int)(x1 - cur.st - unit0);
    if (cur.st >= cur.n) line.next_unit(cur);
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
  static int workers[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int w = dev < 64 ? workers[dev] : 0;
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
  // the line of steps is counted in 32 bits
  if ((double)a.n_layers * a.B * a.Hkv * tiles * ((((double)a.max_pages * a.page) + 16 * P::TB - 1) / (16 * P::TB) + 1) >= 2147483648.0)
    return cudaErrorInvalidConfiguration;
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
