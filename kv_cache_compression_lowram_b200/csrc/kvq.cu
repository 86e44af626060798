// C entry points of the quantised KV cache: argument checks, then the launchers.
#include <string>

#include "kvq.cuh"

namespace lowram {
void set_last_error(const char* msg);
}

namespace {
using namespace lowram;
using namespace lowram::kvq;

lowram_status inval(const char* why) {
  set_last_error(why);
  return LOWRAM_EINVAL;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

lowram_status check(const lowram_kvq_config* c) {
  if (!c) return inval("config is NULL");
  if (c->batch < 1 || c->n_layers < 1 || c->n_kv_heads < 1 || c->n_q_heads < 1 || c->n_pages < 1 || c->max_pages < 1)
    return inval("config sizes must be positive");
  if (c->n_q_heads % c->n_kv_heads || c->n_q_heads / c->n_kv_heads > kMaxG)
    return inval("n_q_heads must be a multiple of n_kv_heads, at most 16 times it");
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return inval("page must be 16, 32, 64, 128 or 256");
  if (c->max_pages > kMaxPagesSeq) return inval("max_pages exceeds 16384");
  if (c->batch > 65535 || c->n_kv_heads > 65535 || c->n_layers > 65535) return inval("batch, n_kv_heads and n_layers are at most 65535");
  // (the product of two of the sizes is below 2^47: the others are compared by division)
  if ((uint64_t)c->n_layers * c->n_pages >= (1ull << 32) / ((uint64_t)c->n_kv_heads * c->page) + 1 ||
      (uint64_t)c->n_layers * c->n_pages * c->n_kv_heads * c->page >= (1ull << 32))
    return inval("rows of the pool (n_layers * n_pages * n_kv_heads * page) must stay below 2^32");
  if (c->bits != 4 && c->bits != 8) return inval("bits must be 4 or 8");
  if (c->dtype != LOWRAM_F32 && c->dtype != LOWRAM_BF16) return inval("unknown dtype");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) {
    set_last_error("the quantised cache takes head_dim 64, 128 or 256");
    return LOWRAM_EUNSUPPORTED;
  }
  return LOWRAM_OK;
}

lowram_status check_cache(const lowram_kvq_config* c, const lowram_kvq_cache* k, int32_t layer0, int32_t n_layers, Args* a) {
  lowram_status st = check(c);
  if (st != LOWRAM_OK) return st;
  if (!k) return inval("cache is NULL");
  const void* need[] = {k->k_code, k->k_scale, k->v_code, k->v_scale};
  for (const void* p : need)
    if (!p || !aligned16(p)) return inval("a cache array is NULL or not 16-byte aligned");
  if (!aligned16(k->k_mean)) return inval("k_mean is not 16-byte aligned");
  if (!aligned4(k->table) || !aligned4(k->err)) return inval("table or err is misaligned");
  if (!k->table && (int64_t)c->batch * c->max_pages > c->n_pages) return inval("without a table the pool needs batch * max_pages pages");
  if (layer0 < 0 || n_layers < 1 || layer0 > c->n_layers - n_layers) return inval("bad layer range");
  int lg = 4;
  while ((1 << lg) < c->page) ++lg;
  *a = Args{c->batch, c->n_kv_heads, c->n_q_heads, c->n_q_heads / c->n_kv_heads, lg, c->page, c->n_pages, c->max_pages, c->bits,
            c->head_dim, layer0, n_layers, 0, static_cast<uint8_t*>(k->k_code), static_cast<uint8_t*>(k->v_code),
            static_cast<__half2*>(k->k_scale), static_cast<__half2*>(k->v_scale), static_cast<__nv_bfloat16*>(k->k_mean),
            k->table, k->err};
  return LOWRAM_OK;
}

lowram_status check_rows(const Args& a, int dtype, const void* p, const int64_t* st, bool writes, Rows* r) {
  if (!p || !st || !aligned16(p)) return inval("k or v is NULL or not 16-byte aligned, or has no strides");
  const int64_t unit = dtype == LOWRAM_F32 ? 4 : 8;
  const int64_t ext[4] = {a.n_layers, a.B, a.n, a.Hkv};
  int64_t use[4];
  for (int i = 0; i < 4; ++i) {
    use[i] = ext[i] > 1 ? st[i] : 0;   // an axis of one is never stepped along
    if (use[i] < 0 || use[i] % unit) return inval("strides of k and v must be multiples of 16 bytes and not negative");
    if (writes && ext[i] > 1 && st[i] == 0) return inval("an output axis longer than one has stride 0");
  }
  *r = Rows{const_cast<void*>(p), use[0], use[1], use[2], use[3]};
  return LOWRAM_OK;
}

lowram_status done(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return LOWRAM_OK;
  const std::string msg = std::string(where) + ": " + cudaGetErrorString(e);
  set_last_error(msg.c_str());
  return LOWRAM_ECUDA;
}

lowram_status rows_call(bool writes, const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers,
                        int32_t n, const void* k, const int64_t* ks, const void* v, const int64_t* vs, const int32_t* pos,
                        const int32_t* count, lowram_stream stream) {
  Args a;
  Rows rk, rv;
  lowram_status st = check_cache(cfg, cache, layer0, n_layers, &a);
  if (st != LOWRAM_OK) return st;
  if (n < 0 || n > (a.max_pages << a.page_log2)) return inval("the token count must lie in [0, max_pages * page]");
  if (n == 0) return LOWRAM_OK;
  a.n = n;
  if (!pos) return inval("pos is NULL");
  if (!aligned4(pos) || !aligned4(count)) return inval("pos or count is misaligned");
  if ((st = check_rows(a, cfg->dtype, k, ks, !writes, &rk)) != LOWRAM_OK) return st;
  if ((st = check_rows(a, cfg->dtype, v, vs, !writes, &rv)) != LOWRAM_OK) return st;
  const long long pieces = ((n - 1) >> a.page_log2) + 2;
  if (pieces * a.n_layers * a.B * a.Hkv >= (1LL << 31)) return inval("too many rows for one call: split the layers");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return writes ? done(launch_write(a, cfg->dtype, rk, rv, pos, count, s), "kvq write")
                : done(launch_read(a, cfg->dtype, rk, rv, pos, count, s), "kvq read");
}

lowram_status check_attn(const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers, int32_t n_q,
                         const void* q, const int32_t* lens, const void* out, Args* a) {
  lowram_status st = check_cache(cfg, cache, layer0, n_layers, a);
  if (st != LOWRAM_OK) return st;
  if (n_q < 1 || n_q > kMaxQ) return inval("n_q must lie in [1, 16]");
  if (!q || !out || !lens || !aligned16(q) || !aligned16(out)) return inval("q, out or lens is NULL, or q or out not 16-byte aligned");
  if (!aligned4(lens)) return inval("lens is misaligned");
  if ((long long)n_layers * a->B * a->Hkv * n_q >= (1LL << 27)) return inval("too many queries for one call: split the layers");
  const uint64_t bytes = (uint64_t)n_layers * a->B * n_q * a->Hq * a->d * (cfg->dtype == LOWRAM_F32 ? 4 : 2);
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  if (q0 != o0 && (q0 < o0 ? o0 - q0 : q0 - o0) < bytes) return inval("out overlaps q in part");
  a->n = n_q;
  return LOWRAM_OK;
}
}  // namespace

extern "C" {

uint64_t lowram_kvq_token_bytes(const lowram_kvq_config* cfg) {
  if (check(cfg) != LOWRAM_OK) return 0;
  return 2ull * ((uint64_t)cfg->head_dim * cfg->bits / 8 + cfg->head_dim / kGroup * 4);
}

lowram_status lowram_kvq_write(const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers,
                               int32_t n_new, const void* k, const int64_t* k_stride, const void* v, const int64_t* v_stride,
                               const int32_t* pos, const int32_t* count, lowram_stream stream) {
  return rows_call(true, cfg, cache, layer0, n_layers, n_new, k, k_stride, v, v_stride, pos, count, stream);
}

lowram_status lowram_kvq_read(const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers,
                              int32_t n_tok, void* k_out, const int64_t* k_stride, void* v_out, const int64_t* v_stride,
                              const int32_t* pos, const int32_t* count, lowram_stream stream) {
  return rows_call(false, cfg, cache, layer0, n_layers, n_tok, k_out, k_stride, v_out, v_stride, pos, count, stream);
}

uint64_t lowram_kvq_workspace_bytes(const lowram_kvq_config* cfg, int32_t n_layers, int32_t n_q) {
  if (check(cfg) != LOWRAM_OK) return 0;
  if (n_layers < 1 || n_layers > cfg->n_layers || n_q < 1 || n_q > kMaxQ) {
    inval("n_layers or n_q out of range");
    return 0;
  }
  Args a{};
  a.B = cfg->batch; a.Hkv = cfg->n_kv_heads; a.Hq = cfg->n_q_heads; a.g = a.Hq / a.Hkv;
  a.d = cfg->head_dim; a.bits = cfg->bits; a.n_layers = n_layers; a.n = n_q;
  return decode_workspace_bytes(a);
}

lowram_status lowram_kvq_decode_attn(const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers,
                                     int32_t n_q, const void* q, const int32_t* lens, void* out, void* workspace,
                                     uint64_t workspace_bytes, lowram_stream stream) {
  Args a;
  lowram_status st = check_attn(cfg, cache, layer0, n_layers, n_q, q, lens, out, &a);
  if (st != LOWRAM_OK) return st;
  if (!decode_line_fits(a)) return inval("too much work for one call: split the layers");
  if (!workspace || !aligned16(workspace) || workspace_bytes < decode_workspace_bytes(a))
    return inval("workspace is NULL, not 16-byte aligned or smaller than lowram_kvq_workspace_bytes");
  return done(launch_decode(a, cfg->dtype, q, lens, out, workspace, reinterpret_cast<cudaStream_t>(stream)), "kvq decode");
}

lowram_status lowram_kvq_sparse_attn(const lowram_kvq_config* cfg, const lowram_kvq_cache* cache, int32_t layer0, int32_t n_layers,
                                     int32_t n_q, int32_t top_k, const void* q, const int32_t* lens, void* out, int32_t* sel,
                                     lowram_stream stream) {
  Args a;
  lowram_status st = check_attn(cfg, cache, layer0, n_layers, n_q, q, lens, out, &a);
  if (st != LOWRAM_OK) return st;
  if (top_k < 1 || top_k > kMaxTopK) return inval("top_k must lie in [1, 512]");
  if (!a.k_mean) return inval("the cache has no k_mean");
  if (!aligned4(sel)) return inval("sel is misaligned");
  return done(launch_sparse(a, cfg->dtype, top_k, q, lens, out, sel, reinterpret_cast<cudaStream_t>(stream)), "kvq sparse");
}

}  // extern "C"
