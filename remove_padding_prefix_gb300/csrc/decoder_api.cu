// C ABI of the decoder-serving calls: the paged key-value cache, causal attention over
// packed prompts, and the attention of one new token over the cache.  Argument checks only;
// the kernels are in kv_cache.cu, attention_causal.cu and attention_decode.cu.
#include "kernels.h"

namespace rpp {
namespace {

// Rows of a call and tokens of a sequence: a page (65536 rows at most) more is still an int, so counts of pages
// and tiles are rounded up without care.  The same for pages and the kernels' strides over them.
constexpr long long kMostRows = 0x7fffffffLL - 65535;
constexpr int kMostPages = 1 << 30;
// The kernels take scale * log2(e), which has to be finite: 0 scores are NaN otherwise.
constexpr float kMostScale = 2.0e38f;

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

rpp_status kv_cfg_ok(const rpp_kv_cfg* c) {
  if (!c || c->layers <= 0 || c->pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 ||
      c->slots <= 0 || c->max_pages <= 0)
    return RPP_EINVAL;
  if (static_cast<long long>(c->slots) * c->max_pages > 0x7fffffffLL ||
      static_cast<long long>(c->max_pages) * c->page_size > kMostRows)
    return RPP_EINVAL;
  if (c->dtype != RPP_F16 && c->dtype != RPP_BF16) return RPP_EUNSUPPORTED;
  if (c->head_dim % 8 || c->slots > kKvMaxSlots || c->layers > 65536 || c->page_size > 65536 ||
      static_cast<long long>(c->kv_heads) * c->head_dim > 65536 || c->pages > kMostPages)
    return RPP_EUNSUPPORTED;
  // bytes of the pool, below 2^62: a layer's pages are at most 2^30 * 2^34 of them
  const long long page = 4LL * c->kv_heads * c->head_dim * c->page_size;
  if (page > (1LL << 62) / c->pages / c->layers) return RPP_EUNSUPPORTED;
  return RPP_OK;
}

KvDims dims(const rpp_kv_cfg* c) {
  return KvDims{c->layers, c->pages, c->page_size, c->kv_heads, c->head_dim, c->slots, c->max_pages};
}
KvState state(const rpp_kv_cache* k) { return KvState{k->pool, k->table, k->lens, k->refs}; }

rpp_status kv_ok(const rpp_kv_cfg* c, const rpp_kv_cache* k) {
  const rpp_status st = kv_cfg_ok(c);
  if (st != RPP_OK) return st;
  if (!k || !k->pool || !k->table || !k->lens || !k->refs) return RPP_EINVAL;
  if (!aligned(k->pool, 16) || !aligned(k->refs, 16)) return RPP_EINVAL;
  return RPP_OK;
}

rpp_status list_ok(const rpp_kv_cfg* c, const int32_t* list, int n) {
  if (!list || n <= 0) return RPP_EINVAL;
  return n > kKvMaxList ? RPP_EUNSUPPORTED : RPP_OK;
}

size_t compact_bytes(const rpp_kv_cfg* c) { return (2 + 2 * (static_cast<size_t>(c->pages) / 2)) * sizeof(int32_t); }

}  // namespace
}  // namespace rpp

using namespace rpp;

size_t rpp_kv_pool_bytes(const rpp_kv_cfg* cfg) {
  if (kv_cfg_ok(cfg) != RPP_OK) return 0;
  return static_cast<size_t>(cfg->layers) * cfg->pages * 2 * cfg->kv_heads * cfg->page_size * cfg->head_dim * 2;
}

rpp_status rpp_kv_reserve(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, const int32_t* slots,
                          const int32_t* counts, int n, int32_t* err, rpp_stream stream) {
  rpp_status st = kv_ok(cfg, cache);
  if (st == RPP_OK) st = list_ok(cfg, slots, n);
  if (st != RPP_OK) return st;
  if (!counts || !err) return RPP_EINVAL;
  return status_from_cuda(
      launch_kv_reserve(dims(cfg), state(cache), slots, counts, n, err, static_cast<cudaStream_t>(stream)));
}

rpp_status rpp_kv_append(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, int layer, const void* k, const void* v,
                         int row_stride, const int32_t* slots, const int32_t* cu_seqlens, int n, int rows_max,
                         int32_t* err, rpp_stream stream) {
  rpp_status st = kv_ok(cfg, cache);
  if (st == RPP_OK) st = list_ok(cfg, slots, n);
  if (st != RPP_OK) return st;
  if (!k || !v || !err || layer < 0 || layer >= cfg->layers || rows_max <= 0) return RPP_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || row_stride % 8 || row_stride < cfg->kv_heads * cfg->head_dim)
    return RPP_EINVAL;
  if (!cu_seqlens && rows_max < n) return RPP_EINVAL;
  if (rows_max > kMostRows) return RPP_EUNSUPPORTED;
  return status_from_cuda(launch_kv_append(dims(cfg), state(cache), layer, k, v, row_stride, slots, cu_seqlens, n,
                                           rows_max, err, static_cast<cudaStream_t>(stream)));
}

rpp_status rpp_kv_fork(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, const int32_t* from, const int32_t* to, int n,
                       int32_t* err, rpp_stream stream) {
  rpp_status st = kv_ok(cfg, cache);
  if (st == RPP_OK) st = list_ok(cfg, from, n);
  if (st != RPP_OK) return st;
  if (!to || !err) return RPP_EINVAL;
  return status_from_cuda(
      launch_kv_fork(dims(cfg), state(cache), from, to, n, err, static_cast<cudaStream_t>(stream)));
}

rpp_status rpp_kv_free(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, const int32_t* slots, int n, int32_t* err,
                       rpp_stream stream) {
  rpp_status st = kv_ok(cfg, cache);
  if (st == RPP_OK) st = list_ok(cfg, slots, n);
  if (st != RPP_OK) return st;
  if (!err) return RPP_EINVAL;
  return status_from_cuda(launch_kv_free(dims(cfg), state(cache), slots, n, err, static_cast<cudaStream_t>(stream)));
}

size_t rpp_kv_compact_workspace_bytes(const rpp_kv_cfg* cfg) {
  if (kv_cfg_ok(cfg) != RPP_OK) return 0;
  return compact_bytes(cfg);
}

rpp_status rpp_kv_compact(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, int32_t* table_out, int32_t* refs_out,
                          int32_t* remap, int32_t* live, void* workspace, size_t workspace_bytes, int32_t* err,
                          rpp_stream stream) {
  const rpp_status st = kv_ok(cfg, cache);
  if (st != RPP_OK) return st;
  if (!table_out || !refs_out || !remap || !live || !workspace || !err) return RPP_EINVAL;
  if ((table_out == cache->table) != (refs_out == cache->refs)) return RPP_EINVAL;   // the cache's two would part
  if (!aligned(workspace, 8)) return RPP_EINVAL;
  if (workspace_bytes < compact_bytes(cfg)) return RPP_EWORKSPACE;
  return status_from_cuda(launch_kv_compact(dims(cfg), state(cache), table_out, refs_out, remap, live,
                                            static_cast<int32_t*>(workspace), err, static_cast<cudaStream_t>(stream)));
}

size_t rpp_attention_decode_workspace_bytes(const rpp_kv_cfg* cfg, int n, int nh) {
  if (kv_cfg_ok(cfg) != RPP_OK || n <= 0 || n > kKvMaxList || nh <= 0 || nh % cfg->kv_heads) return 0;
  return attention_decode_ws_bytes(n, nh, cfg->kv_heads, cfg->head_dim);
}

rpp_status rpp_attention_decode(const rpp_kv_cfg* cfg, const rpp_kv_cache* cache, int layer, const void* q,
                                int q_stride, const int32_t* slots, int n, int nh, float scale, void* out,
                                void* workspace, size_t workspace_bytes, int32_t* err, rpp_stream stream) {
  const rpp_status st = kv_ok(cfg, cache);
  if (st != RPP_OK) return st;
  if (!q || !out || !workspace || layer < 0 || layer >= cfg->layers || n <= 0 || nh <= 0 || nh % cfg->kv_heads)
    return RPP_EINVAL;
  if (!slots && n > cfg->slots) return RPP_EINVAL;
  if (!(scale > 0.f) || scale > kMostScale) return RPP_EINVAL;
  if (n > kKvMaxList || nh > 65535) return RPP_EUNSUPPORTED;
  if ((cfg->head_dim != 64 && cfg->head_dim != 128) || cfg->page_size % 16) return RPP_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 ||
      static_cast<long long>(q_stride) < static_cast<long long>(nh) * cfg->head_dim)
    return RPP_EINVAL;
  if (!aligned(workspace, 256)) return RPP_EINVAL;
  if (workspace_bytes < attention_decode_ws_bytes(n, nh, cfg->kv_heads, cfg->head_dim)) return RPP_EWORKSPACE;
  return status_from_cuda(launch_attention_decode(dims(cfg), state(cache), static_cast<rpp_dtype>(cfg->dtype), layer,
                                                  q, q_stride, slots, n, nh, scale, out, workspace, err,
                                                  static_cast<cudaStream_t>(stream)));
}

rpp_status rpp_attention_causal_varlen(const void* q, const void* k, const void* v, int q_stride, int kv_stride,
                                       const int32_t* cu_seqlens, int B, int T_max, int max_len, int nh, int nkv,
                                       int d, rpp_dtype dtype, float scale, void* out, int32_t* err,
                                       rpp_stream stream) {
  if (!q || !k || !v || !cu_seqlens || !out || B <= 0 || T_max <= 0 || max_len <= 0 || nh <= 0 || nkv <= 0 ||
      nh % nkv || d <= 0)
    return RPP_EINVAL;
  if (!(scale > 0.f) || scale > kMostScale) return RPP_EINVAL;
  if (dtype != RPP_F16 && dtype != RPP_BF16) return RPP_EUNSUPPORTED;
  if (!attention_causal_supported(B, max_len, d)) return RPP_EUNSUPPORTED;
  if (T_max > kMostRows || (static_cast<long long>(T_max) / 128 + B) * nh > 0x7fffffffLL ||
      static_cast<long long>(nh) * d > 0x7fffffffLL)
    return RPP_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || q_stride % 8 || kv_stride % 8 ||
      q_stride < nh * d || kv_stride < nkv * d)
    return RPP_EINVAL;
  const CausalArgs a{q, k, v, q_stride, kv_stride, cu_seqlens, B, T_max, max_len, nh, nkv, d, dtype, scale, out, err};
  return status_from_cuda(launch_attention_causal(a, static_cast<cudaStream_t>(stream)));
}
