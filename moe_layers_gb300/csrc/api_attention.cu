// C ABI of the attention operators: argument checks, workspaces, launches.
#include <algorithm>
#include <cmath>

#include "internal.h"

using namespace dec;

namespace {

constexpr int kMaxAttentionRows = 64;
constexpr int kMaxBatchRequests = 64;
constexpr int kMaxTableRequests = 1024;
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxKeys = 0x7fffff00;  // a tile's end past the last key stays an int

inline bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool block_size_ok(int s) { return s == 16 || s == 32 || s == 64 || s == 128; }
inline dec_status status(cudaError_t e) { return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA; }

}  // namespace

namespace dec {

bool cache_ok(const dec_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || !al(c->k, 16) || !al(c->v, 16)) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (!block_size_ok(c->block_size) || c->kv_heads < 1 || c->kv_heads > 128 || c->blocks < 1) return false;
  if ((long long)c->blocks * c->block_size > 0x7fffffffLL) return false;
  return c->block_stride >= (int64_t)c->kv_heads * c->block_size * c->head_dim && c->block_stride % 8 == 0 &&
         c->block_stride < (int64_t)1 << 38;
}

bool batch_ok(const dec_batch* b) {
  if (b == nullptr || b->requests < 1 || b->requests > kMaxBatchRequests || b->max_new < 1 ||
      b->max_new > kMaxAttentionRows || b->max_blocks < 1 || b->max_blocks > 1 << 24 || b->prefix_len < 0)
    return false;
  if (b->row_start == nullptr || b->own_len == nullptr || b->block_table == nullptr) return false;
  if (b->prefix_len > 0 && b->prefix_table == nullptr) return false;
  return al(b->row_start, 4) && al(b->own_len, 4) && al(b->block_table, 4) && al(b->prefix_table, 4);
}

bool rope_ok(const dec_rope* r, int head_dim) {
  if (r == nullptr || r->rotary_dim < 0 || r->rotary_dim > head_dim || r->rotary_dim % 16 != 0) return false;
  if (r->rotary_dim == 0) return true;
  return r->phases != nullptr && al(r->phases, 16) && std::isfinite(r->magnitude) &&
         (r->interleaved == 0 || r->interleaved == 1);
}

// Far enough from 0 and infinity that a masked score times it is minus infinity
// and a score of zero stays zero.
bool scale_ok(float s) { return s >= 1e-30f && s <= 1e30f; }

bool attention_shape_ok(int M, int q_heads, const dec_kv_cache* c, const dec_batch* b) {
  return M >= 1 && M <= kMaxAttentionRows && cache_ok(c) && batch_ok(b) && q_heads >= c->kv_heads &&
         q_heads % c->kv_heads == 0 && q_heads / c->kv_heads <= 128 && q_heads <= 1024 &&
         (long long)b->max_blocks * c->block_size <= kMaxKeys && b->prefix_len <= kMaxKeys;
}

static AttentionParams attention_params(const uint16_t* q, long long ldq, const dec_kv_cache& cache,
                                        const dec_batch& batch, float scale, uint16_t* out, long long ldo, int M,
                                        int q_heads, bool zero_idle) {
  AttentionParams P;
  P.q = q;
  P.ldq = ldq;
  P.out = out;
  P.ldo = ldo;
  P.k = cache.k;
  P.v = cache.v;
  P.block_stride = cache.block_stride;
  P.blocks = cache.blocks;
  P.shift = 0;
  while ((1 << P.shift) < cache.block_size) ++P.shift;
  P.kv_heads = cache.kv_heads;
  P.q_heads = q_heads;
  P.group = q_heads / cache.kv_heads;
  P.dim = cache.head_dim;
  P.requests = batch.requests;
  P.max_new = batch.max_new;
  P.max_blocks = batch.max_blocks;
  P.prefix_len = batch.prefix_len;
  P.M = M;
  P.row_start = batch.row_start;
  P.own_len = batch.own_len;
  P.block_table = batch.block_table;
  P.prefix_table = batch.prefix_table;
  P.scale = scale;
  P.zero_idle = zero_idle;
  return P;
}

dec_status layer_attention(dec_handle* h, const dec_layer_attention& A, uint16_t* y, long long ldy, uint16_t* out,
                           long long ldo, int M, void* ws, cudaStream_t s) {
  const dec_kv_cache& c = *A.cache;
  const long long q = (long long)A.q_heads * c.head_dim, kv = (long long)c.kv_heads * c.head_dim;
  const dec_rope none = {0, 0, 1.f, nullptr};
  {
    LaunchScope scope(h, "rope_append", s);
    if (launch_rope_append(h, A.rope ? *A.rope : none, y, ldy, y + q, ldy, y + q + kv, ldy, y, ldy, M, A.q_heads,
                           A.positions, A.slots, c, s) != cudaSuccess)
      return DEC_ERR_CUDA;
  }
  return status(
      launch_attention(h, attention_params(y, ldy, c, *A.batch, A.scale, out, ldo, M, A.q_heads, true), ws, s));
}

}  // namespace dec

extern "C" {

dec_status dec_batch_tables(dec_handle* h, const int32_t* ctx_len, const int32_t* new_len, int requests,
                            const int32_t* free_blocks, const int32_t* free_count, int32_t* block_table,
                            int max_blocks, int block_size, int position_offset, int rows,
                            const dec_step_tables* out, cudaStream_t stream) {
  if (h == nullptr || ctx_len == nullptr || new_len == nullptr || free_blocks == nullptr || free_count == nullptr ||
      block_table == nullptr || out == nullptr)
    return DEC_ERR_INVALID_ARG;
  if (!out->row_start || !out->own_len || !out->positions || !out->slots || !out->left) return DEC_ERR_INVALID_ARG;
  for (const void* p : {(const void*)ctx_len, (const void*)new_len, (const void*)free_blocks, (const void*)free_count,
                        (const void*)block_table, (const void*)out->row_start, (const void*)out->own_len,
                        (const void*)out->positions, (const void*)out->slots, (const void*)out->left})
    if (!al(p, 4)) return DEC_ERR_INVALID_ARG;
  if (requests < 1 || requests > kMaxTableRequests || rows < 1 || rows > kMaxTokens || !block_size_ok(block_size) ||
      max_blocks < 1 || max_blocks > 1 << 24 || position_offset < 0)
    return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  LaunchScope scope(h, "batch_tables", stream);
  return status(launch_tables(h, ctx_len, new_len, requests, free_blocks, free_count, block_table, max_blocks,
                              block_size, position_offset, rows, *out, stream));
}

dec_status dec_rope_phases(dec_handle* h, uint64_t* phases, int rotary_dim, double base, int scaling, double factor,
                           double original_len, double low, double high, cudaStream_t stream) {
  if (h == nullptr || phases == nullptr || !al(phases, 16)) return DEC_ERR_INVALID_ARG;
  if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0) return DEC_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return DEC_ERR_INVALID_ARG;
  if (scaling < DEC_ROPE_NONE || scaling > DEC_ROPE_YARN) return DEC_ERR_INVALID_ARG;
  if (scaling >= DEC_ROPE_BANDS &&
      (!(original_len > 0.0) || !std::isfinite(original_len) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  LaunchScope scope(h, "rope_phases", stream);
  return status(
      launch_rope_phases(h, phases, rotary_dim, base, scaling, factor, original_len, low, high, stream));
}

dec_status dec_rope_append(dec_handle* h, const dec_rope* rope, const dec_bf16* q, int64_t ldq, const dec_bf16* k,
                           int64_t ldk, const dec_bf16* v, int64_t ldv, dec_bf16* q_out, int64_t ldqo, int rows,
                           int q_heads, const int32_t* positions, const int32_t* slots, const dec_kv_cache* cache,
                           cudaStream_t stream) {
  if (h == nullptr || !cache_ok(cache) || !rope_ok(rope, cache->head_dim)) return DEC_ERR_INVALID_ARG;
  if (k == nullptr || v == nullptr || positions == nullptr || slots == nullptr) return DEC_ERR_INVALID_ARG;
  if (rows < 1 || rows > kMaxTokens || q_heads < 0 || q_heads > 1024) return DEC_ERR_INVALID_ARG;
  if ((q_heads == 0) != (q == nullptr) || (q == nullptr) != (q_out == nullptr)) return DEC_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(q_out, 16) || !al(k, 16) || !al(v, 16) || !al(positions, 4) || !al(slots, 4))
    return DEC_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)q_heads * cache->head_dim, wk = (int64_t)cache->kv_heads * cache->head_dim;
  const int64_t most = (int64_t)1 << 31;
  if (ldk < wk || ldv < wk || ldk % 8 != 0 || ldv % 8 != 0 || ldk > most || ldv > most) return DEC_ERR_INVALID_ARG;
  if (q != nullptr && (ldq < wq || ldqo < wq || ldq % 8 != 0 || ldqo % 8 != 0 || ldq > most || ldqo > most))
    return DEC_ERR_INVALID_ARG;
  if (q != nullptr && q == q_out && ldq != ldqo) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  LaunchScope scope(h, "rope_append", stream);
  return status(launch_rope_append(h, *rope, q, ldq, k, ldk, v, ldv, q_out, ldqo, rows, q_heads, positions, slots,
                                   *cache, stream));
}

dec_status dec_attention_workspace_size(const dec_handle* h, int M, int q_heads, const dec_kv_cache* cache,
                                        const dec_batch* batch, size_t* bytes) {
  if (h == nullptr || bytes == nullptr || !attention_shape_ok(M, q_heads, cache, batch)) return DEC_ERR_INVALID_ARG;
  *bytes = attention_ws_bytes(h, M, q_heads, *cache, *batch);
  return DEC_OK;
}

dec_status dec_attention(dec_handle* h, const dec_bf16* q, int64_t ldq, const dec_kv_cache* cache,
                         const dec_batch* batch, float scale, dec_bf16* out, int64_t ldo, int M, int q_heads,
                         void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (h == nullptr || q == nullptr || out == nullptr || q == out || !attention_shape_ok(M, q_heads, cache, batch))
    return DEC_ERR_INVALID_ARG;
  const int64_t w = (int64_t)q_heads * cache->head_dim, most = (int64_t)1 << 31;
  if (!al(q, 16) || !al(out, 16) || ldq < w || ldo < w || ldq % 8 != 0 || ldo % 8 != 0 || ldq > most || ldo > most)
    return DEC_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return DEC_ERR_INVALID_ARG;
  const size_t need = attention_ws_bytes(h, M, q_heads, *cache, *batch);
  if (need > 0 && (ws == nullptr || !al(ws, 16) || ws_bytes < need)) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  return status(launch_attention(
      h, attention_params(q, ldq, *cache, *batch, scale, out, ldo, M, q_heads, false), ws, stream));
}

}  // extern "C"
