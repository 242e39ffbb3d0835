// kvq_paged_api.cu -- the C ABI of the paged cache: argument checks and
// dispatch to the per-d kernels.  Declarations and contracts: include/kvq.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvq.h"
#include "kvq_host.h"
#include "kvq_paged_launch.h"

namespace {

using namespace kvq::host;

constexpr float kLog2e = 1.44269504088896340736f;

kvq_status check_dtype(kvq_dtype t) {
  return t == KVQ_F16 || t == KVQ_BF16 ? KVQ_OK : KVQ_ERR_BAD_DTYPE;
}

// The token stride of rows [n_tokens][heads][d]: whole 16-byte pieces, rows
// of different tokens apart, and the last element within a signed 64-bit
// byte offset.
bool stride_ok(int64_t stride, int64_t heads, int32_t d, int64_t n_tokens) {
  return stride % 8 == 0 && stride >= heads * d && stride <= (int64_t(1) << 61) / (n_tokens + 1);
}

int log2_page(int32_t page) {
  for (int s = 4; s <= 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}

kvq_status check_rope(const kvq_rope* r, const int32_t* positions, int32_t d,
                      kvq::RopeTable* out) {
  *out = kvq::RopeTable{nullptr, 0, 0, 0, 0.0f};
  if (r == nullptr) return KVQ_OK;
  if (!std::isfinite(r->eps) || r->eps < 0.0f) return KVQ_ERR_BAD_SIZE;
  out->eps = r->eps;
  if (r->cos_sin == nullptr) return KVQ_OK;
  if (r->rot_dim < 16 || r->rot_dim > d || r->rot_dim % 16 != 0 || r->n_pos < 1 ||
      r->n_pos > kMaxRows)
    return KVQ_ERR_BAD_SIZE;
  if (positions == nullptr) return KVQ_ERR_NULL;
  if (!aligned(r->cos_sin, 16) || !aligned(positions, 4)) return KVQ_ERR_MISALIGNED;
  out->cos_sin = r->cos_sin;
  out->n_pos = r->n_pos;
  out->rot_dim = r->rot_dim;
  out->interleaved = r->interleaved != 0;
  return KVQ_OK;
}

kvq_status check_cache(const kvq_paged_cache* c) {
  if (c == nullptr) return KVQ_ERR_NULL;
  if (kvq_status s = check_shape(c->d, c->group, c->rot)) return s;
  if (c->n_pages < 1 || c->n_pages > kMaxRows || c->n_kv_heads < 1 || c->n_kv_heads > 65535 ||
      log2_page(c->page_size) < 0)
    return KVQ_ERR_BAD_SIZE;
  if (!c->k_packed || !c->v_packed || !c->k_scales || !c->v_scales || !c->signs)
    return KVQ_ERR_NULL;
  if (!aligned(c->k_packed, 16) || !aligned(c->v_packed, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16))
    return KVQ_ERR_MISALIGNED;
  return KVQ_OK;
}

bool dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

}  // namespace

extern "C" {

kvq_status kvq_qk_norm_rope(const void* q, const void* k, kvq_dtype dtype, int64_t n_tokens,
                            int32_t n_heads, int32_t n_k_heads, int32_t d, int64_t q_stride,
                            int64_t k_stride, const int32_t* positions, const float* q_weight,
                            const float* k_weight, const kvq_rope* rope, void* q_out, void* k_out,
                            int64_t q_out_stride, int64_t k_out_stride, kvq_stream stream) {
  if (!dim_ok(d)) return KVQ_ERR_BAD_DIM;
  if (kvq_status s = check_dtype(dtype)) return s;
  if (n_tokens < 0 || n_tokens > kMaxRows || n_heads < 1 || n_heads > 65535 || n_k_heads < 0 ||
      n_k_heads > 65535 || n_tokens * (int64_t(n_heads) + n_k_heads) > kMaxRows ||
      !stride_ok(q_stride, n_heads, d, n_tokens) || !stride_ok(q_out_stride, n_heads, d, n_tokens))
    return KVQ_ERR_BAD_SIZE;
  if (n_k_heads > 0 && (!stride_ok(k_stride, n_k_heads, d, n_tokens) ||
                        !stride_ok(k_out_stride, n_k_heads, d, n_tokens)))
    return KVQ_ERR_BAD_SIZE;
  if (n_tokens == 0) return KVQ_OK;
  if (!q || !q_out || (n_k_heads > 0 && (!k || !k_out))) return KVQ_ERR_NULL;
  if (rope == nullptr && (q_weight || k_weight)) return KVQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4))
    return KVQ_ERR_MISALIGNED;
  kvq::NormRopeArgs a = {};
  if (kvq_status s = check_rope(rope, positions, d, &a.rope)) return s;
  DeviceInfo dev;
  if (kvq_status s = device_info(&dev)) return s;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.positions = positions;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  a.n_rows = n_heads + n_k_heads;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(d == 64    ? kvq::launch_norm_rope<64>(dtype, a, dev.sm_count, st)
                   : d == 128 ? kvq::launch_norm_rope<128>(dtype, a, dev.sm_count, st)
                              : kvq::launch_norm_rope<256>(dtype, a, dev.sm_count, st));
}

kvq_status kvq_paged_append(const void* k, const void* v, kvq_dtype dtype, int64_t n_tokens,
                            int64_t k_stride, int64_t v_stride, const int64_t* slots,
                            const int32_t* positions, const float* k_weight, const kvq_rope* rope,
                            const kvq_paged_cache* cache, void* k_hat, void* v_hat,
                            kvq_stream stream) {
  if (kvq_status s = check_cache(cache)) return s;
  if (kvq_status s = check_dtype(dtype)) return s;
  const int64_t heads = cache->n_kv_heads;
  if (n_tokens < 0 || n_tokens > kMaxRows || n_tokens * heads > kMaxRows / 2 ||
      !stride_ok(k_stride, heads, cache->d, n_tokens) ||
      !stride_ok(v_stride, heads, cache->d, n_tokens))
    return KVQ_ERR_BAD_SIZE;
  if (n_tokens == 0) return KVQ_OK;
  if (!k || !v || !slots || (rope == nullptr && k_weight)) return KVQ_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(k_weight, 16) ||
      !aligned(k_hat, 16) || !aligned(v_hat, 16))
    return KVQ_ERR_MISALIGNED;
  kvq::AppendArgs a = {};
  if (kvq_status s = check_rope(rope, positions, cache->d, &a.rope)) return s;
  DeviceInfo dev;
  if (kvq_status s = device_info(&dev)) return s;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.positions = positions;
  a.k_weight = k_weight;
  a.k_packed = cache->k_packed;
  a.v_packed = cache->v_packed;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.signs = cache->signs;
  a.k_hat = static_cast<uint16_t*>(k_hat);
  a.v_hat = static_cast<uint16_t*>(v_hat);
  a.n_tokens = n_tokens;
  a.n_slots = cache->n_pages * cache->page_size;
  a.n_heads = cache->n_kv_heads;
  a.dtype = dtype;
  a.page_shift = log2_page(cache->page_size);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rot = cache->rot, g = cache->group;
  return from_cuda(cache->d == 64    ? kvq::launch_append<64>(rot, g, a, dev.sm_count, st)
                   : cache->d == 128 ? kvq::launch_append<128>(rot, g, a, dev.sm_count, st)
                                     : kvq::launch_append<256>(rot, g, a, dev.sm_count, st));
}

int64_t kvq_paged_attend_workspace(int64_t n_tokens, int32_t n_kv_heads, int32_t n_q, int32_t d,
                                   int32_t max_q_len) {
  if (!dim_ok(d)) return -KVQ_ERR_BAD_DIM;
  if (n_tokens < 0 || n_tokens > kMaxRows || n_kv_heads < 1 || n_q < 1 || n_q > 64 ||
      int64_t(n_kv_heads) * n_q > 65535 || n_tokens * n_kv_heads * n_q > kMaxRows || max_q_len < 1)
    return -KVQ_ERR_BAD_SIZE;
  return kvq::attn_workspace(d, int64_t(max_q_len) * n_q);
}

kvq_status kvq_paged_attend(const void* q, kvq_dtype dtype, int64_t n_tokens, int64_t q_stride,
                            const kvq_paged_cache* cache, const int32_t* cu_q,
                            const int32_t* kv_len, const int32_t* page_table, int64_t n_seqs,
                            int64_t max_pages, int32_t n_q, int32_t max_q_len, int32_t window,
                            float sm_scale, void* out, int64_t out_stride, void* workspace,
                            int64_t workspace_bytes, kvq_stream stream) {
  if (kvq_status s = check_cache(cache)) return s;
  if (kvq_status s = check_dtype(dtype)) return s;
  const int64_t heads = int64_t(cache->n_kv_heads) * n_q;
  if (n_tokens < 0 || n_tokens > kMaxRows || n_q < 1 || n_q > 64 || heads > 65535 ||
      n_tokens * heads > kMaxRows || n_seqs < 0 || n_seqs > 65535 || max_pages < 0 ||
      max_pages > kMaxRows / cache->page_size || max_q_len < 1 || window < 0 ||
      !std::isfinite(sm_scale) || !stride_ok(q_stride, heads, cache->d, n_tokens) ||
      !stride_ok(out_stride, heads, cache->d, n_tokens))
    return KVQ_ERR_BAD_SIZE;
  if (n_tokens == 0 || n_seqs == 0) return KVQ_OK;
  if (!q || !out || !cu_q || !kv_len || (!page_table && max_pages > 0)) return KVQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(workspace, 256))
    return KVQ_ERR_MISALIGNED;
  DeviceInfo dev;
  if (kvq_status s = device_info(&dev)) return s;
  const int64_t need =
      kvq_paged_attend_workspace(n_tokens, cache->n_kv_heads, n_q, cache->d, max_q_len);
  if (need < 0) return kvq_status(-need);
  if (need > 0 && !workspace) return KVQ_ERR_NULL;
  if (workspace_bytes < need) return KVQ_ERR_BAD_SIZE;
  kvq::PagedAttnArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.k_packed = cache->k_packed;
  a.v_packed = cache->v_packed;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.signs = cache->signs;
  a.n_tokens = n_tokens;
  a.n_pages = cache->n_pages;
  a.max_pages = max_pages;
  a.n_seqs = int(n_seqs);
  a.n_kv = cache->n_kv_heads;
  a.n_q = n_q;
  a.page_shift = log2_page(cache->page_size);
  a.d = cache->d;
  a.group = cache->group;
  a.dtype = dtype;
  a.rot = cache->rot;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.window = window < (1 << 30) ? window : 1 << 30;  // position - window stays in 32 bits
  a.qscale = sm_scale * kLog2e;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(cache->d == 64    ? kvq::launch_paged_attn<64>(a, max_q_len, dev.sm_count, st)
                   : cache->d == 128 ? kvq::launch_paged_attn<128>(a, max_q_len, dev.sm_count, st)
                                     : kvq::launch_paged_attn<256>(a, max_q_len, dev.sm_count, st));
}

}  // extern "C"
