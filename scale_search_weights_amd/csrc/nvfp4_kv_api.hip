// C-ABI entry points of the key/value cache (declared in include/nvfp4_kv.h): host checks of
// every argument, then the launchers.
#include "nvfp4_kv_checks.h"

using namespace nvfp4;

extern "C" {

int nvfp4_kv_write(const nvfp4_kv_cache *cache, const void *k, const void *v, int dtype,
                   int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                   int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                   void *stream) {
  NVFP4_TRY(check_dtype(dtype));
  NVFP4_TRY(check_cache(cache, 1024));
  if (tokens < 0 || tokens > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || cache->kv_heads == 0 || cache->pages == 0) return NVFP4_OK;
  if (!k || !v || !slots) return NVFP4_ERR_NULL;
  if (!aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  NVFP4_TRY(check_rows(k, dtype, tokens, cache->kv_heads, k_token_stride, k_head_stride));
  NVFP4_TRY(check_rows(v, dtype, tokens, cache->kv_heads, v_token_stride, v_head_stride));
  const hipStream_t st = as_stream(stream);
  if (debug_checks_enabled()) {
    debug_check_finite_rows(k, dtype, tokens, cache->kv_heads, cache->head_dim, k_token_stride,
                            k_head_stride, st);
    debug_check_finite_rows(v, dtype, tokens, cache->kv_heads, cache->head_dim, v_token_stride,
                            v_head_stride, st);
    debug_check_scale(cache->S_k, cache->kv_heads, st);
    debug_check_scale(cache->S_v, cache->kv_heads, st);
  }
  return launch_kv_write(*cache, k, v, dtype, tokens, k_token_stride, k_head_stride,
                         v_token_stride, v_head_stride, slots, st);
}

int nvfp4_kv_read(const nvfp4_kv_cache *cache, const int64_t *slots, int64_t n, void *k, void *v,
                  int out_dtype, void *stream) {
  NVFP4_TRY(check_dtype(out_dtype));
  NVFP4_TRY(check_cache(cache, 1024));
  if (n < 0 || n > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (n == 0 || cache->kv_heads == 0) return NVFP4_OK;
  NVFP4_TRY(check_scales(cache));
  if (!slots || (!k && !v)) return NVFP4_ERR_NULL;
  if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return NVFP4_ERR_ALIGN;
  const hipStream_t st = as_stream(stream);
  if (cache->pages > 0 && debug_checks_enabled()) {
    debug_check_scale(cache->S_k, cache->kv_heads, st);
    debug_check_scale(cache->S_v, cache->kv_heads, st);
  }
  return launch_kv_read(*cache, slots, n, k, v, out_dtype, st);
}

size_t nvfp4_kv_attention_workspace_size(const nvfp4_kv_cache *cache, int dtype, int64_t tokens,
                                         int64_t heads, int64_t batch, int64_t max_q,
                                         int64_t max_kv, int64_t prefix_len) {
  KvAttention a;
  if (check_attention(cache, dtype, tokens, heads, batch, max_q, max_kv, prefix_len, &a) != NVFP4_OK)
    return 0;
  if (nothing(a) || !kv_attention_fits(a)) return 0;
  return kv_attention_workspace_size(a);
}

int nvfp4_kv_attention(const nvfp4_kv_cache *cache, const void *q, int dtype, int64_t tokens,
                       int64_t heads, int64_t q_token_stride, int64_t q_head_stride, int64_t batch,
                       const int32_t *q_offsets, int64_t max_q, const int32_t *block_table,
                       int64_t table_width, const int32_t *kv_lens, int64_t max_kv,
                       const int32_t *prefix_pages, int64_t prefix_len, float scale, int causal,
                       void *out, float *lse, void *workspace, size_t workspace_bytes,
                       void *stream) {
  KvAttention a;
  NVFP4_TRY(check_attention(cache, dtype, tokens, heads, batch, max_q, max_kv, prefix_len, &a));
  NVFP4_TRY(check_attention_call(&a, q, q_token_stride, q_head_stride, q_offsets, block_table, table_width,
                                 kv_lens, prefix_pages, scale, out, lse,
                                 [&] { return kv_attention_fits(a); }));
  if (nothing(a)) return NVFP4_OK;
  NVFP4_TRY(check_workspace(kv_attention_workspace_size(a), workspace, workspace_bytes));
  const hipStream_t st = as_stream(stream);
  debug_check_attention(a, st);
  a.causal = causal != 0, a.workspace = workspace;
  return launch_kv_attention(a, st);
}

}  // extern "C"
