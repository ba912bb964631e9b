// Host checks shared by the entry points over the key/value cache.
#pragma once

#include <limits.h>
#include <math.h>

#include "nvfp4_kv.h"

namespace nvfp4 {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) {
  if (a < 0 || b < 0 || (a != 0 && b > INT64_MAX / a)) return false;
  *out = a * b;
  return true;
}

inline hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

#define NVFP4_TRY(expr)               \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != NVFP4_OK) return rc_;  \
  } while (0)

inline int check_dtype(int dtype) {
  return dtype == NVFP4_DTYPE_F32 || dtype == NVFP4_DTYPE_BF16 ? NVFP4_OK : NVFP4_ERR_DTYPE;
}

// the head scales: every kernel reads them, also those that only write zeros
inline int check_scales(const nvfp4_kv_cache *c) {
  if (!c->S_k || !c->S_v) return NVFP4_ERR_NULL;
  return aligned(c->S_k, 4) && aligned(c->S_v, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// sizes of the cache, then its pointers; without pages or heads it needs none here, and what
// launches for it all the same checks the head scales
inline int check_cache(const nvfp4_kv_cache *c, int64_t max_head_dim) {
  if (!c) return NVFP4_ERR_NULL;
  if (c->pages < 0 || c->pages > INT32_MAX || c->kv_heads < 0 || c->kv_heads > 65535)
    return NVFP4_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 32768 || (c->page_size & (c->page_size - 1)))
    return NVFP4_ERR_SHAPE;
  if (c->head_dim < 16 || c->head_dim > max_head_dim || c->head_dim % 16) return NVFP4_ERR_SHAPE;
  int64_t n;
  if (!mul_ok(c->pages * c->page_size, c->kv_heads * c->head_dim, &n)) return NVFP4_ERR_SHAPE;
  if (n == 0) return NVFP4_OK;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return NVFP4_ERR_NULL;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16))
    return NVFP4_ERR_ALIGN;
  return check_scales(c);
}

// rows x[t][h] of a strided tensor: 16-byte pieces, offsets within int64
inline int check_rows(const void *x, int dtype, int64_t tokens, int64_t heads, int64_t ts, int64_t hs) {
  const int64_t size = dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16)) return NVFP4_ERR_ALIGN;
  if (ts < 0 || hs < 0) return NVFP4_ERR_SHAPE;
  int64_t a, b;
  if (!mul_ok(ts, tokens, &a) || !mul_ok(hs, heads, &b) || a > INT64_MAX / 16 || b > INT64_MAX / 16)
    return NVFP4_ERR_SHAPE;
  if ((ts * size) % 16 || (hs * size) % 16) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Everything of an attention call but its pointers; fills what the plan needs.
inline int check_attention(const nvfp4_kv_cache *c, int dtype, int64_t tokens, int64_t heads,
                    int64_t batch, int64_t max_q, int64_t max_kv, int64_t prefix_len,
                    KvAttention *a) {
  NVFP4_TRY(check_dtype(dtype));
  NVFP4_TRY(check_cache(c, 256));
  if (tokens < 0 || heads < 0 || batch < 0 || max_q < 0 || max_kv < 0 || prefix_len < 0)
    return NVFP4_ERR_SHAPE;
  if (tokens > INT32_MAX || heads > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (batch > 65535 || max_q > tokens || max_kv > (1 << 30) || prefix_len > (1 << 30))
    return NVFP4_ERR_SHAPE;
  int64_t n;
  // row indices are 32 bits up to the end of the last tile, at most 256 rows past the last row
  if (!mul_ok(tokens, heads, &n) || n > INT32_MAX - 1024) return NVFP4_ERR_SHAPE;
  if (heads > 0 && (c->kv_heads == 0 || heads % c->kv_heads)) return NVFP4_ERR_SHAPE;
  *a = KvAttention{};
  a->cache = c, a->dtype = dtype, a->tokens = tokens, a->heads = heads, a->batch = batch;
  a->max_q = max_q, a->max_kv = c->pages ? max_kv : 0, a->prefix_len = c->pages ? prefix_len : 0;
  return NVFP4_OK;
}

inline bool nothing(const KvAttention &a) {
  return a.tokens == 0 || a.heads == 0 || a.batch == 0 || a.max_q == 0;
}

// The call's pointers and strides, into `a` of check_attention; fits() says whether the call's launches
// are possible. A call with nothing to do passes.
template <typename Fits>
inline int check_attention_call(KvAttention *a, const void *q, int64_t q_ts, int64_t q_hs, const int32_t *q_offsets,
                                const int32_t *block_table, int64_t table_width, const int32_t *kv_lens,
                                const int32_t *prefix_pages, float scale, void *out, float *lse, Fits fits) {
  const nvfp4_kv_cache *cache = a->cache;
  if (table_width < 0 || table_width > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (!q_offsets && a->batch * a->max_q != a->tokens) return NVFP4_ERR_SHAPE;
  if (!isfinite(scale)) return NVFP4_ERR_ARG;
  if (nothing(*a)) return NVFP4_OK;
  NVFP4_TRY(check_scales(cache));
  if (a->max_kv > table_width * cache->page_size) return NVFP4_ERR_SHAPE;
  if (!fits()) return NVFP4_ERR_SHAPE;
  if (!q || !out || (a->max_kv > 0 && (!kv_lens || !block_table)) || (a->prefix_len > 0 && !prefix_pages))
    return NVFP4_ERR_NULL;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(q_offsets, 4) || !aligned(block_table, 4) ||
      !aligned(kv_lens, 4) || !aligned(prefix_pages, 4))
    return NVFP4_ERR_ALIGN;
  NVFP4_TRY(check_rows(q, a->dtype, a->tokens, a->heads, q_ts, q_hs));
  a->q = q, a->q_ts = q_ts, a->q_hs = q_hs, a->q_offsets = q_offsets;
  a->block_table = block_table, a->table_width = table_width;
  a->kv_lens = a->max_kv > 0 ? kv_lens : nullptr;
  a->prefix_pages = prefix_pages, a->scale = scale, a->out = out, a->lse = lse;
  return NVFP4_OK;
}

inline int check_workspace(size_t need, const void *workspace, size_t bytes) {
  if (need && (!workspace || bytes < need)) return NVFP4_ERR_WORKSPACE;
  return need && !aligned(workspace, 16) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

inline void debug_check_attention(const KvAttention &a, hipStream_t st) {
  if (!debug_checks_enabled()) return;
  debug_check_finite_rows(a.q, a.dtype, a.tokens, a.heads, a.cache->head_dim, a.q_ts, a.q_hs, st);
  if (a.cache->pages > 0) {
    debug_check_scale(a.cache->S_k, a.cache->kv_heads, st);
    debug_check_scale(a.cache->S_v, a.cache->kv_heads, st);
  }
}

}  // namespace nvfp4
