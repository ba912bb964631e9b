// C-ABI entry points of the key/value cache (declared in include/nvfp4_kv.h): host checks of
// every argument, then the launchers.
#include <limits.h>
#include <math.h>

#include "nvfp4_kv.h"

using namespace nvfp4;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool mul_ok(int64_t a, int64_t b, int64_t *out) {
  if (a < 0 || b < 0 || (a != 0 && b > INT64_MAX / a)) return false;
  *out = a * b;
  return true;
}

hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

#define NVFP4_TRY(expr)               \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != NVFP4_OK) return rc_;  \
  } while (0)

int check_dtype(int dtype) {
  return dtype == NVFP4_DTYPE_F32 || dtype == NVFP4_DTYPE_BF16 ? NVFP4_OK : NVFP4_ERR_DTYPE;
}

// the head scales: every kernel reads them, also those that only write zeros
int check_scales(const nvfp4_kv_cache *c) {
  if (!c->S_k || !c->S_v) return NVFP4_ERR_NULL;
  return aligned(c->S_k, 4) && aligned(c->S_v, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// sizes of the cache, then its pointers; without pages or heads it needs none here, and what
// launches for it all the same checks the head scales
int check_cache(const nvfp4_kv_cache *c, int64_t max_head_dim) {
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
int check_rows(const void *x, int dtype, int64_t tokens, int64_t heads, int64_t ts, int64_t hs) {
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
int check_attention(const nvfp4_kv_cache *c, int dtype, int64_t tokens, int64_t heads,
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

bool nothing(const KvAttention &a) {
  return a.tokens == 0 || a.heads == 0 || a.batch == 0 || a.max_q == 0;
}

}  // namespace

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
  if (table_width < 0 || table_width > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (!q_offsets && batch * max_q != tokens) return NVFP4_ERR_SHAPE;
  if (!isfinite(scale)) return NVFP4_ERR_ARG;
  if (nothing(a)) return NVFP4_OK;
  NVFP4_TRY(check_scales(cache));
  if (a.max_kv > table_width * cache->page_size) return NVFP4_ERR_SHAPE;
  if (!kv_attention_fits(a)) return NVFP4_ERR_SHAPE;
  if (!q || !out || (a.max_kv > 0 && (!kv_lens || !block_table)) ||
      (a.prefix_len > 0 && !prefix_pages))
    return NVFP4_ERR_NULL;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(q_offsets, 4) || !aligned(block_table, 4) ||
      !aligned(kv_lens, 4) || !aligned(prefix_pages, 4))
    return NVFP4_ERR_ALIGN;
  NVFP4_TRY(check_rows(q, dtype, tokens, heads, q_token_stride, q_head_stride));
  const size_t need = kv_attention_workspace_size(a);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  const hipStream_t st = as_stream(stream);
  if (debug_checks_enabled()) {
    debug_check_finite_rows(q, dtype, tokens, heads, cache->head_dim, q_token_stride,
                            q_head_stride, st);
    if (cache->pages > 0) {
      debug_check_scale(cache->S_k, cache->kv_heads, st);
      debug_check_scale(cache->S_v, cache->kv_heads, st);
    }
  }
  a.q = q, a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.q_offsets = q_offsets;
  a.block_table = block_table, a.table_width = table_width;
  a.kv_lens = a.max_kv > 0 ? kv_lens : nullptr;
  a.prefix_pages = prefix_pages, a.scale = scale, a.causal = causal != 0;
  a.out = out, a.lse = lse, a.workspace = workspace;
  return launch_kv_attention(a, st);
}

}  // extern "C"
