// Host checks shared by the entry points over the key/value cache.
#pragma once

#include <limits.h>

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

}  // namespace nvfp4
