// C-ABI entry points of the rotation (include/nvfp4_rotary.h) and of the append to the key/value cache
// (include/nvfp4_kv.h): host checks of every argument, then the launchers.
#include <math.h>

#include "nvfp4_kv_checks.h"
#include "nvfp4_rotary.h"

using namespace nvfp4;

namespace {

// The rotation of rows of head_dim channels, its pairs a multiple of `unit`.
int check_rotary(const nvfp4_rotary *r, int64_t head_dim, int64_t unit) {
  if (!r) return NVFP4_ERR_NULL;
  if (r->pairs < unit || r->pairs > 512 || r->pairs % unit || 2 * r->pairs > head_dim)
    return NVFP4_ERR_SHAPE;
  if (r->axes < 1 || r->axes > 16) return NVFP4_ERR_SHAPE;
  return isfinite(r->factor) ? NVFP4_OK : NVFP4_ERR_ARG;
}

int check_positions(const nvfp4_rotary *r, const int64_t *positions, int64_t stride, int64_t tokens,
                    Turn *turn) {
  if (!r->inv_freq || !positions) return NVFP4_ERR_NULL;
  if (!aligned(r->inv_freq, 8) || !aligned(r->axis, 4) || !aligned(positions, 8)) return NVFP4_ERR_ALIGN;
  if (stride < 0 || stride > INT64_MAX / 256 || tokens > INT64_MAX / 256) return NVFP4_ERR_SHAPE;
  *turn = {r->inv_freq, r->axis, positions, stride, r->factor, (int)r->pairs, (int)r->axes};
  return NVFP4_OK;
}

// Rows that are written: one dimension's rows lie within a step of the other, no row on top of another.
int check_out(const void *x, int dtype, int64_t tokens, int64_t heads, int64_t hd, int64_t ts, int64_t hs) {
  NVFP4_TRY(check_rows(x, dtype, tokens, heads, ts, hs));
  const int64_t a = tokens > 1 ? ts : INT64_MAX, b = heads > 1 ? hs : INT64_MAX;
  const bool apart = a < b ? a >= hd && (heads <= 1 || b >= (tokens - 1) * ts + hd)
                           : b >= hd && (tokens <= 1 || a >= (heads - 1) * hs + hd);
  return apart ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

}  // namespace

extern "C" {

int nvfp4_rotate(const nvfp4_rotary *rotary, const int64_t *positions, int64_t position_stride,
                 const void *x, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                 int64_t x_token_stride, int64_t x_head_stride, void *out, int64_t out_token_stride,
                 int64_t out_head_stride, int transpose, void *stream) {
  NVFP4_TRY(check_dtype(dtype));
  if (head_dim < 8 || head_dim > 1024 || head_dim % 8) return NVFP4_ERR_SHAPE;
  NVFP4_TRY(check_rotary(rotary, head_dim, 4));
  if (tokens < 0 || tokens > INT32_MAX || heads < 0 || heads > 65535) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || heads == 0) return NVFP4_OK;
  if (!x || !out) return NVFP4_ERR_NULL;
  Turn turn;
  NVFP4_TRY(check_positions(rotary, positions, position_stride, tokens, &turn));
  NVFP4_TRY(check_rows(x, dtype, tokens, heads, x_token_stride, x_head_stride));
  NVFP4_TRY(check_out(out, dtype, tokens, heads, head_dim, out_token_stride, out_head_stride));
  const hipStream_t st = as_stream(stream);
  if (debug_checks_enabled())
    debug_check_finite_rows(x, dtype, tokens, heads, head_dim, x_token_stride, x_head_stride, st);
  return launch_rotate(turn, rotary->adjacent != 0, transpose != 0, {x, x_token_stride, x_head_stride},
                       {out, out_token_stride, out_head_stride}, dtype, tokens, heads, head_dim, st);
}

int nvfp4_kv_append(const nvfp4_kv_cache *cache, const nvfp4_rotary *rotary, const int64_t *positions,
                    int64_t position_stride, const void *q, const void *k, const void *v, int dtype,
                    int64_t tokens, int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                    int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                    int64_t v_head_stride, void *q_out, int64_t q_out_token_stride,
                    int64_t q_out_head_stride, const int64_t *slots, void *stream) {
  NVFP4_TRY(check_dtype(dtype));
  NVFP4_TRY(check_cache(cache, 1024));
  NVFP4_TRY(check_rotary(rotary, cache->head_dim, 8));
  if (tokens < 0 || tokens > INT32_MAX || heads < 0 || heads > 65535) return NVFP4_ERR_SHAPE;
  const int64_t kv_heads = cache->pages ? cache->kv_heads : 0;
  if (tokens == 0 || (kv_heads == 0 && heads == 0)) return NVFP4_OK;
  if ((kv_heads && (!k || !v || !slots)) || (heads && (!q || !q_out))) return NVFP4_ERR_NULL;
  Turn turn;
  NVFP4_TRY(check_positions(rotary, positions, position_stride, tokens, &turn));
  if (kv_heads) {
    if (!aligned(slots, 8)) return NVFP4_ERR_ALIGN;
    NVFP4_TRY(check_rows(k, dtype, tokens, kv_heads, k_token_stride, k_head_stride));
    NVFP4_TRY(check_rows(v, dtype, tokens, kv_heads, v_token_stride, v_head_stride));
  }
  if (heads) {
    NVFP4_TRY(check_rows(q, dtype, tokens, heads, q_token_stride, q_head_stride));
    NVFP4_TRY(check_out(q_out, dtype, tokens, heads, cache->head_dim, q_out_token_stride, q_out_head_stride));
  }
  const hipStream_t st = as_stream(stream);
  if (debug_checks_enabled()) {
    const int64_t hd = cache->head_dim;
    if (kv_heads) {
      debug_check_finite_rows(k, dtype, tokens, kv_heads, hd, k_token_stride, k_head_stride, st);
      debug_check_finite_rows(v, dtype, tokens, kv_heads, hd, v_token_stride, v_head_stride, st);
      debug_check_scale(cache->S_k, kv_heads, st);
      debug_check_scale(cache->S_v, kv_heads, st);
    }
    if (heads) debug_check_finite_rows(q, dtype, tokens, heads, hd, q_token_stride, q_head_stride, st);
  }
  const RowSpan qs = {q, q_token_stride, q_head_stride}, qo = {q_out, q_out_token_stride, q_out_head_stride};
  if (!kv_heads)
    return launch_rotate(turn, rotary->adjacent != 0, false, qs, qo, dtype, tokens, heads, cache->head_dim, st);
  return launch_kv_append(*cache, turn, rotary->adjacent != 0, qs, qo, {k, k_token_stride, k_head_stride},
                          {v, v_token_stride, v_head_stride}, dtype, tokens, heads, slots, st);
}

}  // extern "C"
