/*
 * libnvfp4, rotary positions — queries and keys turned by their positions, on AMD Instinct MI355X
 * (gfx950). nvfp4_kv.h's append turns keys by the same rule on their way into the cache.
 *
 * A row (one token, one head) has head_dim channels. Its first 2 * pairs are turned in pairs, the
 * others pass through. Pair i of token t turns by the angle theta = p * inv_freq[i], where p is
 * the token's position on the pair's axis, positions[axis[i]][t]: one axis for text, several (time,
 * height, width) for images and video. With c = factor cos(theta), s = factor sin(theta),
 *   y0 = x0 c - x1 s,   y1 = x1 c + x0 s,
 * and x0, x1 are channels i and i + pairs, or 2 i and 2 i + 1 if `adjacent` is non-zero.
 *
 * The angle is taken in 64 bits (with the product's rounding error), c and s are computed in 64
 * bits and rounded to fp32 once; the two products and their sum are rounded to fp32 each, and a
 * bf16 result from that. So a result is the same whatever the call's other tokens and heads are.
 * Angles are good to 2^-50 for |theta| up to 2^31 and |p| up to 2^53; the turn by a larger or not
 * finite angle is unspecified.
 *
 * Conventions (pointers, streams, status codes) are those of nvfp4.h. Rows may be strided as in
 * nvfp4_kv.h: the last dimension is contiguous, strides of the token and the head dimension are in
 * elements, every row starts at a multiple of 16 bytes.
 */
#ifndef NVFP4_ROTARY_H
#define NVFP4_ROTARY_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* inv_freq: device [pairs], 8-byte aligned; axis: device [pairs], 4-byte aligned, or NULL: all on
 * axis 0. An axis outside [0, axes) is read as position 0. pairs is a multiple of 4 up to 512, axes
 * 1 to 16, factor finite. The library reads the struct during the call and keeps nothing of it. */
typedef struct nvfp4_rotary {
  const double *inv_freq;
  const int32_t *axis;
  int64_t pairs, axes;
  double factor;
  int adjacent;
} nvfp4_rotary;

/*
 * out[t][h] = x[t][h] turned by the positions of token t; with `transpose` non-zero by the
 * transposed matrix (the backward pass: s -> -s, which for factor 1 turns back). x, out:
 * [tokens][heads][head_dim] of `dtype`, strided; head_dim is a multiple of 8 up to 1024, at least
 * 2 * pairs. positions: int64 [axes][tokens], axis a at positions + a * position_stride (which may
 * be 0). out may be x itself, with the same strides; otherwise they must not overlap, and no row of
 * out another.
 */
NVFP4_API int nvfp4_rotate(const nvfp4_rotary *rotary, const int64_t *positions,
                           int64_t position_stride, const void *x, int dtype, int64_t tokens,
                           int64_t heads, int64_t head_dim, int64_t x_token_stride,
                           int64_t x_head_stride, void *out, int64_t out_token_stride,
                           int64_t out_head_stride, int transpose, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ROTARY_H */
