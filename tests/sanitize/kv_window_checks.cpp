// Host code of the rotation, the append and windowed attention under sanitizers: bad, extreme and empty
// arguments. Nothing is launched: every call is refused or has nothing to do.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/nvfp4_kv.h"

static int failures = 0;
#define EXPECT(expr, want)                                                            \
  do {                                                                                \
    const long long got_ = (long long)(expr);                                         \
    if (got_ != (long long)(want)) {                                                  \
      printf("line %d: %s = %lld, expected %lld\n", __LINE__, #expr, got_, (long long)(want)); \
      ++failures;                                                                     \
    }                                                                                 \
  } while (0)

int main() {
  uint8_t *F = reinterpret_cast<uint8_t *>(0x7F0000000000ull);  // never dereferenced
  float *S = reinterpret_cast<float *>(F);
  const int64_t *slots = reinterpret_cast<int64_t *>(F), *pos = slots;
  const int32_t *ids = reinterpret_cast<int32_t *>(F);
  const double *freq = reinterpret_cast<double *>(F);
  const int64_t big[] = {INT64_MIN, -1, 0, 1, 8, 16, 64, 128, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 2, INT64_MAX};

  // every size of rotary and cache at its extremes; a call that passes the checks has no tokens
  for (int64_t pairs : big)
    for (int64_t axes : big) {
      nvfp4_rotary r = {freq, ids, pairs, axes, 1.0, 1};
      for (int64_t hd : big) {
        nvfp4_rotate(&r, pos, 0, F, 1, 0, 4, hd, 0, 0, F, 0, 0, 0, nullptr);
        nvfp4_rotate(&r, pos, axes, F, 0, 4, 0, hd, pairs, axes, F, pairs, axes, 1, nullptr);
        for (int64_t pages : big) {
          nvfp4_kv_cache c = {F, F, F, F, S, S, pages, 16, 2, hd};
          nvfp4_kv_append(&c, &r, pos, 0, F, F, F, 1, 0, 4, 0, 0, 0, 0, 0, 0, F, 0, 0, slots, nullptr);
        }
      }
    }
  nvfp4_rotary r = {freq, nullptr, 32, 1, 1.0, 0};
  nvfp4_kv_cache c = {F, F, F, F, S, S, 8, 16, 2, 64};
  for (int64_t a : big)
    for (int64_t b : big) {
      nvfp4_rotate(&r, nullptr, a, F, 1, b, 4, 64, a, b, F, b, a, 0, nullptr);              // never valid: no positions
      nvfp4_rotate(&r, pos, a, F + 8, 0, 4, b, 64, a, b, F, b, a, 0, nullptr);              // or not aligned
      nvfp4_kv_append(&c, &r, pos, a, nullptr, nullptr, F, 1, a, 0, b, b, a, b, a, b, nullptr, a, b, slots, nullptr);
      nvfp4_kv_append(&c, &r, pos, b, F, F, F + 8, 0, 4, a, b, a, a, b, a, b, F, b, a, slots, nullptr);
      for (int64_t d : big) {
        // a NULL query: whatever passes the sizes is refused before a launch
        nvfp4_kv_window_attention(&c, nullptr, 1, a, 4, b, d, 2, nullptr, b, ids, d, ids, a, b, d, 1.0f, F, nullptr, F,
                                  SIZE_MAX, nullptr);
        nvfp4_kv_window_attention_workspace_size(&c, 1, a, 4, b, d, 4096, 64, 4);
        nvfp4_kv_window_attention_workspace_size(&c, 0, 16, 4, 16, 1, a, b, d);
        nvfp4_kv_window_attention_workspace_size(&c, 0, 16, a, 16, 1, b, d, a);
        nvfp4_kv_window_attention_workspace_size(&c, 1, 4096, 64, 1, 4096, a, b, d);
        nvfp4_kv_window_attention_workspace_size(&c, 0, 4096, 64, 2, 4096, a, b, d);
      }
    }
  // offsets that overflow, outputs on top of each other
  EXPECT(nvfp4_rotate(&r, pos, 0, F, 1, INT32_MAX, 4, 64, INT64_MAX / 2, 64, F, 256, 64, 0, nullptr), NVFP4_ERR_SHAPE);
  EXPECT(nvfp4_rotate(&r, pos, 0, F, 1, INT32_MAX, 4, 64, 256, 64, F, 64, 64, 0, nullptr), NVFP4_ERR_SHAPE);
  EXPECT(nvfp4_rotate(&r, pos, INT64_MAX, F, 1, 4, 4, 64, 256, 64, F, 256, 64, 0, nullptr), NVFP4_ERR_SHAPE);
  r.factor = NAN;
  EXPECT(nvfp4_rotate(&r, pos, 0, F, 1, 4, 4, 64, 256, 64, F, 256, 64, 0, nullptr), NVFP4_ERR_ARG);
  EXPECT(nvfp4_kv_append(nullptr, &r, pos, 0, F, F, F, 1, 4, 4, 256, 64, 128, 64, 128, 64, F, 256, 64, slots, nullptr),
         NVFP4_ERR_NULL);
  EXPECT(nvfp4_kv_window_attention(&c, F, 1, 2, 4, 256, 64, 2, nullptr, 1, ids, 256, ids, 4096, 1 << 30, 1 << 30, 1.0f, F,
                                   nullptr, nullptr, 0, nullptr),
         NVFP4_ERR_WORKSPACE);
  if (failures) return 1;
  printf("kv window checks passed\n");
  return 0;
}
