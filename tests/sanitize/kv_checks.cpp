// Host code of the key/value cache's entry points under sanitizers: bad, extreme and empty
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
  const int64_t *slots = reinterpret_cast<int64_t *>(F);
  const int32_t *ids = reinterpret_cast<int32_t *>(F);
  const int64_t big[] = {INT64_MIN, -1, 0, 1, 15, 16, 64, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 2, INT64_MAX};

  // every size of the cache at its extremes; a call that passes the checks has no tokens
  for (int64_t pages : big)
    for (int64_t ps : big)
      for (int64_t heads : big)
        for (int64_t hd : big) {
          nvfp4_kv_cache c = {F, F, F, F, S, S, pages, ps, heads, hd};
          nvfp4_kv_write(&c, F, F, 1, 0, 0, 0, 0, 0, slots, nullptr);
          nvfp4_kv_read(&c, slots, 0, F, F, 1, nullptr);
          nvfp4_kv_attention_workspace_size(&c, 1, 2, heads, 2, 1, 4096, 0);
          nvfp4_kv_attention(&c, F, 1, 0, heads, 64, 64, 2, nullptr, 0, ids, 4, ids, 64, nullptr, 0, 1.0f, 1, F,
                             nullptr, nullptr, 0, nullptr);
        }

  nvfp4_kv_cache c = {F, F, F, F, S, S, 8, 16, 2, 64};
  for (int64_t a : big)
    for (int64_t b : big) {
      nvfp4_kv_write(&c, nullptr, F, 1, a, b, b, b, b, slots, nullptr);         // never valid: k missing
      nvfp4_kv_write(&c, F + 8, F, 0, a, b, a, b, a, slots, nullptr);           // or not aligned
      nvfp4_kv_read(&c, nullptr, a, F, F, 0, nullptr);
      for (int64_t d : big) {
        nvfp4_kv_attention_workspace_size(&c, 1, a, 4, b, d, 4096, 64);
        nvfp4_kv_attention_workspace_size(&c, 0, 16, 4, 16, 1, a, b);
        nvfp4_kv_attention_workspace_size(&c, 0, 16, a, 16, 1, b, d);
        nvfp4_kv_attention(&c, nullptr, 1, a, 4, b, d, 2, nullptr, b, ids, d, ids, a, ids, d, 1.0f, 1, F, nullptr, F,
                           SIZE_MAX, nullptr);                                  // q missing
      }
    }
  // strides whose byte offsets overflow
  EXPECT(nvfp4_kv_write(&c, F, F, 1, INT32_MAX, INT64_MAX / 2, 64, 64, 64, slots, nullptr), NVFP4_ERR_SHAPE);
  EXPECT(nvfp4_kv_write(&c, F, F, 1, 4, 64, INT64_MAX - 7, 64, 64, slots, nullptr), NVFP4_ERR_SHAPE);
  EXPECT(nvfp4_kv_attention(&c, F, 1, 2, 4, 256, 64, 2, nullptr, 1, ids, 256, ids, 4096, nullptr, 0, NAN, 1, F,
                            nullptr, F, SIZE_MAX, nullptr), NVFP4_ERR_ARG);
  EXPECT(nvfp4_kv_attention(&c, F, 1, 2, 4, 256, 64, 2, nullptr, 1, ids, 256, ids, 4096, nullptr, 0, 1.0f, 1, F,
                            nullptr, F, 0, nullptr), NVFP4_ERR_WORKSPACE);
  EXPECT(nvfp4_kv_attention(&c, F, 1, 2, 4, 256, 64, 2, nullptr, 1, ids, INT64_MAX, ids, 4096, nullptr, 0, 1.0f, 1,
                            F, nullptr, F, SIZE_MAX, nullptr), NVFP4_ERR_SHAPE);
  EXPECT(nvfp4_kv_write(nullptr, F, F, 1, 4, 64, 64, 64, 64, slots, nullptr), NVFP4_ERR_NULL);
  if (failures) return 1;
  printf("kv checks passed\n");
  return 0;
}
