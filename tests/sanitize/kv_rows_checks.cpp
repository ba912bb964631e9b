// A sequence's query rows from the offsets, at sizes where sums and products pass 32 bits (run under
// UndefinedBehaviorSanitizer).
#include <stdio.h>

#include <initializer_list>

#include "../../scale_search_weights_amd/csrc/nvfp4_kv_plan.h"

using nvfp4::rows_of;
using nvfp4::Span;

static int failures = 0;

// offsets as they are, each cut to [0, tokens] and to max_q rows, in 64 bits
static void expect(int64_t first, int64_t last, int b, int max_q, int tokens, bool given) {
  int32_t offsets[2] = {(int32_t)first, (int32_t)last};
  const Span s = rows_of(given ? offsets : nullptr, b, max_q, tokens);
  int64_t lo = given ? first : (int64_t)b * max_q, hi = given ? last : lo + max_q;
  lo = lo < 0 ? 0 : lo > tokens ? tokens : lo;
  hi = hi < lo ? lo : hi;
  if (hi > lo + max_q) hi = lo + max_q;
  if (hi > tokens) hi = tokens;
  if (s.lo != lo || s.hi != hi) {
    printf("b %d max_q %d tokens %d: rows %d..%d, expected %lld..%lld\n", b, max_q, tokens, s.lo, s.hi, (long long)lo,
           (long long)hi);
    ++failures;
  }
}

int main() {
  const int big = INT32_MAX - 1024;
  const int64_t ends[] = {INT32_MIN, -1, 0, 1, 7, 65535, big / 2 + 9, big - 1, big, INT32_MAX};
  const int sizes[] = {1, 2, 65535, 65537, big / 2 + 5, big};
  for (int64_t a : ends)
    for (int64_t e : ends)
      for (int tokens : sizes)
        for (int max_q : sizes)
          if (max_q <= tokens) expect(a, e, 0, max_q, tokens, true);
  // many sequences behind a loose max_q: their product is never needed
  static int32_t offsets[65537];
  for (int b = 0; b <= 65536; ++b) offsets[b] = b;
  for (int b : {0, 40000, 65534, 65535}) {
    const Span s = rows_of(offsets, b, 65536, 65536);
    if (s.lo != b || s.hi != b + 1) ++failures;
  }
  for (int b : {0, 1, 999}) expect(0, 0, b, 2000000, 2000000000, false);
  if (failures) return 1;
  printf("kv rows checks passed\n");
  return 0;
}
