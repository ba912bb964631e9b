// The split of rotation and append into workgroups, for Python tests.
#include <initializer_list>

#include "../../scale_search_weights_amd/csrc/nvfp4_rotary_plan.h"

using namespace nvfp4;

// out: channels of a piece, tokens, then units, heads and groups of the rows
extern "C" void rotary_rotate_plan(int bf16, int64_t tokens, int64_t heads, int64_t hd, int pairs, int64_t *out) {
  const RotatePlan p = rotate_plan(bf16 != 0, tokens, heads, hd, pairs);
  out[0] = p.v, out[1] = p.tokens, out[2] = p.rows.units, out[3] = p.rows.heads, out[4] = p.rows.groups;
}

// out: tokens, then units, heads and groups of the key/value rows and of the query rows
extern "C" void rotary_append_plan(int bf16, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t hd, int pairs,
                                   int64_t *out) {
  const AppendPlan p = append_plan(bf16 != 0, tokens, heads, kv_heads, hd, pairs);
  *out++ = p.tokens;
  for (const RowPlan &r : {p.kv, p.q}) *out++ = r.units, *out++ = r.heads, *out++ = r.groups;
}

// out: chunks and first token of every launch; returns their number
extern "C" int64_t rotary_launches(int64_t tokens, int n, int64_t groups, int64_t *out, int64_t most) {
  int64_t k = 0;
  each_chunks(tokens, n, groups, [&](int64_t chunks, int64_t t0) {
    if (k < most) out[2 * k] = chunks, out[2 * k + 1] = t0;
    ++k;
  });
  return k;
}
