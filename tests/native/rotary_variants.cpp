// The split of a rotation or an append and how its rows are stored, for Python tests.
#include <initializer_list>

#include "../../scale_search_weights_amd/csrc/nvfp4_rotary_plan.h"

using namespace nvfp4;

// c: bf16, tokens, heads, head_dim, pairs. out: channels of a piece, tokens of a workgroup, units, heads and
// groups of the rows, stored past the caches
extern "C" void rotary_turn(const int64_t *c, int64_t *out) {
  const RotatePlan p = rotate_plan(c[0] != 0, c[1], c[2], c[3], (int)c[4]);
  out[0] = p.v, out[1] = p.tokens, out[2] = p.rows.units, out[3] = p.rows.heads, out[4] = p.rows.groups;
  out[5] = streams(c[0] != 0, c[1], c[2], c[3]);
}

// c: bf16, tokens, heads, key/value heads, head_dim, pairs. out: tokens of a workgroup, units, heads and groups of
// the key/value rows, of the query rows, queries stored past the caches
extern "C" void rotary_append(const int64_t *c, int64_t *out) {
  const AppendPlan p = append_plan(c[0] != 0, c[1], c[2], c[3], c[4], (int)c[5]);
  *out++ = p.tokens;
  for (const RowPlan &r : {p.kv, p.q}) *out++ = r.units, *out++ = r.heads, *out++ = r.groups;
  *out = streams(c[0] != 0, c[1], c[2], c[4]);
}

// the quotients of 0 .. 2^16 - 1 by d
extern "C" void rotary_quotients(int d, int *out) {
  const Div by(d);
  for (int n = 0; n < 1 << 16; ++n) out[n] = by.of(n);
}
