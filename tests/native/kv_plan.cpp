// The attention's host plan for Python tests: what it chose, and every launch.
#include <initializer_list>

#include "../../scale_search_weights_amd/csrc/nvfp4_kv_plan.h"

using namespace nvfp4;

static KvAttention call(const nvfp4_kv_cache *c, const int64_t *s) {
  KvAttention a = {};
  a.cache = c, a.dtype = (int)s[0], a.tokens = s[1], a.heads = s[2], a.batch = s[3], a.max_q = s[4];
  a.max_kv = s[5], a.prefix_len = s[6];
  return a;
}

// s: dtype, tokens, heads, batch, max_q, max_kv, prefix_len, kv_heads, head_dim.
// out: nt, waves, tile, row_tiles, slots of the prefix, of the own tokens; cut, direct, finish, lead
extern "C" int kv_plan(const int64_t *s, int64_t *out) {
  nvfp4_kv_cache c = {};
  c.pages = 1, c.page_size = 16, c.kv_heads = s[7], c.head_dim = s[8];
  const KvAttention a = call(&c, s);
  const Plan p = plan_of(a);
  for (const Part *r : {&p.prefix, &p.own}) {
    *out++ = r->nt, *out++ = r->waves, *out++ = r->tile, *out++ = r->row_tiles, *out++ = r->slots;
  }
  *out++ = p.own.target > 0.0f, *out++ = p.direct, *out++ = p.finish, *out++ = p.lead;
  return kv_attention_fits(a);
}

// out: for every launch list, first slot, workgroups, threads of a workgroup; returns their number
extern "C" int kv_launches(const int64_t *s, int64_t *out, int most) {
  nvfp4_kv_cache c = {};
  c.pages = 1, c.page_size = 16, c.kv_heads = s[7], c.head_dim = s[8];
  const KvAttention a = call(&c, s);
  int n = 0;
  each_launch(a, plan_of(a), [&](const Launch &l) {
    if (n < most) out[4 * n] = l.list, out[4 * n + 1] = l.slot0, out[4 * n + 2] = l.grid, out[4 * n + 3] = l.threads;
    ++n;
  });
  return n;
}
