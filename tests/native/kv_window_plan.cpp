// The host plan of windowed attention for Python tests: what it chose, and every launch.
#include <initializer_list>

#include "../../scale_search_weights_amd/csrc/nvfp4_kv_window_plan.h"

using namespace nvfp4;

static KvAttention call(const nvfp4_kv_cache *c, const int64_t *s) {
  KvAttention a = {};
  a.cache = c, a.dtype = (int)s[0], a.tokens = s[1], a.heads = s[2], a.batch = s[3], a.max_q = s[4], a.max_kv = s[5];
  return a;
}
static nvfp4_kv_cache cache_of(const int64_t *s) {
  nvfp4_kv_cache c = {};
  c.pages = 1, c.page_size = 16, c.kv_heads = s[8], c.head_dim = s[9];
  return c;
}

// s: dtype, tokens, heads, batch, max_q, max_kv, window, sinks, kv_heads, head_dim.
// out: nt, waves, tile, row_tiles, slots, pieces, direct, workspace bytes
extern "C" int kv_window_plan(const int64_t *s, int64_t *out) {
  const nvfp4_kv_cache c = cache_of(s);
  const KvAttention a = call(&c, s);
  const WindowPlan w = window_plan_of(a, s[6], s[7]);
  const Part &r = w.plan.own;
  for (int64_t x : {(int64_t)r.nt, (int64_t)r.waves, (int64_t)r.tile, (int64_t)r.row_tiles, (int64_t)r.slots,
                    (int64_t)w.pieces, (int64_t)w.plan.direct, (int64_t)kv_attention_workspace_size(a, w.plan)})
    *out++ = x;
  return kv_attention_fits(a, w.plan);
}

// out: for every launch list, first slot, workgroups, threads of a workgroup; returns their number
extern "C" int kv_window_launches(const int64_t *s, int64_t *out, int most) {
  const nvfp4_kv_cache c = cache_of(s);
  const KvAttention a = call(&c, s);
  int n = 0;
  each_launch(a, window_plan_of(a, s[6], s[7]).plan, [&](const Launch &l) {
    if (n < most) out[4 * n] = l.list, out[4 * n + 1] = l.slot0, out[4 * n + 2] = l.grid, out[4 * n + 3] = l.threads;
    ++n;
  });
  return n;
}
