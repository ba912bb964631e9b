// C-ABI entry points of windowed attention over the key/value cache (declared in include/nvfp4_kv.h).
#include "nvfp4_kv_checks.h"
#include "nvfp4_kv_window_plan.h"

using namespace nvfp4;

namespace {

int check_window(int64_t window, int64_t sinks) {
  return window < 1 || window > (1 << 30) || sinks < 0 || sinks > (1 << 30) ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

}  // namespace

extern "C" {

size_t nvfp4_kv_window_attention_workspace_size(const nvfp4_kv_cache *cache, int dtype, int64_t tokens,
                                                int64_t heads, int64_t batch, int64_t max_q,
                                                int64_t max_kv, int64_t window, int64_t sinks) {
  KvAttention a;
  if (check_attention(cache, dtype, tokens, heads, batch, max_q, max_kv, 0, &a) != NVFP4_OK) return 0;
  if (check_window(window, sinks) != NVFP4_OK || nothing(a)) return 0;
  const WindowPlan w = window_plan_of(a, window, sinks);
  return kv_attention_fits(a, w.plan) ? kv_attention_workspace_size(a, w.plan) : 0;
}

int nvfp4_kv_window_attention(const nvfp4_kv_cache *cache, const void *q, int dtype, int64_t tokens,
                              int64_t heads, int64_t q_token_stride, int64_t q_head_stride, int64_t batch,
                              const int32_t *q_offsets, int64_t max_q, const int32_t *block_table,
                              int64_t table_width, const int32_t *kv_lens, int64_t max_kv,
                              int64_t window, int64_t sinks, float scale, void *out, float *lse,
                              void *workspace, size_t workspace_bytes, void *stream) {
  KvAttention a;
  NVFP4_TRY(check_attention(cache, dtype, tokens, heads, batch, max_q, max_kv, 0, &a));
  NVFP4_TRY(check_window(window, sinks));
  NVFP4_TRY(check_attention_call(&a, q, q_token_stride, q_head_stride, q_offsets, block_table, table_width,
                                 kv_lens, nullptr, scale, out, lse,
                                 [&] { return kv_attention_fits(a, window_plan_of(a, window, sinks).plan); }));
  if (nothing(a)) return NVFP4_OK;
  const Plan plan = window_plan_of(a, window, sinks).plan;
  NVFP4_TRY(check_workspace(kv_attention_workspace_size(a, plan), workspace, workspace_bytes));
  const hipStream_t st = as_stream(stream);
  debug_check_attention(a, st);
  a.causal = 1, a.workspace = workspace;
  return launch_kv_window_attention(a, window, sinks, st);
}

}  // extern "C"
