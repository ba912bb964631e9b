// Attention over a window of the cached tokens, and over the first ones (sinks): a row at position P
// sees the tokens t <= P with t > P - window or t < sinks.
//
// The kernels are those of full attention (nvfp4_kv_attn_kernels.h) over a token list with a gap: a
// row tile reads the sinks' groups of 16 tokens, then those that its rows' windows cover, so the work
// is that of sinks + window tokens however long the context is.
#include "nvfp4_kv_attn_kernels.h"
#include "nvfp4_kv_window_plan.h"

namespace nvfp4 {

int launch_kv_window_attention(const KvAttention &a, int64_t window, int64_t sinks, hipStream_t st) {
  const WindowPlan w = window_plan_of(a, window, sinks);
  const Plan &plan = w.plan;
  Attn p = attn_of(a);
  p.direct = plan.direct, p.pieces = w.pieces;
  p.window = (int)window, p.sinks = (int)sinks;
  const int64_t n = own_rows(a, plan);
  float *opart = static_cast<float *>(a.workspace);
  float2 *ml = reinterpret_cast<float2 *>(opart + n * p.hd);
  const bool f32 = a.dtype == NVFP4_DTYPE_F32;
  List &y = p.list[0];
  y.table = a.block_table, y.table_width = a.table_width, y.max_len = (int)a.max_kv, y.causal = 1;
  y.target = plan.own.target, y.row_tiles = plan.own.row_tiles, y.slots = plan.own.slots;
  y.opart = opart, y.ml = ml, y.where = reinterpret_cast<int2 *>(ml + n);
  Join jn = join_of(p, 0, join_per(a, plan));
  jn.opart_own = opart, jn.ml_own = ml, jn.where = y.where;
  each_launch(a, plan, [&](const Launch &l) {
    if (l.list == 2) {
      launch_kv_join(jn, f32, dim3((unsigned)l.grid, (unsigned)a.batch), st);
      return;
    }
    p.first = (int)l.grid, p.slot0 = l.slot0;
    if (f32) launch_hd<true, true>(p, plan.own, (unsigned)l.grid, st);
    else launch_hd<false, true>(p, plan.own, (unsigned)l.grid, st);
  });
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
