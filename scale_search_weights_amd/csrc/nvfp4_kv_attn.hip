// Attention over the key/value cache: the launches of a call (kernels: nvfp4_kv_attn_kernels.h).
#include "nvfp4_kv_attn_kernels.h"

namespace nvfp4 {

namespace {

template <int HD, bool F32, bool EXACT>
void launch_rows(const Attn &p, const Part &r, unsigned grid, hipStream_t st) {
  const dim3 g(grid), b(64 * r.waves);
  if (r.tile) {
    if (r.waves == 8) {
      if constexpr (HD <= 128 || !F32)
        hipLaunchKernelGGL((k_kv_attn_tile<HD, F32 || (HD > 128) ? 1 : 2, F32, EXACT, 8>), g, b, 0, st, p);
    } else if (r.nt == 1) {
      hipLaunchKernelGGL((k_kv_attn_tile<HD, 1, F32, EXACT, 4>), g, b, 0, st, p);
    } else if constexpr (HD <= 128 && !F32) {
      hipLaunchKernelGGL((k_kv_attn_tile<HD, 2, F32, EXACT, 4>), g, b, 0, st, p);
    }
  } else if (r.waves > 4) {
    if constexpr (HD <= 128 && !F32) {
      if (r.waves == 16) hipLaunchKernelGGL((k_kv_attn_rows<HD, 1, F32, EXACT, 16>), g, b, 0, st, p);
      else hipLaunchKernelGGL((k_kv_attn_rows<HD, 1, F32, EXACT, 8>), g, b, 0, st, p);
    }
  } else if (r.nt == 1) {
    hipLaunchKernelGGL((k_kv_attn_rows<HD, 1, F32, EXACT, 4>), g, b, 0, st, p);
  } else if constexpr (HD <= 128 || !F32) {
    hipLaunchKernelGGL((k_kv_attn_rows<HD, 2, F32, EXACT, 4>), g, b, 0, st, p);
  }
}

template <int HD, bool F32>
void launch_exact(const Attn &p, const Part &r, unsigned grid, hipStream_t st) {
  if (p.hd == HD) launch_rows<HD, F32, true>(p, r, grid, st);
  else launch_rows<HD, F32, false>(p, r, grid, st);
}

template <bool F32>
void launch_hd(const Attn &p, const Part &r, unsigned grid, hipStream_t st) {
  if (p.hd <= 64) launch_exact<64, F32>(p, r, grid, st);
  else if (p.hd <= 128) launch_exact<128, F32>(p, r, grid, st);
  else launch_exact<256, F32>(p, r, grid, st);
}

template <int HD>
void launch_join(const Join &p, bool f32, const dim3 &g, hipStream_t st) {
  if (f32) hipLaunchKernelGGL((k_kv_attn_join<HD, true>), g, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_kv_attn_join<HD, false>), g, dim3(256), 0, st, p);
}

}  // namespace

int launch_kv_attention(const KvAttention &a, hipStream_t st) {
  const Plan plan = plan_of(a);
  const nvfp4_kv_cache &c = *a.cache;
  const int64_t n_pre = prefix_rows(a, plan), n_own = own_rows(a, plan);
  Attn p = {};
  p.kc = c.k_codes, p.ks = c.k_scales, p.vc = c.v_codes, p.vs = c.v_scales;
  p.S_k = c.S_k, p.S_v = c.S_v;
  p.q = a.q, p.q_ts = a.q_ts, p.q_hs = a.q_hs, p.q_offsets = a.q_offsets, p.kv_lens = a.kv_lens;
  p.tokens = (int)a.tokens, p.heads = (int)a.heads, p.kv_heads = (int)c.kv_heads;
  p.group = (int)(a.heads / c.kv_heads), p.hd = (int)c.head_dim, p.batch = (int)a.batch;
  p.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  p.pages = (int)c.pages, p.max_q = (int)a.max_q, p.scale = a.scale, p.direct = plan.direct;
  p.out = a.out, p.lse = a.lse;
  if (plan.lead) p.lead = a.prefix_pages, p.lead_len = (int)a.prefix_len;
  float *opart = static_cast<float *>(a.workspace), *own = opart + n_pre * c.head_dim;
  float2 *ml = reinterpret_cast<float2 *>(own + n_own * c.head_dim), *ml_own = ml + n_pre;
  int2 *where = reinterpret_cast<int2 *>(ml_own + n_own);
  const bool f32 = a.dtype == NVFP4_DTYPE_F32;
  List lists[2] = {};
  const Part parts[2] = {plan.prefix, plan.own};
  List &x = lists[0], &y = lists[1];
  x.table = a.prefix_pages, x.max_len = (int)a.prefix_len, x.prefix = 1;
  x.piece = plan.prefix.piece, x.opart = opart, x.ml = ml;
  y.table = a.block_table, y.table_width = a.table_width, y.max_len = (int)a.max_kv;
  y.causal = a.causal, y.target = plan.own.target, y.joined = plan.prefix.slots > 0;
  y.opart = own, y.ml = ml_own, y.where = where, y.finish = plan.finish;
  for (int k = 0; k < 2; ++k)
    lists[k].row_tiles = parts[k].row_tiles, lists[k].slots = parts[k].slots;
  Join jn = {};
  jn.opart = opart, jn.opart_own = own, jn.ml = ml, jn.ml_own = ml_own;
  jn.S_v = c.S_v, jn.out = a.out, jn.lse = a.lse, jn.q_offsets = a.q_offsets, jn.kv_lens = a.kv_lens;
  jn.tokens = p.tokens, jn.heads = p.heads, jn.kv_heads = p.kv_heads, jn.group = p.group, jn.hd = p.hd;
  jn.max_q = p.max_q, jn.n_prefix = plan.prefix.slots, jn.per = join_per(a, plan);
  jn.where = plan.own.target > 0.0f ? where : nullptr;
  each_launch(a, plan, [&](const Launch &l) {
    if (l.list == 2) {
      const dim3 g((unsigned)l.grid, (unsigned)a.batch);
      if (p.hd <= 64) launch_join<64>(jn, f32, g, st);
      else if (p.hd <= 128) launch_join<128>(jn, f32, g, st);
      else launch_join<256>(jn, f32, g, st);
      return;
    }
    p.list[0] = lists[l.list], p.list[1] = lists[!l.list];
    p.first = (int)(l.both ? part_grid(a, plan.prefix) : l.grid), p.slot0 = l.slot0;
    if (f32) launch_hd<true>(p, parts[l.list], (unsigned)l.grid, st);
    else launch_hd<false>(p, parts[l.list], (unsigned)l.grid, st);
  });
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
