// Attention over the key/value cache: the join of partial sums and the launches of a call (kernels:
// nvfp4_kv_attn_kernels.h).
#include "nvfp4_kv_attn_kernels.h"

namespace nvfp4 {

template <int HD, bool F32>
__global__ void __launch_bounds__(256) k_kv_attn_join(Join p) {
  constexpr int LANES = HD / 4, GROUPS = 256 / LANES;
  __shared__ f4 so[GROUPS][LANES];
  __shared__ float sm_m[GROUPS], sm_l[GROUPS];
  const int b = blockIdx.y;
  const int g = threadIdx.x / LANES, c = threadIdx.x % LANES, first = g & -p.per;
  const int r = blockIdx.x * (GROUPS / p.per) + g / p.per;  // of the sequence: token, head
  const int i = r / p.heads, head = r - i * p.heads;
  const Span sp = rows_of(p.q_offsets, b, p.max_q, p.tokens);
  const int lo = sp.lo, hi = sp.hi;
  int own0 = 0, n = p.n_prefix;
  if (p.where) {
    if (p.kv_lens[b] > 0) {
      const int2 x = p.where[b];
      if (x.y == 1 && n == 0) return;  // written by its only piece
      own0 = x.x, n += x.y;
    }
  } else if (p.kv_lens) {
    n += 1;
  }
  const bool here = lo + i < hi;
  const int h = head / p.group, gr = head - h * p.group;
  const float S_v = p.S_v[h];
  const int64_t rows = (int64_t)p.tokens * p.group, own_rows = (int64_t)p.max_q * p.group;
  const int64_t at = h * rows + (int64_t)(lo + i) * p.group + gr;  // in a slot of all tokens
  const int64_t own_at =
      p.where ? ((int64_t)own0 * p.kv_heads + h) * own_rows + (int64_t)i * p.group + gr : at;
  const int64_t step = rows * p.kv_heads, own_step = own_rows * p.kv_heads;
  float M = -INFINITY, L = 0.0f;
  f4 y = {0, 0, 0, 0};
  const bool in = 4 * c < p.hd;
  if (!here) n = 0;
#pragma unroll 4
  for (int k = g - first; k < n; k += p.per) {
    const bool pre = k < p.n_prefix;
    const int64_t row = pre ? at + k * step : own_at + (k - p.n_prefix) * own_step;
    const float2 ml = (pre ? p.ml : p.ml_own)[row];
    f4 o = {0, 0, 0, 0};
    if (in) o = *reinterpret_cast<const f4 *>((pre ? p.opart : p.opart_own) + row * p.hd + 4 * c);
    if (ml.y != 0.0f) {  // else the piece holds nothing the row sees
      const float to = fmaxf(M, ml.x);
      const float a = __builtin_amdgcn_exp2f(M - to), e = __builtin_amdgcn_exp2f(ml.x - to);
      M = to;
      L = L * a + ml.y * e;
      y = y * a + o * e;
    }
  }
  if (c == 0) sm_m[g] = M, sm_l[g] = L;
  so[g][c] = y;
  __syncthreads();
  if (g != first || !here) return;
  for (int k = 1; k < p.per; ++k) M = fmaxf(M, sm_m[g + k]);
  L = 0.0f;
  y = (f4){0, 0, 0, 0};
  for (int k = 0; k < p.per; ++k) {
    if (sm_l[g + k] == 0.0f) continue;
    const float e = __builtin_amdgcn_exp2f(sm_m[g + k] - M);
    L += sm_l[g + k] * e;
    y += so[g + k][c] * e;
  }
  const int64_t to = (int64_t)(lo + i) * p.heads + head;
  if (in) store4<F32>(p.out, to * p.hd + 4 * c, y * out_factor(S_v, L));
  if (c == 0 && p.lse) p.lse[to] = row_lse(M, L);
}

namespace {

template <int HD>
void launch_join(const Join &p, bool f32, const dim3 &g, hipStream_t st) {
  if (f32) hipLaunchKernelGGL((k_kv_attn_join<HD, true>), g, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_kv_attn_join<HD, false>), g, dim3(256), 0, st, p);
}

}  // namespace

void launch_kv_join(const Join &p, bool f32, const dim3 &g, hipStream_t st) {
  if (p.hd <= 64) launch_join<64>(p, f32, g, st);
  else if (p.hd <= 128) launch_join<128>(p, f32, g, st);
  else launch_join<256>(p, f32, g, st);
}

int launch_kv_attention(const KvAttention &a, hipStream_t st) {
  const Plan plan = plan_of(a);
  const nvfp4_kv_cache &c = *a.cache;
  const int64_t n_pre = prefix_rows(a, plan), n_own = own_rows(a, plan);
  Attn p = attn_of(a);
  p.direct = plan.direct;
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
  Join jn = join_of(p, plan.prefix.slots, join_per(a, plan));
  jn.opart = opart, jn.opart_own = own, jn.ml = ml, jn.ml_own = ml_own;
  jn.where = plan.own.target > 0.0f ? where : nullptr;
  each_launch(a, plan, [&](const Launch &l) {
    if (l.list == 2) {
      const dim3 g((unsigned)l.grid, (unsigned)a.batch);
      launch_kv_join(jn, f32, g, st);
      return;
    }
    p.list[0] = lists[l.list], p.list[1] = lists[!l.list];
    p.first = (int)(l.both ? part_grid(a, plan.prefix) : l.grid), p.slot0 = l.slot0;
    if (f32) launch_hd<true, false>(p, parts[l.list], (unsigned)l.grid, st);
    else launch_hd<false, false>(p, parts[l.list], (unsigned)l.grid, st);
  });
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
