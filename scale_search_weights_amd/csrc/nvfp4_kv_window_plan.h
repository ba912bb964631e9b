// How an attention call over a window and sinks is split into launches: host code without HIP.
//
// A row tile reads at most `span` tokens however long the context is: the sinks, the window of its first
// row and as many more as its other rows stand behind that one. Since the spans of a batch are much the
// same, its sequences are cut into the same number of pieces, and the host knows what a call costs.
#pragma once

#include "nvfp4_kv_plan.h"

namespace nvfp4 {

struct WindowPlan {
  Plan plan;  // own tokens only
  int pieces;
};

// Tokens that a tile of `rows` rows reads, in whole groups of 16 at the window's far end.
inline int64_t window_span(const KvAttention &a, int64_t window, int64_t sinks, int64_t rows) {
  const int64_t G = a.heads / a.cache->kv_heads, tokens = cdiv(rows, G) + 1;
  const int64_t span = cdiv(sinks, 16) * 16 + window + 15 + (tokens < a.max_q ? tokens : a.max_q);
  return span < a.max_kv ? span : a.max_kv;
}

// Up to 32 rows a (sequence, key/value head): k_kv_attn_rows. One piece where n workgroups and more hold a
// CU each or a cut saves less than its join costs, 6 us at 5 ns a token; else as many as give the CUs one,
// of 256 tokens (slower kernels 128) at least. Sixteen waves were never the best. us, eight key/value heads
// of 128, waves.pieces; n and span: 8, 512: 8.1 8.3, 4.1 8.5, 16.1 9.9. 8, 1024: 4.4 10.5, 8.1 10.8, 4.1 11.9.
// 8, 4096: 4.16 11.6, 8.8 12.4, 8.1 26.4. 64, 4096: 8.4 16.8, 4.8 17.1, 8.1 27.3. 128, 2048: 8.2 16.2, 8.1
// 16.9. 256, 1024: 8.1 12.4, 4.1 13.8, 8.2 16.6. 512, 1024: 4.1 18.8, 8.1 19.1, 4.2 23.5. 8, 128: 4.1 5.9, 8.1 6.3.
inline WindowPlan window_rows_plan(const KvAttention &a, int64_t window, int64_t sinks) {
  WindowPlan w = {};
  const bool wide = a.cache->head_dim > 128, f32 = a.dtype == NVFP4_DTYPE_F32;
  const int64_t rows = a.max_q * (a.heads / a.cache->kv_heads);
  Part &r = w.plan.own;
  r = rows_part(a, rows, rows <= 16 || (wide && f32) ? 1 : 2);
  const int64_t span = window_span(a, window, sinks, rows), n = a.batch * a.cache->kv_heads * r.row_tiles;
  const bool fast = r.nt == 1 && !wide && !f32;
  const int64_t most = span / (fast ? 256 : 128), fill = kCus / n, cut = fill < most ? fill : most;
  const int64_t slower = fast ? 1 : 2 * (1 + wide + f32);
  w.pieces = cut > 1 && span * (cut - 1) * slower >= 1200 * cut ? (int)cut : 1;
  if (fast && n <= kCus && span > (w.pieces > 1 ? 512 * cut : 256)) r.waves = 8;
  return w;
}

// What workgroups of k_kv_attn_tile take, us, with k of them for a CU: start + more k to begin and end, and for 64
// tokens `alone` and `beside` for each other one of up to `fit` that share the CU; what is beyond them
// takes turns. Fitted to 128 to 1024 workgroups on windows of 512 and 2048 tokens, heads of 64, 128 and 256. Measured
// again in short runs, which clock higher, the estimates are 1 to 30% high, by much the same for all kernels of a
// type and head, for heads of 80, 96 and 160 too; two stand out: fp32 heads of 256, 10 to 22% low (there is one tile
// to choose), and fp32 heads of 64 on four waves, up to 40% high where more than three share a CU.
struct TileCost {
  double start, more, alone, beside;
  int fit;
};
inline TileCost tile_cost(int nt, int waves, int64_t hd, bool f32) {
  if (hd > 128) return waves == 8 ? TileCost{7.0, 8.6, 2.5, 0.0, 1} : TileCost{5.0, 6.5, 2.3, 0.0, 1};
  const bool two = nt == 2 || f32;  // 16-row tiles, or products, of a wave
  if (hd > 64) {
    if (waves == 8) return {5.0, 10.0, 2.0, 0.0, 1};
    return two ? TileCost{8.0, 4.0, 1.75, 0.55, 2} : TileCost{5.0, 2.6, 1.45, 0.4, 2};
  }
  if (waves == 8) return f32 ? TileCost{6.0, 4.2, 1.4, 0.75, 2} : TileCost{3.0, 8.0, 1.4, 0.0, 1};
  return two ? TileCost{6.0, 2.2, 1.35, 0.38, 3} : TileCost{4.5, 1.4, 1.1, 0.27, 4};
}
inline double tile_time(const TileCost &c, double k, double steps) {
  const double turns = floor(k / c.fit), rest = k - turns * c.fit;
  const double step = turns * (c.alone + (c.fit - 1) * c.beside) + (rest > 0.0 ? c.alone + (rest - 1.0) * c.beside : 0.0);
  return c.start + c.more * k + steps * step;
}

// More rows: the tile and number of pieces with the least estimated time. Pieces cost 5 us of join and 0.3 us a
// MB of partial sums. Estimated and measured, eight key/value heads of 128, four query heads each: 2 x 2048
// queries, window 1024: 256 rows a tile 97, 92; 128 rows 108, 99; 64 rows 144, 141. 512 queries, window 1024:
// 64 rows whole 34, 30, in two pieces 39, 36. 8 x 64, window 512: 64 rows 21, 19; 256 rows 33, 30.
// Of 80 calls (eight sizes, heads of 64 to 256, both types) 72 take at most 2% more than the best of all tiles in
// one, two and four pieces, the others 6 to 20%: 100 and 512 queries, which more pieces would serve better.
inline WindowPlan window_tile_plan(const KvAttention &a, int64_t window, int64_t sinks) {
  WindowPlan best = {};
  double least = INFINITY;
  const bool wide = a.cache->head_dim > 128, f32 = a.dtype == NVFP4_DTYPE_F32;
  const int64_t G = a.heads / a.cache->kv_heads, rows = a.max_q * G, units = a.batch * a.cache->kv_heads;
  for (int kind = 0; kind < 3; ++kind) {
    const int nt = kind && !wide && !f32 ? 2 : 1, waves = kind == 2 ? 8 : 4;
    if ((kind == 1 && nt == 1) || (waves == 8 && wide && f32)) continue;
    const int64_t tile = 16 * nt * waves, row_tiles = cdiv(rows, tile);
    const int64_t span = window_span(a, window, sinks, tile < rows ? tile : rows);
    const TileCost c = tile_cost(nt, waves, a.cache->head_dim, f32);
    const int64_t blocks = cdiv(span > 0 ? span : 1, 128);
    for (int64_t per = blocks; per > 0; per = per > 16 ? per / 2 : per - 1) {  // blocks of 128 tokens a piece
      const int64_t pieces = cdiv(blocks, per);
      if (pieces > 1 && units * row_tiles * pieces > 4 * kCus) break;
      double us = tile_time(c, (double)cdiv(units * row_tiles * pieces, kCus), (double)(2 * per));
      if (pieces > 1) us += 5.0 + 0.3e-6 * (double)(a.batch * pieces * rows * a.cache->kv_heads * a.cache->head_dim * 4);
      if (us >= least) continue;
      least = us;
      Part &r = best.plan.own;
      r = Part{};
      r.tile = 1, r.nt = nt, r.waves = waves, r.row_tiles = (int)row_tiles;
      best.pieces = (int)pieces;
    }
  }
  return best;
}

inline WindowPlan window_plan_of(const KvAttention &a, int64_t window, int64_t sinks) {
  const int64_t rows = a.max_q * (a.heads / a.cache->kv_heads);
  WindowPlan w = rows <= 32 ? window_rows_plan(a, window, sinks) : window_tile_plan(a, window, sinks);
  Plan &p = w.plan;
  p.own.slots = (int)(a.batch * w.pieces);
  p.own.target = w.pieces > 1 ? (float)p.own.slots : 0.0f;
  p.direct = w.pieces == 1;
  return w;
}

}  // namespace nvfp4
