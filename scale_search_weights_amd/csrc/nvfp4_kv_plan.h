// How an attention call over the key/value cache is split into launches: host code without HIP.
#pragma once

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/nvfp4_kv.h"

namespace nvfp4 {

#if defined(__HIPCC__)
#define NVFP4_HD __host__ __device__
#else
#define NVFP4_HD
#endif

// Rows lo .. hi - 1 of the call are those of sequence b. Nothing here passes 32 bits: without offsets
// batch * max_q is tokens, with them a loose max_q is cut to the rows that are left before it is added.
struct Span {
  int lo, hi;
};
inline NVFP4_HD Span rows_of(const int32_t *q_offsets, int b, int max_q, int tokens) {
  if (!q_offsets) return {b * max_q, (b + 1) * max_q};
  int lo = q_offsets[b], hi = q_offsets[b + 1];
  lo = lo < 0 ? 0 : lo > tokens ? tokens : lo;
  const int end = lo + (max_q < tokens - lo ? max_q : tokens - lo);
  return {lo, hi < lo ? lo : hi > end ? end : hi};
}

struct KvAttention {
  const nvfp4_kv_cache *cache;
  const void *q;
  int dtype;
  int64_t tokens, heads, q_ts, q_hs, batch;
  const int32_t *q_offsets;
  int64_t max_q;
  const int32_t *block_table;
  int64_t table_width;
  const int32_t *kv_lens;
  int64_t max_kv;
  const int32_t *prefix_pages;
  int64_t prefix_len;
  float scale;
  int causal;
  void *out;
  float *lse;
  void *workspace;
};

struct Part {      // one launch: the prefix or the sequences' own tokens
  int nt, waves;   // 16-row tiles of a wave; waves of a workgroup
  int tile;        // k_kv_attn_tile, not k_kv_attn_rows
  int row_tiles, slots, piece;
  int resident;    // workgroups that the chip holds at once
  float target;
};

struct Plan {
  Part prefix, own;
  int direct;  // no partial sums
  int finish;  // the own tokens' workgroups add the prefix's pieces: no join
  int lead;    // the own tokens' workgroups go over the prefix first: no pieces at all
};

constexpr int kCus = 256;  // compute units of the chip

// Tiles of many rows cut the contexts into pieces only where the chip holds this many times the
// workgroups that whole contexts make: a row's partial sums cost more than a workgroup's wait.
constexpr float kTileCut = 1.5f;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// k_kv_attn_rows with 16 NT rows a workgroup; workgroups a CU holds, by registers.
inline Part rows_part(const KvAttention &a, int64_t rows, int nt) {
  Part r = {};
  const bool wide = a.cache->head_dim > 128, f32 = a.dtype == NVFP4_DTYPE_F32;
  const int one = wide ? 2 : (f32 ? 3 : 4);
  r.nt = nt, r.waves = 4;
  r.resident = kCus * (nt == 1 ? one : (one + 1) / 2);
  r.row_tiles = (int)cdiv(rows, 16 * nt);
  return r;
}

// k_kv_attn_tile: workgroups a CU holds, by LDS (at HD 256 1 KiB a token, two stages).
// Tiles of 64 rows are taken where tiles of 256 rows and pieces of 128 tokens would give fewer than
// 512 workgroups (8 heads, 240 rows x 700 tokens 23 -> 17 us, 500 x 2500 34 -> 30), and for up to 2048
// own tokens where they give three quarters of the CUs a whole context and the larger tiles (one
// workgroup a CU) would have to be cut into pieces (2800 rows x 1000 tokens 51 -> 28 us, 1600 x 2000
// 54 -> 47). On longer contexts it goes either way (larger, smaller: 2000 rows x 2500 tokens 59, 52;
// 2 x 2000 x 2500 69, 72); elsewhere equal or slower.
inline Part tile_part(const KvAttention &a, int64_t rows, int64_t jobs, int64_t len, bool own) {
  Part r = {};
  const int64_t hd = a.cache->head_dim, n = jobs * a.cache->kv_heads;
  const bool wide = hd > 128, f32 = a.dtype == NVFP4_DTYPE_F32;
  const bool small = n * cdiv(rows, 256) * cdiv(len, 128) < 512 ||
                     (own && len <= 2048 && kTileCut * (float)(n * cdiv(rows, wide || f32 ? 128 : 256)) <= kCus &&
                      4 * n * cdiv(rows, 64) >= 3 * kCus);
  r.tile = 1;
  r.nt = wide || f32 || small || rows <= 64 ? 1 : 2;
  r.waves = small || rows <= 64 * r.nt || (wide && f32) ? 4 : 8;
  r.resident = kCus * (wide ? 1 : (hd > 64 || r.waves == 8 ? 8 / r.waves : 3));
  r.row_tiles = (int)cdiv(rows, 16 * r.nt * r.waves);
  return r;
}

// Rows a (sequence, key/value head): up to 32 to k_kv_attn_rows, whose waves work alone; more to
// k_kv_attn_tile, whose waves share what they dequantise.
inline Part plan_rows(const KvAttention &a, int64_t rows, int64_t jobs, int64_t len, bool own) {
  if (rows > 32) return tile_part(a, rows, jobs, len, own);
  const bool one = rows <= 16 || (a.cache->head_dim > 128 && a.dtype == NVFP4_DTYPE_F32);
  return rows_part(a, rows, one ? 1 : 2);
}

inline Plan plan_of(const KvAttention &a) {
  Plan p = {};
  const int64_t G = a.heads / a.cache->kv_heads, kvh = a.cache->kv_heads;
  const bool own = a.max_kv > 0 || a.prefix_len == 0;
  if (own) p.own = plan_rows(a, a.max_q * G, a.batch, a.max_kv, true);
  if (a.prefix_len > 0) {
    p.prefix = plan_rows(a, a.tokens * G, 1, a.prefix_len, false);
    // one launch for both lists where the prefix is so short that the own tokens' kernel does it
    // in one round of 128-token pieces
    if (own && !p.own.tile) {
      const Part r = rows_part(a, a.tokens * G, p.own.nt);
      if (r.row_tiles * kvh * cdiv(a.prefix_len, 128) <= r.resident) p.prefix = r;
    }
    Part &r = p.prefix;
    const int64_t units = kvh * r.row_tiles;
    const int64_t n = units < r.resident ? r.resident / units : 1;
    r.piece = (int)(cdiv(a.prefix_len, 128 * n) * 128);
    r.slots = (int)cdiv(a.prefix_len, r.piece);
  }
  if (own) {
    Part &r = p.own;
    const int64_t units = kvh * r.row_tiles;
    // pieces wanted: with the half piece that a sequence adds on average, as many as the chip
    // holds at once (64 sequences of 512 to 8192 tokens: 52 -> 48 us against not counting it)
    const float held = (float)r.resident / (float)units;
    const float target = fmaxf(held - 0.5f * (float)a.batch, 0.75f * held);
    r.slots = (int)a.batch;
    // Short contexts: one piece a sequence, with more waves the fewer the sequences, saves the
    // partial sums and the join (about 5 us); an iteration of such a workgroup costs 1 to 2 us
    // however little it reads, so the fewer workgroups there are to share the chip, the fewer
    // iterations it may take. Calls that are launched one by one need 12.7 us for two launches and
    // 9 for one, calls from a graph only the GPU's time; a context is whole while that is faster in
    // one way at little cost in the other. Cut and whole, us, one by one | from a graph, 8 key/value
    // heads of 128: 4 x 1000 tokens 12.7, 11.6 | 10.6, 11.7; 4 x 1500 12.6, 14.1 | 12.2, 14.1; from a
    // graph 10 x 1000 13.2, 12.0; 7 x 1200 13.4, 12.6; 7 x 1500 13.6, 13.9; 30 x 6000 43.0, 37.8. 20
    // heads of 64: 1 x 1500 12.7, 11.3 | 10.4, 11.1; 5 x 1500 13.1, 11.3 | 13.1, 11.4.
    bool whole = a.max_kv <= 128;
    if (!r.tile && r.nt == 1 && a.cache->head_dim <= 128 && a.dtype != NVFP4_DTYPE_F32 &&
        !(p.prefix.slots && !p.prefix.tile)) {
      const int64_t n = a.batch * units, least = a.cache->head_dim <= 64 || n > 40 ? 3 : 2;
      const int64_t most = n / 20 < least ? least : n / 20 > 12 ? 12 : n / 20;
      const int w = n <= 256 ? 16 : n <= 512 ? 8 : 4;
      whole = a.max_kv <= 32 * w * most;
      if (whole) r.waves = w, p.finish = p.prefix.slots > 0;
    }
    if (!whole && held >= (r.tile ? kTileCut * (float)a.batch : 1.0f)) {
      r.target = target;
      const int64_t n = (int64_t)target + 1 + a.batch, most = a.batch * cdiv(a.max_kv, 128);
      r.slots = (int)(n < most ? n : most);
    }
  }
  // A short prefix that tiles of many rows read: the own tokens' workgroups go over it first. That
  // saves the partial sums (2 KiB a row and head of 128, and the join; about as much time as the
  // products of 1024 tokens) and costs the products of the rows that its tiles hold in vain (of ragged
  // sequences half a tile each): 3 x up to 772 queries of 56 heads on 843 tokens, 79 before them: 83
  // -> 41 us, 64 x up to 10 of 32 heads on 1000 behind 500: 47 -> 39. The other way round 32 x up to
  // 65 on 2000 behind 1500: 170 us, 127 shared, and 16 x 64 on 64 behind 4000: 112, 105.
  if (own && p.own.tile && p.own.target == 0.0f && p.prefix.slots && a.prefix_len <= a.max_kv) {
    const int64_t tile = 16 * p.own.nt * p.own.waves, rows = a.tokens * G;
    const int64_t vain = a.batch * (a.tokens == a.batch * a.max_q ? p.own.row_tiles * tile - a.max_q * G : tile / 2);
    if ((double)a.prefix_len * (double)vain <= 1024.0 * (double)rows) p.lead = 1, p.prefix = Part{};
  }
  p.direct = p.prefix.slots == 0 ? p.own.target == 0.0f : p.prefix.slots == 1 && p.own.slots == 0;
  return p;
}

inline int64_t part_grid(const KvAttention &a, const Part &r) {
  return (int64_t)r.slots * a.cache->kv_heads * r.row_tiles;
}

// partial rows of the two launches
inline int64_t prefix_rows(const KvAttention &a, const Plan &p) {
  return (int64_t)p.prefix.slots * a.tokens * a.heads;
}
inline int64_t own_rows(const KvAttention &a, const Plan &p) {
  if (p.own.target > 0.0f) return (int64_t)p.own.slots * a.max_q * a.heads;
  return p.own.slots && !p.finish ? a.tokens * a.heads : 0;
}

// The join: groups of HD / 4 lanes in a workgroup of 256, and how many of them share a row (a power
// of two, about the pieces of a row).
inline int join_groups(const KvAttention &a) {
  return a.cache->head_dim <= 64 ? 16 : a.cache->head_dim <= 128 ? 8 : 4;
}
inline int join_per(const KvAttention &a, const Plan &p) {
  const float n = (float)p.prefix.slots + p.own.target / (float)a.batch;
  int per = 1;
  while (per < join_groups(a) && (float)per < n) per *= 2;
  return per;
}
inline bool joins(const Plan &p) { return !p.direct && !p.finish; }
inline int64_t join_grid(const KvAttention &a, const Plan &p) {
  return cdiv(a.max_q * a.heads, join_groups(a) / join_per(a, p));
}

// HIP launches less than 2^32 threads a dimension. A part of more (many sequences behind a loose
// max_q) goes in several launches of whole slots; 0 if one slot is too many.
constexpr int64_t kMaxThreads = UINT32_MAX;
inline int64_t slots_a_launch(const KvAttention &a, const Part &r) {
  return kMaxThreads / (64 * r.waves) / (a.cache->kv_heads * r.row_tiles);
}

struct Launch {
  int list;        // 0 the prefix, 1 own tokens, 2 the join
  int both;        // the own tokens' workgroups follow the prefix's
  int slot0;       // the first slot
  int64_t grid;    // workgroups (of the prefix and the own tokens: all)
  int threads;     // of a workgroup
};

// f(Launch) for every launch of the call, in order.
template <typename F>
void each_launch(const KvAttention &a, const Plan &p, F f) {
  const int64_t n0 = part_grid(a, p.prefix), n1 = part_grid(a, p.own);
  const bool both = n0 && n1 && p.prefix.nt == p.own.nt && p.prefix.waves == p.own.waves &&
                    p.prefix.tile == p.own.tile && (n0 + n1) * 64 * p.own.waves <= kMaxThreads;
  const auto part = [&](int k, const Part &r) {
    const int64_t most = slots_a_launch(a, r);
    for (int64_t at = 0; at < r.slots; at += most) {
      const int64_t n = r.slots - at < most ? r.slots - at : most;
      f(Launch{k, 0, (int)at, n * a.cache->kv_heads * r.row_tiles, 64 * r.waves});
    }
  };
  if (both) {
    f(Launch{0, 1, 0, n0 + n1, 64 * p.own.waves});
  } else {
    if (n0) part(0, p.prefix);
    if (n1) part(1, p.own);
  }
  if (joins(p)) f(Launch{2, 0, 0, join_grid(a, p), 256});
}

// whether the call can be launched
inline bool kv_attention_fits(const KvAttention &a, const Plan &p) {
  for (int k = 0; k < 2; ++k) {
    const Part &r = k ? p.own : p.prefix;
    if (r.slots && (part_grid(a, r) > INT32_MAX || slots_a_launch(a, r) < 1)) return false;
  }
  return !joins(p) || join_grid(a, p) * 256 <= kMaxThreads;
}
inline bool kv_attention_fits(const KvAttention &a) { return kv_attention_fits(a, plan_of(a)); }

inline size_t kv_attention_workspace_size(const KvAttention &a, const Plan &p) {
  if (p.direct) return 0;
  return (size_t)((prefix_rows(a, p) + own_rows(a, p)) * (a.cache->head_dim * 4 + 8) + a.batch * 8);
}
inline size_t kv_attention_workspace_size(const KvAttention &a) { return kv_attention_workspace_size(a, plan_of(a)); }

}  // namespace nvfp4
