// How the rotation and the append are split into workgroups, and the quotients by which a lane finds its item:
// code that compiles without HIP.
#pragma once

#include <stdint.h>

namespace nvfp4 {

#if defined(__HIPCC__)
#define NVFP4_HD __host__ __device__
#else
#define NVFP4_HD
#endif

// Quotients of numbers below 2^16 by a divisor d up to 2^16, by one multiplication: m = floor(2^32 / d) + 1
// exceeds 2^32 / d by at most 1, so n m / 2^32 exceeds n / d by less than 2^-16, less than 1 / d.
struct Div {
  int d;
  uint32_t m;
  explicit Div(int d) : d(d), m(d == 1 ? 0 : (uint32_t)((1ull << 32) / (uint32_t)d + 1)) {}
  inline NVFP4_HD int of(int n) const { return m ? (int)((uint64_t)(uint32_t)n * m >> 32) : n; }
};

constexpr int kTable = 2048;  // cosine and sine pairs of a workgroup: 16 KiB of LDS
constexpr int kHeads = 64;    // key/value heads a workgroup takes at most (their scales are in LDS too)

// Workgroups wanted before they take more tokens each: two a CU.
constexpr int64_t kEnough = 512;

// Rows by (tokens of a workgroup, heads of a workgroup); a row is `units` items.
struct RowPlan {
  int units, heads;
  int64_t groups;  // of heads
};

// `most` items a token at most; few items in all: one a lane.
inline RowPlan heads_of(int64_t tokens, int64_t heads, int units, int64_t most, int64_t cap) {
  if (tokens * heads * units < kEnough * 256) most = 256;
  int64_t per = most / units;
  per = per < 1 ? 1 : per;
  per = per < cap ? per : cap;
  per = per < heads ? per : heads;
  per = per < 1 ? 1 : per;
  return {units, (int)per, (heads + per - 1) / per};
}

// Tokens of a workgroup: so many that it has `items`, as far as its table holds them and enough
// workgroups are left.
inline int tokens_of(int64_t tokens, int pairs, int64_t items_a_token, int64_t items, int64_t groups) {
  int n = 1;
  while (2 * n * items_a_token <= items && 2 * n * pairs <= kTable && tokens / (2 * n) * groups >= kEnough) n *= 2;
  return n;
}

struct RotatePlan {
  int v;  // channels of a piece
  int tokens;
  RowPlan rows;
};

// Pieces of 16 bytes, or of 8 where the halves of bf16 rows do not begin at multiples of 16. 16384 tokens of
// 32 heads of 128 in bf16: 42.4 us with 512 items a workgroup, 43.8 with 1024, 47.6 with 256; 32 tokens of 40
// heads: 3.1 us with an item a lane, 3.6 with two, 4.4 with four.
inline RotatePlan rotate_plan(bool bf16, int64_t tokens, int64_t heads, int64_t head_dim, int pairs) {
  RotatePlan p;
  p.v = bf16 && pairs % 8 == 0 && head_dim % 16 == 0 ? 8 : 4;
  p.rows = heads_of(tokens, heads, (int)head_dim / (2 * p.v), 1024, heads);
  p.tokens = tokens_of(tokens, pairs, (int64_t)p.rows.heads * p.rows.units, 512, p.rows.groups);
  return p;
}

// 16384 tokens of 8 key/value heads of 128, us, with 256 and with 512 items a workgroup of keys or values: 32
// query heads 65, 71; 64 120, 125; 8 38.7, 37.2; none 31, 28.
struct AppendPlan {
  int tokens;
  RowPlan kv, q;  // kv for keys and for values
};

inline AppendPlan append_plan(bool bf16, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int pairs) {
  AppendPlan p;
  const int units = (int)head_dim / 16;
  p.kv = heads_of(tokens, kv_heads, units, 4096, kHeads);
  const int q_units = bf16 ? units : 2 * units;
  const int64_t q_items = heads * q_units;
  const int64_t groups = 2 * p.kv.groups + (q_items + 2047) / 2048;
  p.tokens = tokens_of(tokens, pairs, (int64_t)p.kv.heads * units, heads >= 2 * kv_heads ? 256 : 512, groups);
  p.q = heads_of(tokens, heads, q_units, 2048 / p.tokens, heads);
  return p;
}

// Whether the rows of a rotation, or of an append's queries, are stored non-temporally: where they pass the dies'
// L2, 32 MB in all; fewer are left for whoever reads them next. us, non-temporal and ordinary, 32 bf16 heads of
// 128. On inputs and outputs that no cache holds: 16 MB 7.9, 8.0; 32 14.0, 14.0; 48 19.7, 21.6; 64 24.9, 25.9; 96
// 35.7, 38.3; 128 47.3, 49.1; 256 92.6, 95.0; 512 187.2, 186.9. Two of each in turn: 64 21.0, 22.1; 96 30.4, 38.2;
// 128 40.7, 48.4 (ordinary rows put inputs out of the last cache). Between a kernel that writes the input and one
// that reads the output, all three: 16 MB 20.5, 19.4; 32 34.4, 32.9; 48 48.0, 46.2; 64 62.5, 60.6; 96 95.6, 100.7;
// 128 125.9, 133.5; 256 279, 271. The append of 16384 tokens of 32 and 8 heads: 66, 69.
inline bool streams(bool bf16, int64_t tokens, int64_t heads, int64_t head_dim) {
  return tokens * heads * head_dim * (bf16 ? 2 : 4) > (32 << 20);
}

// f(chunks of this launch, the first one's first token), for all tokens in chunks of n: with `groups`
// workgroups a chunk, of 256 threads, a launch stays under 2^32 threads.
template <typename F>
void each_chunks(int64_t tokens, int n, int64_t groups, F f) {
  const int64_t chunks = (tokens + n - 1) / n, fit = ((1 << 24) - 1) / groups / 8 * 8, most = fit < 8 ? 8 : fit;
  for (int64_t at = 0; at < chunks; at += most) f(chunks - at < most ? chunks - at : most, at * n);
}

}  // namespace nvfp4
