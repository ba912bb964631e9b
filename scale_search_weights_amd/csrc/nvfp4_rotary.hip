// Rotary positions, and the append to the key/value cache that turns keys on the way.
//
// Both are bound by memory: a turned value is read and written once, and its cosine and sine are shared by
// all heads. A workgroup takes a few tokens: it computes their cosines and sines once, in 64 bits, into a
// table in LDS, and goes over the rows of its heads in the order of memory. (With a lane per token and pair
// group that goes over the heads, without a table, 12000 tokens of 32 heads of 128 took 40 us, 31 so: 6.3 TB/s,
// over a copy's 5.1 since half of the input of two such calls in turn stays in the last cache; 9801 x 16 fp32
// heads of 72, 90 MB, 17 us, 5.3 TB/s.) The append adds the quantiser, about 260 vector instructions a
// block of 16, and runs at 5.4 TB/s with queries (16384 tokens of 32 and 8 heads of 128: 65 us); without
// them vector work bounds it (27 us, 21 for the write without rotation).
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_rotary.h"
#include "nvfp4_rotary_plan.h"
#include "nvfp4_rows.h"

namespace nvfp4 {

// ---------------------------------------------------------------- angles

// Taylor's coefficients of sin r / r and cos r by powers of r^2, highest first. In memory, so that they are
// scalar operands: as literals they took 30 vector registers.
__constant__ double kSin[7] = {-1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0, 1.0 / 362880.0,
                               -1.0 / 5040.0, 1.0 / 120.0, -1.0 / 6.0};
__constant__ double kCos[7] = {-1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0, 1.0 / 40320.0,
                               -1.0 / 720.0, 1.0 / 24.0, -0.5};

// c = fp32(factor cos(p w)), s = fp32(factor sin(p w)), each from 64 bits. The product is kept as a
// sum of two doubles; it is reduced by multiples of pi/2 (pi/2 too in two doubles) to |r| <= pi/4,
// where the sums to r^15 and r^14 are off by less than 1e-15.
__device__ __forceinline__ void turn_of(double p, double w, double factor, float &c, float &s) {
  const double a = p * w, low = __builtin_fma(p, w, -a);
  const double n = __builtin_rint(a * 0.63661977236758134308);
  double r = __builtin_fma(-n, 1.57079632679489661923, a);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r) + low;
  const double z = r * r;
  double si = kSin[0], co = kCos[0];
#pragma unroll
  for (int i = 1; i < 7; ++i) si = __builtin_fma(si, z, kSin[i]), co = __builtin_fma(co, z, kCos[i]);
  si = __builtin_fma(si * z, r, r);
  co = __builtin_fma(co, z, 1.0);
  // quarter turns: n mod 4 without passing 32 bits
  const int quarter = (int)(n - 4.0 * __builtin_floor(0.25 * n));
  const double x = quarter & 1 ? si : co, y = quarter & 1 ? co : si;
  c = (float)((quarter == 1 || quarter == 2 ? -x : x) * factor);
  s = (float)((quarter >= 2 ? -y : y) * factor);
}

// ---------------------------------------------------------------- rows

// V values as they lie in memory, converted where they are used, so that a load can stay on its way.
template <int DT, int V>
struct Piece {
  static constexpr int W = DT == NVFP4_DTYPE_BF16 ? V / 2 : V;  // words
  static constexpr int N = W < 4 ? 2 : 4;                       // of a load
  typedef unsigned Load __attribute__((ext_vector_type(N)));
  Load w[W / N];

  __device__ __forceinline__ void load(const void *x, int64_t e) {
    const Load *p = reinterpret_cast<const Load *>(static_cast<const char *>(x) + e * (DT == NVFP4_DTYPE_BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < W / N; ++i) w[i] = p[i];
  }
  __device__ __forceinline__ float operator[](int i) const {
    if (DT != NVFP4_DTYPE_BF16) return __uint_as_float(w[i / N][i % N]);
    const unsigned x = w[i / 2 / N][i / 2 % N];
    return i & 1 ? bf16_hi(x) : bf16_lo(x);
  }
  template <bool STREAM>
  static __device__ __forceinline__ void store(void *x, int64_t e, const float *v) {
    Load *p = reinterpret_cast<Load *>(static_cast<char *>(x) + e * (DT == NVFP4_DTYPE_BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < W / N; ++i) {
      Load y;
#pragma unroll
      for (int k = 0; k < N; ++k)
        y[k] = DT == NVFP4_DTYPE_BF16 ? bf16x2_bits(v[2 * (i * N + k)], v[2 * (i * N + k) + 1])
                                      : __float_as_uint(v[i * N + k]);
      if (STREAM) __builtin_nontemporal_store(y, p + i);
      else p[i] = y;
    }
  }
};

// The items of a workgroup: (token, head, unit of the row), units fastest.
struct Items {
  int64_t t0;
  int n, h0, heads, units;
  Div by_units, by_heads, by_last;  // by_last: the heads of the last group

  // a workgroup's chunk of the tokens and group of the heads
  __device__ __forceinline__ void take(int chunk, int group, int64_t tokens, int all) {
    t0 += (int64_t)chunk * n;
    n = (int)max((int64_t)0, min((int64_t)n, tokens - t0));
    h0 = group * heads;
    if (h0 + heads > all) heads = all - h0, by_heads = by_last;
  }

  __device__ __forceinline__ int count() const { return n * heads * units; }
  __device__ __forceinline__ void find(int item, int &tok, int &h, int &unit) const {
    const int row = by_units.of(item);
    unit = item - row * units;
    tok = by_heads.of(row);
    h = row - tok * heads;
  }
};

// Where entry j of the table lies: two spare entries after every 16, so that lanes that read 8 or 16
// entries each begin in different banks. N entries from a multiple of N on (N 2, 4 or 8) are read at once.
__device__ __forceinline__ int table_at(int j) { return j + (j >> 4) * 2; }

template <int N>
struct Turns {
  float4 e[N / 2];

  __device__ __forceinline__ Turns(const float2 *table, int j) {
    const float4 *p = reinterpret_cast<const float4 *>(table + table_at(j));
#pragma unroll
    for (int i = 0; i < N / 2; ++i) e[i] = p[i];
  }
  __device__ __forceinline__ float2 operator[](int i) const {
    return i & 1 ? make_float2(e[i / 2].z, e[i / 2].w) : make_float2(e[i / 2].x, e[i / 2].y);
  }
};

// The table: cosines and sines of the pairs of a workgroup's tokens. An entry's axis leads to its position:
// two loads that wait for each other, so the axis is loaded two entries ahead of the arithmetic and the
// position one, and a lane's first entry before its rows, since loads come back in order.
struct Angle {
  double w;
  int64_t p;
  int axis, tok;

  __device__ __forceinline__ void look(const Turn &r, const Items &it, const Div &by_pairs, int j) {
    axis = -1, tok = 0;
    if (j >= it.n * r.pairs) return;
    tok = by_pairs.of(j);
    const int pair = j - tok * r.pairs;
    axis = r.axis ? r.axis[pair] : 0;
    w = r.inv_freq[pair];
  }
  __device__ __forceinline__ void place(const Turn &r, const Items &it) {
    p = axis >= 0 && axis < r.axes ? r.positions[axis * r.stride + it.t0 + tok] : 0;
  }
};
struct Angles {
  Angle now, next;

  __device__ __forceinline__ void open(const Turn &r, const Items &it, const Div &by_pairs) {
    now.look(r, it, by_pairs, threadIdx.x);
    next.look(r, it, by_pairs, threadIdx.x + 256);
    now.place(r, it);
  }
  __device__ __forceinline__ void build(const Turn &r, const Items &it, const Div &by_pairs, bool transpose,
                                        float2 *table) {
#pragma unroll 1
    for (int j = threadIdx.x; j < it.n * r.pairs; j += 256) {
      const Angle x = now;
      now = next;
      now.place(r, it);
      next.look(r, it, by_pairs, j + 512);
      float2 e;
      turn_of((double)x.p, x.w, r.factor, e.x, e.y);
      if (transpose) e.y = -e.y;
      table[table_at(j)] = e;
    }
  }
};

// ---------------------------------------------------------------- rotate

struct Rotate {
  Turn turn;
  const void *x;
  void *out;
  int64_t ts, hs, out_ts, out_hs;
  int transpose;
  Div by_pairs;
};

// A unit of a row: V channels of the first half and V of the second half of those that turn, or of those
// that pass through. Pieces of 16 bytes (8 where halves do not begin at 16), so the lanes of a load or
// store are contiguous; adjacent pairs lie within a piece.
template <int DT, int V, bool ADJACENT>
struct Unit {
  Piece<DT, V> x0, x1;
  int64_t out;     // the output row
  int entry, a, b; // first table entry, -1 if the unit passes through; first channels of x0 and x1

  __device__ __forceinline__ void load(const Rotate &p, const Items &it, int item) {
    int tok, h, u;
    it.find(item, tok, h, u);
    const bool turned = u < p.turn.pairs / V;
    const int P = p.turn.pairs;
    a = turned ? V * u : V * u + P;
    b = turned ? a + P : a + it.units * V - P;
    entry = turned ? tok * P + (ADJACENT ? V / 2 : V) * u : -1;
    const int64_t t = it.t0 + tok, e = t * p.ts + (it.h0 + h) * p.hs;
    out = t * p.out_ts + (it.h0 + h) * p.out_hs;
    x0.load(p.x, e + a);
    x1.load(p.x, e + b);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(const Rotate &p, const float2 *table) {
    float y[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = x0[i], y[V + i] = x1[i];
    if (entry >= 0) {
      constexpr int N = ADJACENT ? V / 2 : V;  // pairs of a piece
      const Turns<N> ra(table, entry), rb(table, ADJACENT ? entry + p.turn.pairs / 2 : entry);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int i0 = ADJACENT ? 2 * i : i, i1 = ADJACENT ? 2 * i + 1 : V + i;
        const float2 r = i < N ? ra[i] : rb[i - N];
        const float z = y[i0] * r.x - y[i1] * r.y;
        y[i1] = y[i1] * r.x + y[i0] * r.y;
        y[i0] = z;
      }
    }
    Piece<DT, V>::template store<STREAM>(p.out, out + a, y);
    Piece<DT, V>::template store<STREAM>(p.out, out + b, y + V);
  }
};

template <int DT, int V, bool ADJACENT, bool STREAM>
__device__ __forceinline__ void rotate_items(const Rotate &p, const Items &it, float2 *table) {
  const int items = it.count();
  Unit<DT, V, ADJACENT> x;
  int i = threadIdx.x;
  Angles angles;
  angles.open(p.turn, it, p.by_pairs);
  if (i < items) x.load(p, it, i);  // on its way beside the table
  angles.build(p.turn, it, p.by_pairs, p.transpose, table);
  lds_barrier();
#pragma unroll 1
  while (i < items) {
    Unit<DT, V, ADJACENT> y = x;
    i += 256;
    if (i < items) x.load(p, it, i);
    y.template store<STREAM>(p, table);
  }
}

template <int DT, int V, bool ADJACENT, bool STREAM>
__global__ void __launch_bounds__(256) k_rotate(Rotate p, Items it, int64_t tokens, int all_heads) {
  __shared__ __align__(16) float2 table[kTable + kTable / 8];
  it.take(blockIdx.x, blockIdx.y, tokens, all_heads);
  rotate_items<DT, V, ADJACENT, STREAM>(p, it, table);
}

static Items items_of(int n, const RowPlan &r, int64_t heads) {
  const int last = heads ? (int)((heads - 1) % r.heads) + 1 : 1;
  return {0, n, 0, r.heads, r.units, Div(r.units), Div(r.heads), Div(last)};
}

// f(adjacent, stream) with both as types.
template <typename F>
static void with_flags(bool adjacent, bool stream, F f) {
  if (adjacent && stream) f(std::true_type{}, std::true_type{});
  else if (adjacent) f(std::true_type{}, std::false_type{});
  else if (stream) f(std::false_type{}, std::true_type{});
  else f(std::false_type{}, std::false_type{});
}

int launch_rotate(const Turn &turn, bool adjacent, bool transpose, const RowSpan &x,
                  const RowSpan &out, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                  hipStream_t st) {
  const bool bf16 = dtype == NVFP4_DTYPE_BF16;
  const RotatePlan plan = rotate_plan(bf16, tokens, heads, head_dim, turn.pairs);
  const Rotate p = {turn, x.x, const_cast<void *>(out.x), x.ts, x.hs, out.ts, out.hs, transpose, Div(turn.pairs)};
  Items it = items_of(plan.tokens, plan.rows, heads);
  with_flags(adjacent, streams(bf16, tokens, heads, head_dim), [&](auto adj, auto stream) {
    each_chunks(tokens, plan.tokens, plan.rows.groups, [&](int64_t chunks, int64_t t0) {
      it.t0 = t0;
      const dim3 g((unsigned)chunks, (unsigned)plan.rows.groups), b(256);
      constexpr int BF = NVFP4_DTYPE_BF16, F = NVFP4_DTYPE_F32;
      if (plan.v == 8)
        hipLaunchKernelGGL((k_rotate<BF, 8, adj.value, stream.value>), g, b, 0, st, p, it, tokens, (int)heads);
      else if (bf16)
        hipLaunchKernelGGL((k_rotate<BF, 4, adj.value, stream.value>), g, b, 0, st, p, it, tokens, (int)heads);
      else
        hipLaunchKernelGGL((k_rotate<F, 4, adj.value, stream.value>), g, b, 0, st, p, it, tokens, (int)heads);
    });
  });
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- append

struct Append {
  Rotate q;
  const void *x[2];
  int64_t ts[2], hs[2];
  uint8_t *codes[2], *scales[2];
  const float *S[2];
  const int64_t *slots;
  int64_t n_slots;
  int kv_heads, page_shift;
};

// A block of 16 channels of a key (turned) or value row.
template <int DT, bool ADJACENT>
struct Block {
  Piece<DT, 8> x0, x1, o0, o1;  // its halves, and the other channels of their pairs
  int64_t slot;
  int tok, h, part;

  // the half's first channel is on which side of its pairs: 0, 1, or 2 for channels that pass through
  static __device__ __forceinline__ int side(const Append &p, int ch) {
    return ADJACENT ? (ch < 2 * p.q.turn.pairs ? 0 : 2) : ch < p.q.turn.pairs ? 0 : ch < 2 * p.q.turn.pairs ? 1 : 2;
  }
  __device__ __forceinline__ void load(const Append &p, const Items &it, int kv, int item) {
    it.find(item, tok, h, part);
    const int64_t t = it.t0 + tok, e = t * p.ts[kv] + (it.h0 + h) * p.hs[kv];
    const int ch = 16 * part, P = p.q.turn.pairs;
    slot = p.slots[t];
    x0.load(p.x[kv], e + ch);
    x1.load(p.x[kv], e + ch + 8);
    if (kv == 0 && !ADJACENT) {
      const int s0 = side(p, ch), s1 = side(p, ch + 8);
      if (s0 < 2) o0.load(p.x[0], e + ch + (s0 ? -P : P));
      if (s1 < 2) o1.load(p.x[0], e + ch + 8 + (s1 ? -P : P));
    }
  }
  // y = x c - other s (first of a pair) or x c + other s
  __device__ __forceinline__ void turn(const Append &p, const float2 *table, int ch, const Piece<DT, 8> &x,
                                       const Piece<DT, 8> &o, float *y) const {
    const int s = side(p, ch), P = p.q.turn.pairs;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    if (s == 2) return;
    const Turns<ADJACENT ? 4 : 8> r(table, tok * P + (ADJACENT ? ch / 2 : s ? ch - P : ch));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 e = r[ADJACENT ? i / 2 : i];
      const float other = ADJACENT ? x[i ^ 1] : o[i];
      y[i] = x[i] * e.x - other * ((ADJACENT ? i & 1 : s) ? -e.y : e.y);
    }
  }
  __device__ __forceinline__ void store(const Append &p, const Items &it, int kv, const float2 *table,
                                        const float4 *heads) const {
    if (slot < 0 || slot >= p.n_slots) return;
    float y[16];
    if (kv == 0) {
      turn(p, table, 16 * part, x0, o0, y);
      turn(p, table, 16 * part + 8, x1, o1, y + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x0[i], y[8 + i] = x1[i];
    }
    const float4 S = heads[h];
    uint2 codes;
    const int byte = quantise16(y, S.y, S.z, S.x, codes);
    const int64_t row = (((slot >> p.page_shift) * p.kv_heads + it.h0 + h) << p.page_shift) +
                        (slot & (((int64_t)1 << p.page_shift) - 1));
    reinterpret_cast<uint2 *>(p.codes[kv])[row * it.units + part] = codes;
    p.scales[kv][row * it.units + part] = (uint8_t)byte;
  }
};

template <int DT, bool ADJACENT>
__device__ __forceinline__ void append_items(const Append &p, const Items &it, int kv, float2 *table, float4 *heads) {
  const int items = it.count();
  Block<DT, ADJACENT> x;
  int i = threadIdx.x;
  Angles angles;
  if (kv == 0) angles.open(p.q.turn, it, p.q.by_pairs);
  float4 S = {i < it.heads ? p.S[kv][it.h0 + i] : 1.0f, 0.0f, 0.0f, 0.0f};
  if (i < items) x.load(p, it, kv, i);
  if (kv == 0) angles.build(p.q.turn, it, p.q.by_pairs, false, table);
  if (i < it.heads) {  // tensor scales and the brackets of 1 / (6 S)
    recip_bracket(6.0 * (double)S.x, S.y, S.z);
    heads[i] = S;
  }
  lds_barrier();
#pragma unroll 1
  while (i < items) {
    x.store(p, it, kv, table, heads);
    i += 256;
    if (i < items) x.load(p, it, kv, i);
  }
}

// The roles of a chunk of tokens (groups of key heads, of value heads, of query heads) follow each other on
// one die: workgroups go to the 8 dies in turn. So those that quantise run beside those that only move
// queries (16384 tokens of 32 and 8 heads of 128: 66 us, 74 with one role after the other). Six
// workgroups a CU, 80 registers: 66 us, 68 with as many registers as it asks for, 83 with 64 (one role
// after the other); fp32 needs 96. With pairs in halves that is five registers short: they are spilled around
// the quantiser's exact search, which a block reaches only next to a rounding boundary, so scratch is
// reserved but hardly touched.
template <int DT, bool ADJACENT, bool STREAM>
__global__ void __launch_bounds__(256, DT == NVFP4_DTYPE_F32 ? 5 : 6) k_kv_append(Append p, Items kv, Items q, int64_t tokens, int q_heads) {
  __shared__ __align__(16) float2 table[kTable + kTable / 8];
  __shared__ float4 heads[kHeads];
  const int groups = (p.kv_heads + kv.heads - 1) / kv.heads, all = groups * 2 + (q_heads + q.heads - 1) / q.heads;
  const int j = blockIdx.x >> 3, y = j % all, chunk = j / all * 8 + (blockIdx.x & 7);
  const int role = y < groups ? 0 : y < 2 * groups ? 1 : 2;
  Items it = role == 2 ? q : kv;
  it.take(chunk, y - role * groups, tokens, role == 2 ? q_heads : p.kv_heads);
  if (role == 2) rotate_items<DT, DT == NVFP4_DTYPE_BF16 ? 8 : 4, ADJACENT, STREAM>(p.q, it, table);
  else append_items<DT, ADJACENT>(p, it, role, table, heads);
}

int launch_kv_append(const nvfp4_kv_cache &c, const Turn &turn, bool adjacent, const RowSpan &q,
                     const RowSpan &q_out, const RowSpan &k, const RowSpan &v, int dtype,
                     int64_t tokens, int64_t heads, const int64_t *slots, hipStream_t st) {
  const bool bf16 = dtype == NVFP4_DTYPE_BF16;
  const AppendPlan plan = append_plan(bf16, tokens, heads, c.kv_heads, c.head_dim, turn.pairs);
  Append p = {{turn, q.x, const_cast<void *>(q_out.x), q.ts, q.hs, q_out.ts, q_out.hs, 0, Div(turn.pairs)}};
  p.x[0] = k.x, p.x[1] = v.x, p.ts[0] = k.ts, p.ts[1] = v.ts, p.hs[0] = k.hs, p.hs[1] = v.hs;
  p.codes[0] = c.k_codes, p.codes[1] = c.v_codes;
  p.scales[0] = c.k_scales, p.scales[1] = c.v_scales;
  p.S[0] = c.S_k, p.S[1] = c.S_v;
  p.slots = slots, p.n_slots = c.pages * c.page_size;
  p.kv_heads = (int)c.kv_heads, p.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  Items ikv = items_of(plan.tokens, plan.kv, c.kv_heads), iq = items_of(plan.tokens, plan.q, heads);
  const int64_t groups = 2 * plan.kv.groups + plan.q.groups;
  with_flags(adjacent, streams(bf16, tokens, heads, c.head_dim), [&](auto adj, auto stream) {
    each_chunks(tokens, plan.tokens, groups, [&](int64_t chunks, int64_t t0) {
      ikv.t0 = iq.t0 = t0;
      const dim3 g((unsigned)((chunks + 7) / 8 * 8 * groups)), b(256);
      constexpr int BF = NVFP4_DTYPE_BF16, F = NVFP4_DTYPE_F32;
      if (bf16)
        hipLaunchKernelGGL((k_kv_append<BF, adj.value, stream.value>), g, b, 0, st, p, ikv, iq, tokens, (int)heads);
      else
        hipLaunchKernelGGL((k_kv_append<F, adj.value, stream.value>), g, b, 0, st, p, ikv, iq, tokens, (int)heads);
    });
  });
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
