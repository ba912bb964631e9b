// Softmax attention of new queries over keys and values cached in NVFP4.
//
// For a query row r and a cached token t (codes G, block scales s, head scale S):
//   score = scale * S_k * sum_d q[d] G[d] s[d/16],  out = S_v * sum_t p_t G[t] s[t] / sum_t p_t.
// G s has at most 6 significant bits and lies in [2^-10, 2688], so it is exact in fp16: one
// hardware convert of two codes and one packed multiply by the scale give MFMA operands, S
// stays outside as one fp32 factor.
//
// Transposed tiles. The scores are computed as K Q^T (16 tokens x 16 rows) and the output as
// V^T P^T, so a lane keeps one query row (lane & 15) throughout: its running maximum and sum
// are lane values, and the probabilities come out of the first product in the operand layout
// of the second, with no exchange between lanes. The contraction indices may be permuted
// freely as long as both operands agree, which lets every lane load whole 4..16-byte pieces
// of the cache: lane (i, quad) takes channels [quad HD/4, ..) of key token i, and channels
// [i HD/16, ..) of the value tokens 4 quad + 0..3 and 16 + 4 quad + 0..3.
//
// Two kernels. With up to 32 rows a (sequence, key/value head) the cache is read at the rate of
// memory: k_kv_attn_rows, every wave dequantising its own tokens in registers (about 260 vector
// instructions for 32 tokens and 16 rows; 524000 tokens of 8 heads of 128, 604 MB, in 117 us,
// 5.2 TB/s). With more rows the products bound it: k_kv_attn_tile, where the waves share what they
// dequantise through LDS (2 x 2048 queries of 32 heads on 8192 tokens, 481 GFLOP, in 433 us,
// 1.1 PFLOP/s). The sequence axis is cut into pieces where there are few rows; their sums are
// joined in a fixed order, by k_kv_attn_join or, where only a prefix is cut, by the workgroups of
// the sequences' own tokens (finish_rows).
//
// Running maximum: it is raised (and the sums rescaled) only when a probability relative to it
// leaves fp16's range, a few times per sequence instead of once per tile, and no maximum is
// taken in between: the sums show the overflow (2048-query chunk 577 -> 560 us).
#include "nvfp4_device.h"
#include "nvfp4_kv.h"

namespace nvfp4 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A token list and the query rows that read it: the shared prefix (all rows of the call over one
// page list), or the sequences' own tokens.
struct List {
  const int32_t *table;
  int64_t table_width;
  int max_len, causal, prefix;
  int row_tiles, slots;
  float target;  // own tokens: pieces wanted in all; 0 for one piece a sequence
  int piece;     // prefix: tokens of a piece
  int joined;    // own tokens: their rows have prefix pieces too
  int finish;    // own tokens in one piece: its workgroup adds that many prefix pieces and writes out
  float *opart;
  float2 *ml;
  int2 *where;   // own tokens: first slot and pieces of a sequence that has any
};

struct Attn {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *S_k, *S_v;
  const void *q;
  int64_t q_ts, q_hs;
  const int32_t *q_offsets, *kv_lens;
  int tokens, heads, kv_heads, group, hd, page_shift, pages, max_q, batch;
  float scale;
  int direct;    // one piece a row, written straight to out
  int first;     // workgroups of list[0]; the others are list[1]'s
  int slot0;     // the launch's first slot of list[0]
  int lead_len;  // tokens of the prefix, if the own tokens' workgroups take it first
  const int32_t *lead;  // and its pages
  void *out;
  float *lse;
  List list[2];
};

// One sequence's share of the call.
struct Job {
  int q0, nq, len, causal;
  const int32_t *pages;
};

// len: the sequence's own tokens (not of the prefix's job).
__device__ __forceinline__ Job job_of(const Attn &p, const List &k, int b, int len) {
  Job j;
  if (k.prefix) {
    j.q0 = 0, j.nq = p.tokens, j.len = k.max_len, j.causal = 0, j.pages = k.table;
  } else {
    const Span s = rows_of(p.q_offsets, b, p.max_q, p.tokens);
    j.q0 = s.lo, j.nq = s.hi - s.lo;
    j.len = len;
    j.causal = k.causal;
    j.pages = k.table + b * k.table_width;
  }
  return j;
}

// Sums over the wave's lanes in six DPP steps: lane l gets the sum of lanes 0 .. l.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_add(T x) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false);
  return x + __builtin_bit_cast(T, o);
}
template <typename T>
__device__ __forceinline__ T prefix_sum(T x) {
  x = dpp_add<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8
  x = dpp_add<0x112, 0xF>(x);
  x = dpp_add<0x114, 0xF>(x);
  x = dpp_add<0x118, 0xF>(x);
  x = dpp_add<0x142, 0xA>(x);  // row_bcast 15, 31
  return dpp_add<0x143, 0xC>(x);
}

// The sequences' own tokens are cut into pieces of at most a length chosen from the lengths found
// on the device so that about `target` pieces come out in all (at most target + batch: every
// sequence may add one that is not full); a sequence's pieces are equal, in units of 128 tokens.
// Slots number the pieces over all sequences, so the grid has few workgroups without work however
// unequal the lengths are. Every wave finds its piece by itself: two passes over the lengths.
// (64 sequences of 512 to 8192 tokens: 92 us with pieces of one length for the bound, 60 us so.)
struct Piece {
  int b, first, count, tokens, len;  // sequence, its first slot, pieces, tokens of each, length
};

__device__ __forceinline__ int length_of(const int32_t *kv_lens, int b, int batch, int max_len) {
  return b < batch ? min(max(kv_lens[b], 0), max_len) : 0;
}

// The piece of `slot`; b = -1: there is none.
__device__ __forceinline__ Piece find_piece(const int32_t *kv_lens, int batch, int max_len,
                                            float target, int slot, int lane) {
  const int mine = length_of(kv_lens, lane, batch, max_len);  // the only load for 64 sequences
  float sum = (float)(mine + 127 >> 7);
  for (int b = lane + 64; b < batch; b += 64)
    sum += (float)(length_of(kv_lens, b, batch, max_len) + 127 >> 7);
  sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(prefix_sum(sum)), 63));
  const float x = ceilf(sum / target);  // the same in every wave: same order, same bits
  const int per = x < 1.0f ? 1 : (x > 8388608.0f ? 8388608 : (int)x);
  Piece r = {-1, 0, 0, 0, 0};
  int before = 0;
  for (int b0 = 0; b0 < batch; b0 += 64) {
    const int len = b0 ? length_of(kv_lens, b0 + lane, batch, max_len) : mine;
    const int n = ((len + 127 >> 7) + per - 1) / per;
    const int upto = prefix_sum(n);
    const unsigned long long hit =
        __ballot(slot >= before + upto - n && slot < before + upto);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      r.b = b0 + at;
      r.len = __builtin_amdgcn_readlane(len, at);
      r.count = __builtin_amdgcn_readlane(n, at);
      r.first = before + __builtin_amdgcn_readlane(upto, at) - r.count;
      r.tokens = ((r.len + 127 >> 7) + r.count - 1) / r.count << 7;
      return r;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return r;
}

// A workgroup's share of the call: a row tile of one key/value head, tokens t0 .. t1 - 1, and
// its list and slot (where its partial rows go, unless direct).
struct Share {
  Job j;
  int h, rt, t0, t1, direct, list, slot;
};

// The job's first partial row. A slot holds the rows of all tokens (prefix), of one sequence (own
// tokens in pieces), or, of own tokens in one piece, the rows of all tokens are one slot.
__device__ __forceinline__ int64_t part_of(const Attn &p, const Share &s) {
  const List &k = p.list[s.list];
  if (k.prefix || k.target > 0.0f)
    return ((int64_t)s.slot * p.kv_heads + s.h) * ((k.prefix ? p.tokens : p.max_q) * p.group);
  return ((int64_t)s.h * p.tokens + s.j.q0) * p.group;
}

__device__ __forceinline__ bool share_of(const Attn &p, int lane, Share &s) {
  // slots last: those without a piece come at the end, and the pieces, which are dealt to the
  // chip's eight dies in turn, fall on all of them
  int w = blockIdx.x;
  const int second = w >= p.first;
  if (second) w -= p.first;  // only where both lists start at slot 0
  const List &k = p.list[second];
  s.h = w % p.kv_heads;
  w /= p.kv_heads;
  s.rt = k.row_tiles - 1 - w % k.row_tiles;  // the tiles that see most tokens first
  const int slot = p.slot0 + w / k.row_tiles;
  s.direct = p.direct;
  if (k.prefix || k.target == 0.0f) {
    const int len = k.prefix || !p.kv_lens ? 0 : length_of(p.kv_lens, slot, p.batch, k.max_len);
    s.j = job_of(p, k, k.prefix ? 0 : slot, len);
    s.t0 = k.prefix ? slot * k.piece : 0;
    s.t1 = k.prefix ? min(s.j.len, s.t0 + k.piece) : s.j.len;
  } else {
    const Piece x = find_piece(p.kv_lens, p.batch, k.max_len, k.target, slot, lane);
    if (x.b < 0) return false;
    s.direct = x.count == 1 && !k.joined;  // the join skips such sequences
    if (slot == x.first && s.h == 0 && s.rt == 0 && threadIdx.x == 0)
      k.where[x.b] = make_int2(x.first, x.count);  // for the join
    s.j = job_of(p, k, x.b, x.len);
    s.t0 = (slot - x.first) * x.tokens;
    s.t1 = min(s.j.len, s.t0 + x.tokens);
  }
  s.list = second, s.slot = slot;
  return true;
}

__device__ __forceinline__ h2 codes2(unsigned w, int b) {
  return b == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)
         : b == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)
         : b == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)
                  : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
}

// Two scale bytes (half 0 or 1 of w) as fp16: the magnitude, 0x7F as zero (the convert gives
// NaN there, and the maximum with 0 drops it).
__device__ __forceinline__ h2 scales2(unsigned w, int half) {
  const h2 s = half ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w & 0x7F7F7F7Fu, 1.0f, true)
                    : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w & 0x7F7F7F7Fu, 1.0f, false);
  return __builtin_elementwise_max(s, (h2){0, 0});
}

// Rows' power-of-two scaling: |q| max in [2^14, 2^15) as fp16, or as an fp16 pair hi + lo.
__device__ __forceinline__ float row_factor(float amax, float &inverse) {
  int e = (int)(__float_as_uint(amax) >> 23);
  e = 141 - (e < 21 ? 21 : e);  // 14 - exponent
  inverse = __uint_as_float((unsigned)(127 - e) << 23);
  return __uint_as_float((unsigned)(127 + e) << 23);
}

// The ends of a row with sum l over the maximum m (log2): the sums' factor and lse. A row that sees
// nothing has l = 0 exactly, every other one at least 2^base (base_of), and a query that is not
// finite NaN, which stays NaN: piece by piece, however many pieces there are.
__device__ __forceinline__ float out_factor(float S_v, float l) { return l == 0.0f ? 0.0f : S_v / l; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(l));
}

// ---------------------------------------------------------------- raw groups of 16 tokens

constexpr int more(int a) { return a > 1 ? a : 1; }

// One lane's share of 16 tokens of one head, as cached. A group lies in one page.
template <int HD>
struct Group {
  unsigned k[HD / 32];             // HD/4 key codes of token i, from channel quad HD/4
  unsigned ks;                     // a word of scales with theirs in it (scale_bits)
  unsigned v[4][more(HD / 128)];   // HD/16 value codes of tokens 4 quad + 0..3, from channel i HD/16
  unsigned vs;                     // the same for HD/64 value scales of token lane / 4
};

// Scales are loaded as whole words, so that nothing is done to them before they are used (a
// narrow load's zero extension would wait for it at once). Part q of a token's four: the
// lane's HD/64 bytes, moved down.
template <int HD, bool EXACT>
__device__ __forceinline__ unsigned scale_bits(unsigned w, unsigned q) {
  if (!EXACT || HD > 128) return w;
  return HD == 128 ? w >> 16 * (q & 1) : w >> 8 * q;
}

// Page ids of a token range: lane k of `ids` holds the id of the k-th group of 16 tokens of the
// run of 1024 at t, `next` those of the run after it, so a group takes its id from a register
// and its loads wait for nothing. A run is left (`advance`) outside the loop over its tiles:
// a conditional load inside it would have every iteration wait for its own new loads.
constexpr int kRun = 1024;

struct Pages {
  int t, ids, next;
};

__device__ __forceinline__ int load_ids(const Job &j, int page_shift, int t, int t_end, int lane) {
  t += 16 * lane;
  return t < t_end ? j.pages[t >> page_shift] : -1;
}

__device__ __forceinline__ Pages open_pages(const Job &j, int page_shift, int t0, int t_end, int lane) {
  return {t0, load_ids(j, page_shift, t0, t_end, lane), load_ids(j, page_shift, t0 + kRun, t_end, lane)};
}

__device__ __forceinline__ void advance(Pages &pg, const Job &j, int page_shift, int t_end, int lane) {
  pg.t += kRun;
  pg.ids = pg.next;
  pg.next = load_ids(j, page_shift, pg.t + kRun, t_end, lane);
}

__device__ __forceinline__ int page_of(const Pages &pg, int t) {
  const int g = (t - pg.t) >> 4;
  if (g < kRun / 16) return __builtin_amdgcn_readlane(pg.ids, g);
  return __builtin_amdgcn_readlane(pg.next, g - kRun / 16);
}

#define GLOBAL __attribute__((address_space(1)))

// An unsigned lane offset that stays 32 bits beside a scalar base address (hoisted out of a loop
// as 64 bits it would take two registers, and every load a 64-bit addition).
__device__ __forceinline__ unsigned lane_offset(unsigned o) {
  asm volatile("" : "+v"(o));
  return o;
}

// Loads the group at t of page `id`; returns whether the page is one of the cache's. A group
// that is not there is read from page 0 and never used.
// (`part` 1: keys only, 2: values only.)
template <int HD, bool EXACT>
__device__ __forceinline__ int load_group(const Attn &p, int id, int h, int t, int lane, Group<HD> &x,
                                          int part = 3) {
  // uniform base addresses and unsigned lane offsets
  const unsigned i = lane & 15, quad = lane >> 4, l = lane;
  const unsigned nb = EXACT ? HD / 16 : (unsigned)p.hd >> 4;  // blocks of a row
  const int ok = id >= 0 && id < p.pages;
  const int64_t row = (((int64_t)(ok ? id : 0) * p.kv_heads + h) << p.page_shift) +
                      (t & ((1 << p.page_shift) - 1));
  typedef const GLOBAL uint8_t *Bytes;
  Bytes kc = (Bytes)(p.kc + row * (nb * 8)), ks = (Bytes)(p.ks + row * nb);
  Bytes vc = (Bytes)(p.vc + row * (nb * 8)), vs = (Bytes)(p.vs + row * nb);
  const unsigned kq = HD == 64 ? 0 : HD == 128 ? quad & 2 : quad * 4;
  const unsigned vq = HD == 64 ? 0 : HD == 128 ? l & 2 : (l & 3) * 4;
  if (part & 1) {
    if (EXACT) {
      const unsigned ko = lane_offset(i * (nb * 8) + quad * (HD / 8));
      if constexpr (HD == 64) {
        const u2 a = *(const GLOBAL u2 *)(kc + ko);
        x.k[0] = a.x, x.k[1] = a.y;
      } else {
#pragma unroll
        for (int w = 0; w < HD / 128; ++w) {
          const u4 a = *(const GLOBAL u4 *)(kc + ko + 16 * w);
          x.k[4 * w] = a.x, x.k[4 * w + 1] = a.y, x.k[4 * w + 2] = a.z, x.k[4 * w + 3] = a.w;
        }
      }
      const unsigned kso = lane_offset(i * nb + (HD == 128 ? kq * 2 : kq));
      x.ks = *(const GLOBAL unsigned *)(ks + kso);
    } else {
      x.ks = 0;
#pragma unroll
      for (unsigned w = 0; w < HD / 64; ++w) {
        const unsigned b = quad * (HD / 64) + w;
        u2 a = (u2){0, 0};
        if (b < nb) {
          a = *(const GLOBAL u2 *)(kc + (i * nb + b) * 8);
          x.ks |= (unsigned)ks[i * nb + b] << (8 * w);
        }
        x.k[2 * w] = a.x, x.k[2 * w + 1] = a.y;
      }
    }
  }
  if (part & 2) {
    if (EXACT) {
      const unsigned vso = lane_offset((l >> 2) * nb + (HD == 128 ? vq * 2 : vq));
      x.vs = *(const GLOBAL unsigned *)(vs + vso);
    } else {
      x.vs = 0;
#pragma unroll
      for (unsigned w = 0; w < HD / 64; ++w) {
        const unsigned c = (l & 3) * (HD / 64) + w;
        if (c < nb) x.vs |= (unsigned)vs[(l >> 2) * nb + c] << (8 * w);
      }
    }
    const bool in = EXACT || (int)(i * (HD / 16)) < p.hd;
    const unsigned vo = lane_offset(4 * quad * (nb * 8) + i * (HD / 32));
#pragma unroll
    for (unsigned e = 0; e < 4; ++e) {
      const Bytes v = vc + e * (nb * 8);
      x.v[e][0] = 0;
      if constexpr (HD > 128) x.v[e][1] = 0;
      if (in) {
        if constexpr (HD == 64) x.v[e][0] = *(const GLOBAL uint16_t *)(v + vo);
        else if constexpr (HD == 128) x.v[e][0] = *(const GLOBAL unsigned *)(v + vo);
        else {
          const u2 a = *(const GLOBAL u2 *)(v + vo);
          x.v[e][0] = a.x, x.v[e][1] = a.y;
        }
      }
    }
  }
  return ok;
}

// Key operands of a group: out[s] holds eight channels of the lane's token, contraction step s.
template <int HD, bool EXACT>
__device__ __forceinline__ void key_frags(const Group<HD> &x, int lane, h8 *out) {
  h2 sc[more(HD / 128)];
#pragma unroll
  for (int k = 0; k < more(HD / 128); ++k) sc[k] = scales2(scale_bits<HD, EXACT>(x.ks, lane >> 4), k);
#pragma unroll
  for (int s = 0; s < HD / 32; ++s) {
    const _Float16 f = (s >> 1) & 1 ? sc[s >> 2][1] : sc[s >> 2][0];
    const h2 two = {f, f};
    union { h8 v; h2 p[4]; } r;
#pragma unroll
    for (int b = 0; b < 4; ++b) r.p[b] = codes2(x.k[s], b) * two;
    out[s] = r.v;
  }
}

// Value scales of a group as fp16, transposed through LDS to [block][token]: 20 halves a row so
// that the eight-byte reads of a half wave fall on different banks.
constexpr int kVsRow = 20;

template <int HD, bool EXACT>
__device__ __forceinline__ void stage_value_scales(const Group<HD> &x, int lane, _Float16 *lds) {
  const int tok = lane >> 2, b0 = (lane & 3) * (HD / 64);
#pragma unroll
  for (int w = 0; w < more(HD / 128); ++w) {
    const h2 s = scales2(scale_bits<HD, EXACT>(x.vs, lane & 3), w);
    lds[(b0 + 2 * w) * kVsRow + tok] = s[0];
    if (HD > 64) lds[(b0 + 2 * w + 1) * kVsRow + tok] = s[1];
  }
}

__device__ __forceinline__ void order_wave_lds() {
  // data from other lanes of the wave: order the reads after their writes
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Scales of the lane's four value tokens, in pairs.
template <int HD>
__device__ __forceinline__ void value_scales(int lane, const _Float16 *lds, h2 *sc) {
  const h4 s = *reinterpret_cast<const h4 *>(lds + (((lane & 15) * (HD / 16)) >> 4) * kVsRow + 4 * (lane >> 4));
  sc[0] = (h2){s[0], s[1]}, sc[1] = (h2){s[2], s[3]};
}

// The codes of token pair e (0 or 1), interleaved nibble by nibble: byte b of `even` holds
// channel 2 b of both tokens, of `odd` channel 2 b + 1, so that one convert gives a pair.
template <int HD>
__device__ __forceinline__ void value_nibbles(const Group<HD> &x, int e, int word, unsigned &even,
                                              unsigned &odd) {
  const unsigned a = x.v[2 * e][word], b = x.v[2 * e + 1][word];
  even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
  odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}

// Value operands of a group: out[c] holds channel i HD/16 + c of the lane's four tokens.
template <int HD>
__device__ __forceinline__ void value_frags(const Group<HD> &x, int lane, const _Float16 *lds, h4 *out) {
  h2 sc[2];
  value_scales<HD>(lane, lds, sc);
  constexpr int C = HD >= 128 ? 8 : HD / 16;  // channels of a word
#pragma unroll
  for (int word = 0; word < more(HD / 128); ++word) {
    union { h4 v; h2 p[2]; } r[C];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      unsigned even, odd;
      value_nibbles(x, e, word, even, odd);
#pragma unroll
      for (int c = 0; c < C; ++c) r[c].p[e] = codes2(c & 1 ? odd : even, c >> 1) * sc[e];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) out[8 * word + c] = r[c].v;
  }
}

template <bool F32>
__device__ __forceinline__ void store_out(void *out, int64_t e, float a, float b) {
  if (F32) *reinterpret_cast<float2 *>(static_cast<float *>(out) + e) = make_float2(a, b);
  else *reinterpret_cast<unsigned *>(static_cast<uint16_t *>(out) + e) = bf16x2_bits(a, b);
}

template <bool F32>
__device__ __forceinline__ void store4(void *out, int64_t e, f4 y) {
  if (F32) *reinterpret_cast<f4 *>(static_cast<float *>(out) + e) = y;
  else *reinterpret_cast<u2 *>(static_cast<uint16_t *>(out) + e) =
      (u2){bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3])};
}

// ---------------------------------------------------------------- query rows of a wave

// Probabilities are held times 2^base over the running maximum's, and the maximum is raised
// when one passes 2^16, fp16's range. The row's largest is held at 2^base or more, so what is
// smaller than 2^-32 of it (2^-38 for fp32 q) is lost under fp16's smallest step.
constexpr float base_of(bool f32) { return f32 ? 13.0f : 7.0f; }

// 16 NT query rows: lane (i, quad) serves row 16 n + i of each tile n.
template <int HD, int NT, bool F32>
struct Rows {
  h8 q[NT][F32 ? 2 : 1][HD / 32];  // fp16 halves: channels quad HD/4 + 8 s ..
  float c[NT];                     // score times c = log2 of the unnormalised probability
  float off[NT];                   // base - running maximum (log2); +inf before the first token
  float l[NT];                     // this lane's share of the sum of the probabilities
  int lim[NT];                     // the first token that the row does not see
  f4 acc[NT][HD / 16];             // channel (4 quad + r) HD/16 + d of row i in acc[n][d][r]
};

// Issue the loads of the lane's share of the rows; use_rows makes operands of them when other
// loads are on their way too.
template <int HD, int NT, bool F32>
struct RawRows {
  u4 q[NT][HD / 32][F32 ? 2 : 1];
};

// lim[n]: the first token of the job that the lane's row of tile n does not see.
template <int NT>
__device__ __forceinline__ void row_ends(const Attn &p, const Job &j, int r0, int rows, int i, int *lim) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = min(r0 + 16 * n + i, rows - 1) / p.group;
    lim[n] = j.causal ? min(j.len, j.len - j.nq + tok + 1) : j.len;
  }
}

template <int HD, int NT, bool F32, bool EXACT>
__device__ __forceinline__ void load_rows(const Attn &p, const Job &j, int h, int r0, int rows,
                                          int lane, RawRows<HD, NT, F32> &y, Rows<HD, NT, F32> &x) {
  const int i = lane & 15, quad = lane >> 4;
  row_ends<NT>(p, j, r0, rows, i, x.lim);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = min(r0 + 16 * n + i, rows - 1);
    const int tok = r / p.group, head = h * p.group + (r - tok * p.group);
    const int64_t at = (int64_t)(j.q0 + tok) * p.q_ts + head * p.q_hs + quad * (HD / 4);
#pragma unroll
    for (int s = 0; s < HD / 32; ++s)
#pragma unroll
      for (int w = 0; w < (F32 ? 2 : 1); ++w) {
        y.q[n][s][w] = (u4){0, 0, 0, 0};
        if (EXACT || quad * (HD / 4) + 8 * s < p.hd)
          y.q[n][s][w] = F32 ? *reinterpret_cast<const u4 *>(static_cast<const float *>(p.q) + at + 8 * s + 4 * w)
                             : *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(p.q) + at + 8 * s);
      }
  }
}

template <int HD, int NT, bool F32>
__device__ __forceinline__ void use_rows(const RawRows<HD, NT, F32> &y, float scale, Rows<HD, NT, F32> &x) {
  const float sign = scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float v[HD / 4], amax = 0.0f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (F32) v[8 * s + e] = __uint_as_float(y.q[n][s][F32 ? e >> 2 : 0][e & 3]);
        else v[8 * s + e] = e & 1 ? bf16_hi(y.q[n][s][0][e >> 1]) : bf16_lo(y.q[n][s][0][e >> 1]);
        amax = fmaxf(amax, fabsf(v[8 * s + e]));
      }
    amax = fmaxf(amax, xor16(amax));
    amax = fmaxf(amax, xor32(amax));
    float inv;
    const float f = row_factor(amax, inv) * (amax < INFINITY ? sign : NAN);  // infinite: all scores NaN
    x.c[n] = fmaxf(fabsf(scale) * inv, 1e-37f);  // positive, so a hidden score stays -inf
    x.off[n] = INFINITY;
    x.l[n] = 0.0f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = v[8 * s + e] * f;
        const _Float16 hi = (_Float16)z;
        x.q[n][0][s][e] = hi;
        if (F32) x.q[n][F32 ? 1 : 0][s][e] = (_Float16)(z - (float)hi);
      }
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) x.acc[n][d] = (f4){0, 0, 0, 0};
  }
}

// Rows r0 .. r1 - 1 all see the tokens below lo, and none sees one from hi on.
__device__ __forceinline__ void row_limits(const Attn &p, const Job &j, int r0, int r1, int &lo,
                                           int &hi) {
  lo = hi = j.len;
  if (j.causal) {
    lo = min(j.len, max(0, j.len - j.nq + r0 / p.group + 1));
    hi = min(j.len, max(0, j.len - j.nq + (r1 - 1) / p.group + 1));
  }
}

// Scores of hidden tokens of the tile at t: -inf.
template <int NT>
__device__ __forceinline__ void hide(f4 (*s)[2], const int *lim, int t, int t1, int ok, int quad) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tt = t + 16 * u + 4 * quad + r;
        if (tt >= lim[n] || tt >= t1 || !((ok >> u) & 1)) s[n][u][r] = -INFINITY;
      }
}

// exp2(score c + off) as fp16 (two halves for fp32 q), the second product's operand; returns
// the sum of the lane's eight before that rounding.
template <bool F32>
__device__ __forceinline__ float exponentials(const f4 *s, float c, float off, h8 *pf) {
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][r], c, off));
      sum += e;
      const _Float16 hi = (_Float16)e;
      pf[0][4 * u + r] = hi;
      if (F32) pf[F32 ? 1 : 0][4 * u + r] = (_Float16)(e - (float)hi);
    }
  return sum;
}

// Scores of a 32-token tile to probabilities, held times 2^base over the running maximum's. No
// maximum is taken while a lane's eight sum to less than fp16's range (before the first
// visible token the offset is +inf, and the sum infinite or NaN); only then is the maximum
// raised and everything so far rescaled.
template <int HD, int NT, bool F32>
__device__ __forceinline__ void probabilities(f4 (*s)[2], Rows<HD, NT, F32> &x, h8 (*pf)[F32 ? 2 : 1]) {
  constexpr float kBase = base_of(F32);
  float sum[NT];
  bool fits = true;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    sum[n] = exponentials<F32>(s[n], x.c[n], x.off[n], pf[n]);
    fits = fits && sum[n] < 65504.0f;
  }
  if (!__all(fits)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                       fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3]))) * x.c[n];
      mx = fmaxf(mx, xor16(mx));
      mx = fmaxf(mx, xor32(mx));
      const float m = kBase - x.off[n];  // -inf before the first visible token
      const float to = fmaxf(m, mx);
      const bool none = to == -INFINITY;
      const float a = none ? 1.0f : __builtin_amdgcn_exp2f(m - to);
      x.off[n] = kBase - to;
      x.l[n] *= a;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) x.acc[n][d] *= a;
      sum[n] = exponentials<F32>(s[n], x.c[n], none ? 0.0f : x.off[n], pf[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) x.l[n] += sum[n];
}

// Rows r0 .. r0 + n - 1 (n <= 16) of a sequence whose own sums are in LDS: row i's channels at
// own[i (HD + 4)], its maximum and sum in m[i] and l[i]. Adds the prefix's pieces and writes out:
// HD / 4 lanes take four channels each, and groups of such lanes share a row's pieces.
template <int HD, bool F32, int W>
__device__ __forceinline__ void finish_rows(const Attn &p, const Job &j, int h, int r0, int n, float S_v,
                                            float *own, const float *m, const float *l) {
  constexpr int LANES = HD / 4, GROUPS = 64 * W / LANES, OROW = HD + 4;
  f4 *so = reinterpret_cast<f4 *>(own + 16 * OROW);  // [GROUPS][LANES], behind the own sums
  float *sml = own + 16 * OROW + GROUPS * HD;        // [GROUPS][2]
  const List &k0 = p.list[0].prefix ? p.list[0] : p.list[1];
  const int slots = k0.slots, g = threadIdx.x / LANES, c = threadIdx.x % LANES;
  int per = GROUPS;
  while (per > 1 && per * n > GROUPS) per >>= 1;
  const int64_t rows = (int64_t)p.tokens * p.group, step = rows * p.kv_heads;
  for (int i0 = 0; i0 < n; i0 += GROUPS / per) {
    const int i = i0 + g / per, sub = g & (per - 1);
    const bool here = i < n, in = here && 4 * c < p.hd;
    const int64_t at = h * rows + (int64_t)j.q0 * p.group + r0 + i;
    float M = -INFINITY, L = 0.0f;
    f4 y = {0, 0, 0, 0};
    if (here && sub == 0) {
      M = m[i], L = l[i];
      if (in) y = *reinterpret_cast<const f4 *>(own + i * OROW + 4 * c);
    }
#pragma unroll 4
    for (int k = sub; k < (here ? slots : 0); k += per) {
      const float2 ml = k0.ml[at + k * step];
      f4 o = {0, 0, 0, 0};
      if (in) o = *reinterpret_cast<const f4 *>(k0.opart + (at + k * step) * p.hd + 4 * c);
      if (ml.y != 0.0f) {
        const float to = fmaxf(M, ml.x);
        const float a = __builtin_amdgcn_exp2f(M - to), e = __builtin_amdgcn_exp2f(ml.x - to);
        M = to;
        L = L * a + ml.y * e;
        y = y * a + o * e;
      }
    }
    if (c == 0) sml[2 * g] = M, sml[2 * g + 1] = L;
    so[g * LANES + c] = y;
    __syncthreads();
    if (here && sub == 0) {
      for (int k = 1; k < per; ++k) M = fmaxf(M, sml[2 * (g + k)]);
      L = 0.0f;
      y = (f4){0, 0, 0, 0};
      for (int k = 0; k < per; ++k) {
        if (sml[2 * (g + k) + 1] == 0.0f) continue;
        const float e = __builtin_amdgcn_exp2f(sml[2 * (g + k)] - M);
        L += sml[2 * (g + k) + 1] * e;
        y += so[(g + k) * LANES + c] * e;
      }
      const int r = r0 + i, tok = r / p.group, head = h * p.group + (r - tok * p.group);
      const int64_t to = (int64_t)(j.q0 + tok) * p.heads + head;
      if (in) store4<F32>(p.out, to * p.hd + 4 * c, y * out_factor(S_v, L));
      if (c == 0 && p.lse) p.lse[to] = row_lse(M, L);
    }
    __syncthreads();
  }
}

// W waves take the 32-token tiles of a piece in turn, each for the same 16 NT query rows, and
// join their sums at the end.
template <int HD, int NT, bool F32, bool EXACT, int W>
__global__ void __launch_bounds__(64 * W, NT == 1 && HD <= 128 && !F32 ? 4 : 1) k_kv_attn_rows(Attn p) {
  constexpr int HALVES = F32 ? 2 : 1, DV = HD / 16, OROW = HD + 4;
  constexpr float kBase = base_of(F32);
  __shared__ __align__(16) float smem[W * 16 * OROW];
  __shared__ __align__(16) _Float16 vs_lds[W][2][DV * kVsRow];
  __shared__ float sm_m[W][16 * NT], sm_l[W][16 * NT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, quad = lane >> 4;
  Share sh;
  if (!share_of(p, lane, sh)) return;
  const Job j = sh.j;
  const int h = sh.h, rows = j.nq * p.group, r0 = sh.rt * (16 * NT), t0 = sh.t0;
  if (r0 >= rows) return;
  const float S_k = p.S_k[h], S_v = p.S_v[h];
  int t1 = sh.t1;

  int lim_lo, lim_hi;
  row_limits(p, j, r0, min(r0 + 16 * NT, rows), lim_lo, lim_hi);
  t1 = min(t1, lim_hi);

  Group<HD> g[2], nxt[2];  // raw codes: this tile's, and the next one's on their way
  int ok = 0, nxt_ok = 0;
  Pages pg = open_pages(j, p.page_shift, t0, t1, lane);
  Rows<HD, NT, F32> x;
  int t = t0 + 32 * wave;
  {
    RawRows<HD, NT, F32> raw;
    load_rows<HD, NT, F32, EXACT>(p, j, h, r0, rows, lane, raw, x);
    __builtin_amdgcn_sched_barrier(0);
    if (t < t1) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        ok |= load_group<HD, EXACT>(p, page_of(pg, t + 16 * u), h, t + 16 * u, lane, g[u]) << u;
    }
    __builtin_amdgcn_sched_barrier(0);
    use_rows<HD, NT, F32>(raw, p.scale * kLog2e * S_k, x);
  }
  for (; t < t1; advance(pg, j, p.page_shift, t1, lane))
  for (const int te = min(t1, pg.t + kRun); t < te; t += 32 * W) {  // the tiles of a run
    if (t + 32 * W < t1) {
      nxt_ok = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tt = t + 32 * W + 16 * u;
        nxt_ok |= load_group<HD, EXACT>(p, page_of(pg, tt), h, tt, lane, nxt[u]) << u;
      }
    }
    f4 s[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      stage_value_scales<HD, EXACT>(g[u], lane, vs_lds[wave][u]);
      h8 kf[HD / 32];
      key_frags<HD, EXACT>(g[u], lane, kf);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][u] = (f4){0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < HD / 32; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < HALVES; ++q)
            s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[k], x.q[n][q][k], s[n][u], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);  // one group's operands at a time: registers
    }
    order_wave_lds();
    if (t + 32 > lim_lo || ok != 3) hide<NT>(s, x.lim, t, t1, ok, quad);
    h8 pf[NT][HALVES];
    probabilities<HD, NT, F32>(s, x, pf);
    __builtin_amdgcn_sched_barrier(0);
    // as value_frags, two channels of all eight tokens at a time
    h2 sc[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) value_scales<HD>(lane, vs_lds[wave][u], sc[u]);
#pragma unroll
    for (int word = 0; word < more(HD / 128); ++word) {
      unsigned even[4], odd[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) value_nibbles(g[e >> 1], e & 1, word, even[e], odd[e]);
#pragma unroll
      for (int c = 0; c < (HD >= 128 ? 8 : HD / 16); ++c) {
        union { h8 v; h2 p[4]; } a;
#pragma unroll
        for (int e = 0; e < 4; ++e) a.p[e] = codes2(c & 1 ? odd[e] : even[e], c >> 1) * sc[e >> 1][e & 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < HALVES; ++q)
            x.acc[n][8 * word + c] =
                __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v, pf[n][q], x.acc[n][8 * word + c], 0, 0, 0);
        if (c & 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
    order_wave_lds();
#pragma unroll
    for (int u = 0; u < 2; ++u) g[u] = nxt[u];
    ok = nxt_ok;
  }

  // join the waves
  const int64_t part = part_of(p, sh);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    x.l[n] += xor16(x.l[n]);
    x.l[n] += xor32(x.l[n]);
    if (quad == 0) sm_m[wave][16 * n + i] = kBase - x.off[n], sm_l[wave][16 * n + i] = x.l[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) M = fmaxf(M, sm_m[k][16 * n + i]);
    const float m = kBase - x.off[n];
    const float a = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
    if (n) __syncthreads();
    float *o = smem + (wave * 16 + i) * OROW;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int d = 0; d < DV; ++d) o[DV * (4 * quad + r) + d] = x.acc[n][d][r] * a;
    __syncthreads();
    // 4 W lanes a row, pairs of channels
    const int row = threadIdx.x / (4 * W), col = threadIdx.x % (4 * W), r = r0 + 16 * n + row;
    const bool finish = NT == 1 && p.list[sh.list].finish > 0;
    float mm = -INFINITY, ll = 0.0f;
    if (r < rows) {
#pragma unroll
      for (int k = 0; k < W; ++k) mm = fmaxf(mm, sm_m[k][16 * n + row]);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float mk = sm_m[k][16 * n + row];
        if (sm_l[k][16 * n + row] != 0.0f) ll += sm_l[k][16 * n + row] * __builtin_amdgcn_exp2f(mk - mm);
      }
      const int tok = r / p.group, head = h * p.group + (r - tok * p.group);
      const int64_t at = (int64_t)(j.q0 + tok) * p.heads + head;
      const float f = sh.direct ? out_factor(S_v, ll) : 1.0f;
      for (int d = 2 * col; d < p.hd; d += 8 * W) {
        f2 y = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < W; ++k) y += *reinterpret_cast<const f2 *>(smem + (k * 16 + row) * OROW + d);
        if (finish) *reinterpret_cast<f2 *>(smem + row * OROW + d) = y;  // read by this lane alone
        else if (sh.direct) store_out<F32>(p.out, at * p.hd + d, y[0] * f, y[1] * f);
        else *reinterpret_cast<f2 *>(p.list[sh.list].opart + (part + r) * p.hd + d) = y;
      }
      if (col == 0 && !finish) {
        if (sh.direct) {
          if (p.lse) p.lse[at] = row_lse(mm - kBase, ll);
        } else {
          p.list[sh.list].ml[part + r] = make_float2(mm - kBase, ll);
        }
      }
    }
    if (finish) {
      __syncthreads();  // sm_m and sm_l have been read
      if (col == 0) sm_m[0][row] = mm - kBase, sm_l[0][row] = ll;
      __syncthreads();
      finish_rows<HD, F32, W>(p, j, h, r0, min(16, rows - r0), S_v, smem, sm_m[0], sm_l[0]);
    }
  }
}

// Many query rows over one token list (a shared prefix, a prompt): each of W waves holds 16 NT
// rows. A stage is 16 W tokens: every wave dequantises a group of 16 into LDS, as ready MFMA
// operands in lane order (bank conflicts in 3% of the cycles), and all waves read all tiles. Two stages
// are in LDS, so the next one is dequantised beside the products of this one by whichever
// wave comes to it. Score products run at a raised wave priority: of a SIMD's two waves, one in
// its products then goes ahead of one in its exponentials, which fills the gaps between
// them (456 -> 433 us on two 2048-query chunks; at both products the same, at the second alone
// in between). Eight waves: four (half the rows a dequantised group serves) take 495 us. Matrix
// instructions hold the SIMDs for 43% of the time and vector instructions (exponentials,
// dequantising) issue for 46% of it, so what is left to overlap is small. With `lead` the rows go over the prefix and then over their own tokens, and nothing is left to join.
template <int HD, int NT, bool F32, bool EXACT, int W>
__global__ void __launch_bounds__(64 * W, 2) k_kv_attn_tile(Attn p) {
  // Groups of a stage. At HD 256 LDS holds half as many: of eight waves two take a group, one its
  // keys, one its values, against four waves on a SIMD each: 2000 x 4000 queries 229 -> 169 us. In
  // fp32 eight cost 172 us against 152 (2 x 1000 x 3000): four.
  constexpr int GS = HD > 128 && W > 4 ? W / 2 : W, STAGE = 16 * GS;
  constexpr int HALVES = F32 ? 2 : 1, DV = HD / 16, KS = HD / 32;
  __shared__ h8 kfrag[2][GS][KS][64], vfrag[2][GS / 2][DV][64];
  __shared__ __align__(16) _Float16 vs_lds[GS][DV * kVsRow];
  __shared__ int oks[2][GS];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, quad = lane >> 4;
  Share sh;
  if (!share_of(p, lane, sh)) return;
  Job j = sh.j;
  const int h = sh.h, rows = j.nq * p.group, R0 = sh.rt * (16 * NT * W);
  if (R0 >= rows) return;
  const float S_k = p.S_k[h], S_v = p.S_v[h];
  const int r0 = R0 + wave * 16 * NT;

  // the token list in hand, and what of it the wave's rows see
  int t0 = sh.t0, t1 = sh.t1, lim_lo, lim_hi;
  bool lead = p.lead_len > 0;
  if (lead) j.pages = p.lead, j.len = p.lead_len, j.causal = 0, t0 = 0, t1 = p.lead_len;
  Pages pg;
  const auto open = [&]() {
    int none;
    row_limits(p, j, R0, min(R0 + 16 * NT * W, rows), none, lim_hi);
    t1 = min(t1, lim_hi);
    row_limits(p, j, min(r0, rows - 1), min(r0 + 16 * NT, rows), lim_lo, lim_hi);
    if (r0 >= rows) lim_hi = 0;  // a wave without rows only dequantises
    pg = open_pages(j, p.page_shift, t0, t1, lane);
  };
  open();
  Group<HD> g;
  int ok = 0;
  const int mine = wave % GS, part_kv = GS == W ? 3 : 1 + wave / GS;
  const auto fetch = [&](int t) {  // this wave's group of the stage at t
    t += 16 * mine;
    ok = load_group<HD, EXACT>(p, page_of(pg, t), h, t, lane, g, part_kv);
  };
  const auto dequantise = [&](int b) {
    if (part_kv & 2) stage_value_scales<HD, EXACT>(g, lane, vs_lds[mine]);
    if (part_kv & 1) {
      if (lane == 0) oks[b][mine] = ok;
      h8 kf[KS];
      key_frags<HD, EXACT>(g, lane, kf);
#pragma unroll
      for (int k = 0; k < KS; ++k) kfrag[b][mine][k][lane] = kf[k];
    }
    if (part_kv & 2) {
      order_wave_lds();
      h4 vf[DV];
      value_frags<HD>(g, lane, vs_lds[mine], vf);
#pragma unroll
      for (int d = 0; d < DV; ++d)
        reinterpret_cast<h4 *>(&vfrag[b][mine >> 1][d][lane])[mine & 1] = vf[d];
      order_wave_lds();
    }
  };
  Rows<HD, NT, F32> x;
  {
    RawRows<HD, NT, F32> raw;
    load_rows<HD, NT, F32, EXACT>(p, j, h, r0, rows, lane, raw, x);
    __builtin_amdgcn_sched_barrier(0);
    if (t0 < t1) fetch(t0);
    __builtin_amdgcn_sched_barrier(0);
    use_rows<HD, NT, F32>(raw, p.scale * kLog2e * S_k, x);
  }
  for (;;) {
    if (t0 < t1) {
      dequantise(0);
      if (t0 + STAGE < t1) fetch(t0 + STAGE);
    }
    __syncthreads();
    int b = 0;
    for (int t = t0; t < t1; advance(pg, j, p.page_shift, t1, lane))
    for (const int te = min(t1, pg.t + kRun); t < te; t += STAGE, b ^= 1) {  // the stages of a run
      // operands are read one step ahead of their products: the values' before the exponentials,
      // the next tile's keys before the second product
      // (at HD 256 they would not fit beside the sums)
      constexpr bool AHEAD = HD <= 128;
      const int tiles = min(GS / 2, (min(t1, lim_hi) - t + 31) >> 5);
      h8 kf[AHEAD ? 2 * KS : 1];
      if constexpr (AHEAD) {
  #pragma unroll
        for (int k = 0; k < 2 * KS; ++k) kf[k] = kfrag[b][k / KS][k % KS][lane];
      }
  #pragma unroll 1
      for (int c = 0; c < tiles; ++c) {
        const int tt = t + 32 * c;
        __builtin_amdgcn_s_setprio(1);
        f4 s[NT][2];
  #pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = (f4){0, 0, 0, 0};
  #pragma unroll
        for (int k = 0; k < KS; ++k)
  #pragma unroll
          for (int u = 0; u < 2; ++u) {
            const h8 a = AHEAD ? kf[AHEAD ? u * KS + k : 0] : kfrag[b][2 * c + u][k][lane];
  #pragma unroll
            for (int n = 0; n < NT; ++n)
  #pragma unroll
              for (int q = 0; q < HALVES; ++q)
                s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, x.q[n][q][k], s[n][u], 0, 0, 0);
          }
        h8 vf[AHEAD ? DV : 1];
        if constexpr (AHEAD) {
  #pragma unroll
          for (int d = 0; d < DV; ++d) vf[d] = vfrag[b][c][d][lane];
        }
        const int seen = __builtin_amdgcn_readfirstlane(oks[b][2 * c] | oks[b][2 * c + 1] << 1);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        if (tt + 32 > lim_lo || seen != 3) hide<NT>(s, x.lim, tt, t1, seen, quad);
        h8 pf[NT][HALVES];
        probabilities<HD, NT, F32>(s, x, pf);
        if constexpr (AHEAD) {
          const int nc = min(c + 1, GS / 2 - 1);
  #pragma unroll
          for (int k = 0; k < 2 * KS; ++k) kf[k] = kfrag[b][2 * nc + k / KS][k % KS][lane];
          __builtin_amdgcn_sched_barrier(0);
        }
  #pragma unroll
        for (int d = 0; d < DV; ++d) {
          const h8 a = AHEAD ? vf[AHEAD ? d : 0] : vfrag[b][c][d][lane];
  #pragma unroll
          for (int n = 0; n < NT; ++n)
  #pragma unroll
            for (int q = 0; q < HALVES; ++q)
              x.acc[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pf[n][q], x.acc[n][d], 0, 0, 0);
        }
      }
      if (t + STAGE < t1) {
        dequantise(b ^ 1);
        if (t + 2 * STAGE < t1) fetch(t + 2 * STAGE);
      }
      __syncthreads();
    }
    if (!lead) break;
    lead = false, j = sh.j, t0 = sh.t0, t1 = sh.t1;  // the own tokens
    open();
    row_ends<NT>(p, j, r0, rows, i, x.lim);
    if (t0 < t1) fetch(t0);
  }

  // each lane holds HD/16 consecutive channels of its row four times
  const int64_t part = part_of(p, sh);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float l = x.l[n];
    l += xor16(l);
    l += xor32(l);
    const int r = r0 + 16 * n + i;
    if (r >= rows) continue;
    const int tok = r / p.group, head = h * p.group + (r - tok * p.group);
    const int64_t at = (int64_t)(j.q0 + tok) * p.heads + head;
    const float f = sh.direct ? out_factor(S_v, l) : 1.0f;
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int ch = DV * (4 * quad + r4);
      if (EXACT || ch < p.hd) {
#pragma unroll
        for (int d = 0; d < DV; d += 4) {
          const f4 y = {x.acc[n][d][r4] * f, x.acc[n][d + 1][r4] * f, x.acc[n][d + 2][r4] * f,
                        x.acc[n][d + 3][r4] * f};
          if (sh.direct)
            store4<F32>(p.out, at * p.hd + ch + d, y);
          else
            *reinterpret_cast<f4 *>(p.list[sh.list].opart + (part + r) * p.hd + ch + d) = y;
        }
      }
    }
    if (quad == 0) {
      if (sh.direct) {
        if (p.lse) p.lse[at] = row_lse(-x.off[n], l);
      } else {
        p.list[sh.list].ml[part + r] = make_float2(-x.off[n], l);
      }
    }
  }
}

// Join the partial sums of the rows: HD / 4 lanes take four channels each; of a workgroup's
// groups of such lanes `per` (join_per) share a row and take its pieces in turn. The prefix's pieces come first, then those of the sequence's own tokens.
struct Join {
  const float *opart, *opart_own, *S_v;
  const float2 *ml, *ml_own;
  void *out;
  float *lse;
  const int32_t *q_offsets, *kv_lens;
  const int2 *where;  // NULL: one piece a sequence
  int tokens, heads, kv_heads, group, hd, max_q, n_prefix, per;
};

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

// ---------------------------------------------------------------- launch

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
