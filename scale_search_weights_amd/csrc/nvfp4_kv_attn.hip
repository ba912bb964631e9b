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
// Running maximum: it is raised (and the sums rescaled) only when a score exceeds it by more
// than 2^kLazy; until then probabilities may exceed 1, which fp16 holds. A wave rescales a
// few times per sequence instead of once per tile.
#include "nvfp4_device.h"
#include "nvfp4_kv.h"

namespace nvfp4 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Attn {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *S_k, *S_v;
  const void *q;
  int64_t q_ts, q_hs;
  const int32_t *q_offsets, *table, *kv_lens;
  int64_t table_width;
  int tokens, heads, kv_heads, group, hd, page_shift, pages, max_q, max_len, causal;
  float scale;
  int prefix;               // the job is the shared prefix: all tokens over one page list
  int piece, pieces, row_tiles, slot0, direct;
  void *out;
  float *lse, *opart;
  float2 *ml;
};

// One sequence's share of the call.
struct Job {
  int q0, nq, len, causal;
  const int32_t *pages;
};

__device__ __forceinline__ Job job_of(const Attn &p, int b) {
  Job j;
  if (p.prefix) {
    j.q0 = 0, j.nq = p.tokens, j.len = p.max_len, j.causal = 0, j.pages = p.table;
  } else {
    int lo = b * p.max_q, hi = lo + p.max_q;
    if (p.q_offsets) {
      lo = min(max(p.q_offsets[b], 0), p.tokens);
      hi = min(max(p.q_offsets[b + 1], lo), min(p.tokens, lo + p.max_q));
    }
    j.q0 = lo, j.nq = hi - lo;
    j.len = p.kv_lens ? min(max(p.kv_lens[b], 0), p.max_len) : 0;
    j.causal = p.causal;
    j.pages = p.table + b * p.table_width;
  }
  return j;
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

// ---------------------------------------------------------------- raw tiles of 32 tokens

template <int HD>
struct Tile {
  unsigned k[2][HD / 32];                 // lane's HD/4 key codes of token i, two 16-token halves
  unsigned ks[2];                         // their HD/64 scale bytes
  unsigned v[8][HD > 128 ? HD / 128 : 1]; // lane's HD/16 value codes of its eight tokens
  unsigned vs[HD > 128 ? HD / 128 : 1];   // HD/32 value scale bytes of token lane / 2
  int ok;                                 // bit u: half u lies in a page of the cache
};

template <int HD, bool EXACT>
__device__ __forceinline__ void load_tile(const Attn &p, const Job &j, int h, int t, int t_end,
                                          int lane, Tile<HD> &x) {
  const int i = lane & 15, quad = lane >> 4;
  const int nb = EXACT ? HD / 16 : p.hd >> 4;  // blocks of a row
  int64_t row[2];
  x.ok = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tb = t + 16 * u;
    int id = 0;
    if (tb < t_end) {
      id = j.pages[tb >> p.page_shift];
      if (id >= 0 && id < p.pages) x.ok |= 1 << u;
      else id = 0;
    }
    // rows of a half that is not there are read from page 0 and never used
    row[u] = ((int64_t)id * p.kv_heads + h) << p.page_shift;
    row[u] += tb & ((1 << p.page_shift) - 1);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t *kc = p.kc + row[u] * (nb * 8), *ks = p.ks + row[u] * nb;
    const uint8_t *vc = p.vc + row[u] * (nb * 8);
    if (EXACT) {
      const unsigned *k = reinterpret_cast<const unsigned *>(kc + i * (nb * 8) + quad * (HD / 8));
      if constexpr (HD == 64) {
        const uint2 a = *reinterpret_cast<const uint2 *>(k);
        x.k[u][0] = a.x, x.k[u][1] = a.y;
        x.ks[u] = ks[i * nb + quad];
      } else {
#pragma unroll
        for (int w = 0; w < HD / 128; ++w) {
          const uint4 a = *reinterpret_cast<const uint4 *>(k + 4 * w);
          x.k[u][4 * w] = a.x, x.k[u][4 * w + 1] = a.y, x.k[u][4 * w + 2] = a.z, x.k[u][4 * w + 3] = a.w;
        }
        if constexpr (HD == 128) x.ks[u] = *reinterpret_cast<const uint16_t *>(ks + i * nb + 2 * quad);
        else x.ks[u] = *reinterpret_cast<const unsigned *>(ks + i * nb + 4 * quad);
      }
    } else {
      x.ks[u] = 0;
#pragma unroll
      for (int w = 0; w < HD / 64; ++w) {
        const int b = quad * (HD / 64) + w;
        uint2 a = make_uint2(0, 0);
        if (b < nb) {
          a = *reinterpret_cast<const uint2 *>(kc + (i * nb + b) * 8);
          x.ks[u] |= (unsigned)ks[i * nb + b] << (8 * w);
        }
        x.k[u][2 * w] = a.x, x.k[u][2 * w + 1] = a.y;
      }
    }
    const bool in = EXACT || i * (HD / 16) < p.hd;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t *v = vc + (4 * quad + e) * (nb * 8) + i * (HD / 32);
      unsigned *to = x.v[4 * u + e];
      to[0] = 0;
      if constexpr (HD > 128) to[1] = 0;
      if (in) {
        if constexpr (HD == 64) to[0] = *reinterpret_cast<const uint16_t *>(v);
        else if constexpr (HD == 128) to[0] = *reinterpret_cast<const unsigned *>(v);
        else {
          const uint2 a = *reinterpret_cast<const uint2 *>(v);
          to[0] = a.x, to[1] = a.y;
        }
      }
    }
  }
  // value scales: lane / 2 is the token, each lane half of its blocks
  const int64_t vrow = (lane < 32 ? row[0] : row[1]) + ((lane >> 1) & 15);
  const uint8_t *vs = p.vs + vrow * nb;
  if (EXACT) {
    vs += (lane & 1) * (HD / 32);
    if constexpr (HD == 64) x.vs[0] = *reinterpret_cast<const uint16_t *>(vs);
    else if constexpr (HD == 128) x.vs[0] = *reinterpret_cast<const unsigned *>(vs);
    else {
      const uint2 a = *reinterpret_cast<const uint2 *>(vs);
      x.vs[0] = a.x, x.vs[1] = a.y;
    }
  } else {
#pragma unroll
    for (int w = 0; w < (HD > 128 ? HD / 128 : 1); ++w) x.vs[w] = 0;
#pragma unroll
    for (int w = 0; w < HD / 32; ++w) {
      const int b = (lane & 1) * (HD / 32) + w;
      if (b < nb) x.vs[w >> 2] |= (unsigned)vs[b] << (8 * (w & 3));
    }
  }
}

// Key operand of contraction step s for one 16-token half: eight channels of the lane's token.
template <int HD>
__device__ __forceinline__ h8 key_step(const Tile<HD> &x, int u, int s, const h2 *ksc) {
  const h2 two = ksc[s >> 2];
  const _Float16 f = (s >> 1) & 1 ? two[1] : two[0];
  const h2 sc = {f, f};
  const unsigned w = x.k[u][s];
  union { h8 v; h2 p[4]; } r;
#pragma unroll
  for (int b = 0; b < 4; ++b) r.p[b] = codes2(w, b) * sc;
  return r.v;
}

// Value scales of a tile as fp16, transposed through LDS to [block][token]: 36 halves a row so
// that the eight-byte reads of a half wave fall on different banks.
constexpr int kVsRow = 36;

template <int HD>
__device__ __forceinline__ void stage_value_scales(const Tile<HD> &x, int lane, _Float16 *lds) {
  const int tok = lane >> 1, b0 = (lane & 1) * (HD / 32);
#pragma unroll
  for (int w = 0; w < HD / 64; ++w) {
    const h2 s = scales2(x.vs[w >> 1], w & 1);
    lds[(b0 + 2 * w) * kVsRow + tok] = s[0];
    lds[(b0 + 2 * w + 1) * kVsRow + tok] = s[1];
  }
}

// Value operands: out[c] holds channel i HD/16 + c of the lane's eight tokens. The codes of
// two tokens are interleaved nibble by nibble first, so that one convert gives a pair of
// tokens of one channel.
template <int HD>
__device__ __forceinline__ void value_frags(const Tile<HD> &x, int lane, const _Float16 *lds,
                                            int word, h8 *out) {
  const int i = lane & 15, quad = lane >> 4;
  const _Float16 *row = lds + ((i * (HD / 16)) >> 4) * kVsRow + 4 * quad;
  union { uint2 w[2]; h2 s[4]; } sc;
  sc.w[0] = *reinterpret_cast<const uint2 *>(row);
  sc.w[1] = *reinterpret_cast<const uint2 *>(row + 16);
  constexpr int C = HD >= 128 ? 8 : HD / 16;  // channels of a word
  union { h8 v; h2 p[4]; } r[C];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned a = x.v[2 * e][word], b = x.v[2 * e + 1][word];
    const unsigned even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    const unsigned odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      r[c].p[e] = codes2(even, c >> 1) * sc.s[e];
      r[c + 1].p[e] = codes2(odd, c >> 1) * sc.s[e];
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) out[c] = r[c].v;
}

template <bool F32>
__device__ __forceinline__ void store_out(void *out, int64_t e, float a, float b) {
  if (F32) *reinterpret_cast<float2 *>(static_cast<float *>(out) + e) = make_float2(a, b);
  else *reinterpret_cast<unsigned *>(static_cast<uint16_t *>(out) + e) = bf16x2_bits(a, b);
}

// Four waves take the 32-token tiles of a piece in turn, each for the same 16 NT query rows,
// and join their sums at the end.
template <int HD, int NT, bool F32, bool EXACT>
__global__ void __launch_bounds__(256) k_kv_attn_rows(Attn p) {
  constexpr int HALVES = F32 ? 2 : 1;        // fp16 halves of q and p
  constexpr float kLazy = F32 ? 2.0f : 8.0f; // log2
  // probabilities are held times 2^kBase, at most 2^15: what is smaller than 2^-32 of the
  // largest (2^-38 for fp32 q) is lost under fp16's smallest step
  constexpr float kBase = F32 ? 13.0f : 7.0f;
  constexpr int DV = HD / 16, OROW = HD + 4;
  __shared__ __align__(16) float smem[4 * 16 * OROW];
  __shared__ _Float16 vs_lds[4][DV * kVsRow];
  __shared__ float sm_m[4][16 * NT], sm_l[4][16 * NT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, quad = lane >> 4;
  int w = blockIdx.x;
  const int piece = w % p.pieces;
  w /= p.pieces;
  const int rt = w % p.row_tiles;
  w /= p.row_tiles;
  const int h = w % p.kv_heads;
  const Job j = job_of(p, w / p.kv_heads);
  const int rows = j.nq * p.group, r0 = rt * (16 * NT);
  if (r0 >= rows) return;
  int t0 = piece * p.piece, t1 = min(j.len, t0 + p.piece);
  if (t0 >= t1 && !p.direct) return;

  // query rows: operands, score factors and the first token each may not see
  h8 qf[NT][HALVES][HD / 32];
  float c[NT], m[NT], l[NT];
  int lim[NT];
  f4 acc[NT][DV];
  int lim_lo = j.len, lim_hi = j.len;
  if (j.causal) {
    lim_lo = min(j.len, max(0, j.len - j.nq + r0 / p.group + 1));
    lim_hi = min(j.len, max(0, j.len - j.nq + (min(r0 + 16 * NT, rows) - 1) / p.group + 1));
  }
  t1 = min(t1, lim_hi);
  const float sc = p.scale * kLog2e * p.S_k[h];
  const float sign = sc < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = min(r0 + 16 * n + i, rows - 1);
    const int tok = r / p.group, head = h * p.group + (r - tok * p.group);
    lim[n] = j.causal ? min(j.len, j.len - j.nq + tok + 1) : j.len;
    const int64_t at = (int64_t)(j.q0 + tok) * p.q_ts + head * p.q_hs + quad * (HD / 4);
    float v[HD / 4], amax = 0.0f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      if (EXACT || quad * (HD / 4) + 8 * s < p.hd) {
        if (F32) {
          const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at + 8 * s);
          const float4 a = f[0], b = f[1];
          v[8 * s] = a.x, v[8 * s + 1] = a.y, v[8 * s + 2] = a.z, v[8 * s + 3] = a.w;
          v[8 * s + 4] = b.x, v[8 * s + 5] = b.y, v[8 * s + 6] = b.z, v[8 * s + 7] = b.w;
        } else {
          const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at + 8 * s);
          v[8 * s] = bf16_lo(a.x), v[8 * s + 1] = bf16_hi(a.x), v[8 * s + 2] = bf16_lo(a.y);
          v[8 * s + 3] = bf16_hi(a.y), v[8 * s + 4] = bf16_lo(a.z), v[8 * s + 5] = bf16_hi(a.z);
          v[8 * s + 6] = bf16_lo(a.w), v[8 * s + 7] = bf16_hi(a.w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * s + e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[8 * s + e]));
    }
    amax = fmaxf(amax, xor16(amax));
    amax = fmaxf(amax, xor32(amax));
    float inv;
    const float f = row_factor(amax, inv) * sign;
    c[n] = fmaxf(fabsf(sc) * inv, 1e-37f);  // positive, so a hidden score stays -inf
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = v[8 * s + e] * f;
        const _Float16 hi = (_Float16)y;
        qf[n][0][s][e] = hi;
        if (F32) qf[n][HALVES - 1][s][e] = (_Float16)(y - (float)hi);
      }
#pragma unroll
    for (int d = 0; d < DV; ++d) acc[n][d] = (f4){0, 0, 0, 0};
  }

  Tile<HD> cur, nxt;
  int t = t0 + 32 * wave;
  if (t < t1) load_tile<HD, EXACT>(p, j, h, t, t1, lane, cur);
  for (; t < t1; t += 128) {
    if (t + 128 < t1) load_tile<HD, EXACT>(p, j, h, t + 128, t1, lane, nxt);
    stage_value_scales<HD>(cur, lane, vs_lds[wave]);
    f4 s[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      h2 ksc[HD / 128 > 0 ? HD / 128 : 1];
#pragma unroll
      for (int k = 0; k < (HD / 128 > 0 ? HD / 128 : 1); ++k) ksc[k] = scales2(cur.ks[u], k);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][u] = (f4){0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) {
        const h8 a = key_step<HD>(cur, u, k, ksc);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < HALVES; ++q)
            s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qf[n][q][k], s[n][u], 0, 0, 0);
      }
    }
    if (t + 32 > lim_lo || cur.ok != 3) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int tt = t + 16 * u + 4 * quad + r;
            if (tt >= lim[n] || tt >= t1 || !((cur.ok >> u) & 1)) s[n][u][r] = -INFINITY;
          }
    }
    h8 pf[NT][HALVES];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                       fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3]))) * c[n];
      if (__any(mx > m[n] + kLazy)) {
        mx = fmaxf(mx, xor16(mx));
        mx = fmaxf(mx, xor32(mx));
        const float to = fmaxf(m[n], mx);
        const float a = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[n] - to);
        m[n] = to;
        l[n] *= a;
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[n][d] *= a;
      }
      const float base = (m[n] == -INFINITY ? 0.0f : m[n]) - kBase;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][u][r], c[n], -base));
          l[n] += e;
          const _Float16 hi = (_Float16)e;
          pf[n][0][4 * u + r] = hi;
          if (F32) pf[n][HALVES - 1][4 * u + r] = (_Float16)(e - (float)hi);
        }
    }
#pragma unroll
    for (int word = 0; word < (HD > 128 ? HD / 128 : 1); ++word) {
      constexpr int C = HD >= 128 ? 8 : HD / 16;
      h8 a[C];
      value_frags<HD>(cur, lane, vs_lds[wave], word, a);
#pragma unroll
      for (int d = 0; d < C; ++d)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < HALVES; ++q)
            acc[n][8 * word + d] =
                __builtin_amdgcn_mfma_f32_16x16x32_f16(a[d], pf[n][q], acc[n][8 * word + d], 0, 0, 0);
    }
    cur = nxt;
  }

  // join the four waves
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += xor16(l[n]);
    l[n] += xor32(l[n]);
    if (quad == 0) sm_m[wave][16 * n + i] = m[n], sm_l[wave][16 * n + i] = l[n];
  }
  __syncthreads();
  const float S_v = p.S_v[h];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) M = fmaxf(M, sm_m[k][16 * n + i]);
    const float a = m[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[n] - M);
    if (n) __syncthreads();
    float *o = smem + (wave * 16 + i) * OROW;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int d = 0; d < DV; ++d) o[DV * (4 * quad + r) + d] = acc[n][d][r] * a;
    __syncthreads();
    // sixteen lanes a row, pairs of channels
    const int row = threadIdx.x >> 4, r = r0 + 16 * n + row;
    if (r < rows) {
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) mm = fmaxf(mm, sm_m[k][16 * n + row]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float mk = sm_m[k][16 * n + row];
        if (mk != -INFINITY) ll += sm_l[k][16 * n + row] * __builtin_amdgcn_exp2f(mk - mm);
      }
      const int tok = r / p.group, head = h * p.group + (r - tok * p.group);
      const int64_t at = (int64_t)(j.q0 + tok) * p.heads + head;
      const float f = p.direct ? (ll > 0.0f ? S_v / ll : 0.0f) : 1.0f;
      for (int d = 2 * (threadIdx.x & 15); d < p.hd; d += 32) {
        float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 z = *reinterpret_cast<const float2 *>(smem + (k * 16 + row) * OROW + d);
          y.x += z.x, y.y += z.y;
        }
        if (p.direct)
          store_out<F32>(p.out, at * p.hd + d, y.x * f, y.y * f);
        else
          *reinterpret_cast<float2 *>(
              p.opart + (((int64_t)(p.slot0 + piece) * p.tokens * p.heads + at) * p.hd + d)) = y;
      }
      if ((threadIdx.x & 15) == 0) {
        if (p.direct) {
          if (p.lse) p.lse[at] = ll > 0.0f ? kLn2 * (mm - kBase + __builtin_amdgcn_logf(ll)) : -INFINITY;
        } else {
          p.ml[(int64_t)(p.slot0 + piece) * p.tokens * p.heads + at] = make_float2(mm - kBase, ll);
        }
      }
    }
  }
}

// Join the partial sums of a row: one wave per (token, head). Slots 0 .. n_prefix - 1 are the
// prefix's pieces, then those of the sequence's own tokens.
struct Join {
  const float *opart, *S_v;
  const float2 *ml;
  void *out;
  float *lse;
  const int32_t *q_offsets, *kv_lens;
  int tokens, heads, group, hd, max_q, max_len, n_prefix, piece;
};

template <bool F32>
__global__ void __launch_bounds__(256) k_kv_attn_join(Join p) {
  const int lane = threadIdx.x & 63, b = blockIdx.y;
  const int idx = blockIdx.x * 4 + ((int)threadIdx.x >> 6);
  const int i = idx / p.heads, head = idx - i * p.heads;
  int lo = b * p.max_q, hi = lo + p.max_q;
  if (p.q_offsets) {
    lo = min(max(p.q_offsets[b], 0), p.tokens);
    hi = min(max(p.q_offsets[b + 1], lo), min(p.tokens, lo + p.max_q));
  }
  if (lo + i >= hi) return;
  int n = p.n_prefix;
  if (p.kv_lens) {
    const int len = min(max(p.kv_lens[b], 0), p.max_len);
    n += (len + p.piece - 1) / p.piece;
  }
  const int64_t rows = (int64_t)p.tokens * p.heads, at = (int64_t)(lo + i) * p.heads + head;
  float M = -INFINITY, L = 0.0f;
  for (int k = lane; k < n; k += 64) M = fmaxf(M, p.ml[k * rows + at].x);
#pragma unroll
  for (int off = 32; off; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
  const float S = p.S_v[head / p.group];
  float2 y[2] = {};  // head_dim <= 256
  const int d = 2 * lane;
  for (int k0 = 0; k0 < n; k0 += 64) {
    float2 mine = make_float2(-INFINITY, 0.0f);
    if (k0 + lane < n) mine = p.ml[(k0 + lane) * rows + at];
    const float wgt = mine.y > 0.0f ? __builtin_amdgcn_exp2f(mine.x - M) : 0.0f;
    float part = mine.y * wgt;
#pragma unroll
    for (int off = 32; off; off >>= 1) part += __shfl_xor(part, off, 64);
    L += part;
    const int end = min(64, n - k0);
    for (int k = 0; k < end; ++k) {
      const float a = __shfl(wgt, k, 64);
      if (a == 0.0f) continue;  // the same for the wave: the piece may be unwritten
      const float *o = p.opart + ((k0 + k) * rows + at) * p.hd;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (d + 128 * s < p.hd) {
          const float2 z = *reinterpret_cast<const float2 *>(o + d + 128 * s);
          y[s].x = __builtin_fmaf(a, z.x, y[s].x), y[s].y = __builtin_fmaf(a, z.y, y[s].y);
        }
    }
  }
  const float f = L > 0.0f ? S / L : 0.0f;
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (d + 128 * s < p.hd) store_out<F32>(p.out, at * p.hd + d + 128 * s, y[s].x * f, y[s].y * f);
  if (lane == 0 && p.lse) p.lse[at] = L > 0.0f ? kLn2 * (M + __builtin_amdgcn_logf(L)) : -INFINITY;
}

// ---------------------------------------------------------------- plan and launch

namespace {

struct Part {  // one launch: the prefix or the sequences' own tokens
  int nt, row_tiles, piece, pieces;
};

struct Plan {
  Part prefix, own;
  int max_len;
};

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pieces so that about `want` workgroups run, each at least 128 tokens (a tile for each wave).
Part plan_part(const KvAttention &a, int64_t rows, int64_t jobs, int64_t len) {
  Part r;
  const int top = a.cache->head_dim > 128 ? 2 : (a.dtype == NVFP4_DTYPE_F32 ? 2 : 4);
  r.nt = rows <= 16 ? 1 : (rows <= 32 || top == 2 ? 2 : 4);
  r.row_tiles = (int)cdiv(rows, 16 * r.nt);
  const int64_t units = jobs * a.cache->kv_heads * r.row_tiles;
  const int64_t want = 2048;
  int64_t pieces = cdiv(want, units);
  int64_t piece = cdiv(cdiv(len, pieces), 128) * 128;
  if (piece < 128) piece = 128;
  r.piece = (int)piece;
  r.pieces = (int)(len > 0 ? cdiv(len, piece) : 1);
  return r;
}

Plan plan_of(const KvAttention &a) {
  Plan p;
  const int64_t G = a.heads / a.cache->kv_heads;
  p.max_len = (int)a.max_kv;
  p.prefix = Part{0, 0, 0, 0};
  p.own = Part{0, 0, 0, 0};
  if (a.prefix_len > 0) p.prefix = plan_part(a, a.tokens * G, 1, a.prefix_len);
  if (a.max_kv > 0 || a.prefix_len == 0) p.own = plan_part(a, a.max_q * G, a.batch, a.max_kv);
  return p;
}

template <int HD, bool F32, bool EXACT>
void launch_rows(const Attn &p, int nt, unsigned grid, hipStream_t st) {
  const dim3 g(grid), b(256);
  if (nt == 1) hipLaunchKernelGGL((k_kv_attn_rows<HD, 1, F32, EXACT>), g, b, 0, st, p);
  else if (nt == 2) hipLaunchKernelGGL((k_kv_attn_rows<HD, 2, F32, EXACT>), g, b, 0, st, p);
  else if constexpr (HD <= 128 && !F32)
    hipLaunchKernelGGL((k_kv_attn_rows<HD, 4, F32, EXACT>), g, b, 0, st, p);
}

template <int HD, bool F32>
void launch_exact(const Attn &p, int nt, unsigned grid, hipStream_t st) {
  if (p.hd == HD) launch_rows<HD, F32, true>(p, nt, grid, st);
  else launch_rows<HD, F32, false>(p, nt, grid, st);
}

template <bool F32>
void launch_hd(const Attn &p, int nt, unsigned grid, hipStream_t st) {
  if (p.hd <= 64) launch_exact<64, F32>(p, nt, grid, st);
  else if (p.hd <= 128) launch_exact<128, F32>(p, nt, grid, st);
  else launch_exact<256, F32>(p, nt, grid, st);
}

int64_t part_grid(const KvAttention &a, const Part &r, int64_t jobs) {
  return jobs * a.cache->kv_heads * r.row_tiles * r.pieces;
}

}  // namespace

bool kv_attention_fits(const KvAttention &a) {
  const Plan p = plan_of(a);
  return part_grid(a, p.prefix, 1) <= INT32_MAX && part_grid(a, p.own, a.batch) <= INT32_MAX;
}

size_t kv_attention_workspace_size(const KvAttention &a) {
  const Plan p = plan_of(a);
  const int64_t slots = p.prefix.pieces + p.own.pieces;
  if (slots <= 1) return 0;
  return (size_t)(slots * a.tokens * a.heads * (a.cache->head_dim * 4 + 8));
}

int launch_kv_attention(const KvAttention &a, hipStream_t st) {
  const Plan plan = plan_of(a);
  const nvfp4_kv_cache &c = *a.cache;
  const int slots = plan.prefix.pieces + plan.own.pieces;
  const int64_t rows = a.tokens * a.heads;
  Attn p = {};
  p.kc = c.k_codes, p.ks = c.k_scales, p.vc = c.v_codes, p.vs = c.v_scales;
  p.S_k = c.S_k, p.S_v = c.S_v;
  p.q = a.q, p.q_ts = a.q_ts, p.q_hs = a.q_hs, p.q_offsets = a.q_offsets, p.kv_lens = a.kv_lens;
  p.tokens = (int)a.tokens, p.heads = (int)a.heads, p.kv_heads = (int)c.kv_heads;
  p.group = (int)(a.heads / c.kv_heads), p.hd = (int)c.head_dim;
  p.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  p.pages = (int)c.pages, p.max_q = (int)a.max_q, p.scale = a.scale;
  p.direct = slots <= 1;
  p.out = a.out, p.lse = a.lse;
  p.opart = static_cast<float *>(a.workspace);
  p.ml = reinterpret_cast<float2 *>(p.opart + (size_t)slots * rows * c.head_dim);
  const bool f32 = a.dtype == NVFP4_DTYPE_F32;
  if (plan.prefix.pieces) {
    Attn x = p;
    x.prefix = 1, x.table = a.prefix_pages, x.max_len = (int)a.prefix_len;
    x.piece = plan.prefix.piece, x.pieces = plan.prefix.pieces, x.row_tiles = plan.prefix.row_tiles;
    const unsigned g = (unsigned)part_grid(a, plan.prefix, 1);
    if (f32) launch_hd<true>(x, plan.prefix.nt, g, st);
    else launch_hd<false>(x, plan.prefix.nt, g, st);
  }
  if (plan.own.pieces) {
    Attn x = p;
    x.table = a.block_table, x.table_width = a.table_width, x.max_len = plan.max_len;
    x.causal = a.causal, x.slot0 = plan.prefix.pieces;
    x.piece = plan.own.piece, x.pieces = plan.own.pieces, x.row_tiles = plan.own.row_tiles;
    const unsigned g = (unsigned)part_grid(a, plan.own, a.batch);
    if (f32) launch_hd<true>(x, plan.own.nt, g, st);
    else launch_hd<false>(x, plan.own.nt, g, st);
  }
  if (slots > 1) {
    Join x = {};
    x.opart = p.opart, x.ml = p.ml, x.S_v = c.S_v, x.out = a.out, x.lse = a.lse;
    x.q_offsets = a.q_offsets, x.kv_lens = a.kv_lens;
    x.tokens = p.tokens, x.heads = p.heads, x.group = p.group, x.hd = p.hd, x.max_q = p.max_q;
    x.max_len = plan.max_len, x.n_prefix = plan.prefix.pieces, x.piece = plan.own.piece;
    const dim3 g((unsigned)cdiv(a.max_q * a.heads, 4), (unsigned)a.batch);
    if (f32) hipLaunchKernelGGL(k_kv_attn_join<true>, g, dim3(256), 0, st, x);
    else hipLaunchKernelGGL(k_kv_attn_join<false>, g, dim3(256), 0, st, x);
  }
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
