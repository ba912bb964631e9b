// Rotary positions, and the append to the key/value cache that turns keys on the way.
//
// Both take (token, head) rows. The lanes of a row own its pairs, so the cosines and sines of a lane
// are the same for every head: a lane computes its own once, in 64 bits, and goes over the heads.
#include "nvfp4_device.h"
#include "nvfp4_rotary.h"
#include "nvfp4_rows.h"

namespace nvfp4 {

// ---------------------------------------------------------------- angles

// c = fp32(factor cos(p w)), s = fp32(factor sin(p w)), each from 64 bits. The product is kept as a
// sum of two doubles; it is reduced by multiples of pi/2 (pi/2 too in two doubles) to |r| <= pi/4,
// where the Taylor sums to r^15 and r^14 are off by less than 1e-15.
__device__ __forceinline__ void turn_of(double p, double w, double factor, float &c, float &s) {
  const double a = p * w, low = __builtin_fma(p, w, -a);
  const double n = __builtin_rint(a * 0.63661977236758134308);
  double r = __builtin_fma(-n, 1.57079632679489661923, a);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r) + low;
  const double z = r * r;
  double si = -1.0 / 1307674368000.0;
  si = __builtin_fma(si, z, 1.0 / 6227020800.0);
  si = __builtin_fma(si, z, -1.0 / 39916800.0);
  si = __builtin_fma(si, z, 1.0 / 362880.0);
  si = __builtin_fma(si, z, -1.0 / 5040.0);
  si = __builtin_fma(si, z, 1.0 / 120.0);
  si = __builtin_fma(si, z, -1.0 / 6.0);
  si = __builtin_fma(si * z, r, r);
  double co = -1.0 / 87178291200.0;
  co = __builtin_fma(co, z, 1.0 / 479001600.0);
  co = __builtin_fma(co, z, -1.0 / 3628800.0);
  co = __builtin_fma(co, z, 1.0 / 40320.0);
  co = __builtin_fma(co, z, -1.0 / 720.0);
  co = __builtin_fma(co, z, 1.0 / 24.0);
  co = __builtin_fma(co, z, -0.5);
  co = __builtin_fma(co, z, 1.0);
  // quarter turns: n mod 4 without passing 32 bits
  const int quarter = (int)(n - 4.0 * __builtin_floor(0.25 * n));
  const double x = quarter & 1 ? si : co, y = quarter & 1 ? co : si;
  c = (float)((quarter == 1 || quarter == 2 ? -x : x) * factor);
  s = (float)((quarter >= 2 ? -y : y) * factor);
}

__device__ __forceinline__ double position_of(const Turn &r, int pair, int64_t t) {
  const int a = r.axis ? r.axis[pair] : 0;
  return a >= 0 && a < r.axes ? (double)r.positions[a * r.stride + t] : 0.0;
}

// ---------------------------------------------------------------- rotate

template <int DT, int V>
__device__ __forceinline__ void load_values(const void *x, int64_t e, float *v) {
  if constexpr (V == 8) {
    load8<DT>(x, e, v);
  } else if (DT == NVFP4_DTYPE_BF16) {
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + e);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  } else {
    const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + e);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
}
template <int DT, int V>
__device__ __forceinline__ void store_values(void *x, int64_t e, const float *v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (DT == NVFP4_DTYPE_BF16)
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(x) + e + i) =
          make_uint2(bf16x2_bits(v[i], v[i + 1]), bf16x2_bits(v[i + 2], v[i + 3]));
    else
      *reinterpret_cast<float4 *>(static_cast<float *>(x) + e + i) =
          make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

struct Rotate {
  Turn turn;
  const void *x;
  void *out;
  int64_t ts, hs, out_ts, out_hs, tokens;
  int heads, head_dim, transpose;
};

// A lane's V pairs of a row (2 V channels): pairs V u .. of the turned part, or 2 V channels that
// pass through.
template <int DT, int V, bool ADJACENT>
__device__ __forceinline__ void rotate_rows(const Rotate &p, int64_t t, int u, int h0, int h1) {
  float c[V], s[V];
  const bool turned = u < p.turn.pairs / V;
  const int a = !turned || ADJACENT ? 2 * V * u : V * u, b = !turned || ADJACENT ? a + V : a + p.turn.pairs;
  if (turned) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      turn_of(position_of(p.turn, V * u + i, t), p.turn.inv_freq[V * u + i], p.turn.factor, c[i], s[i]);
      if (p.transpose) s[i] = -s[i];
    }
  }
  for (int h = h0; h < h1; ++h) {
    const int64_t e = t * p.ts + h * p.hs, o = t * p.out_ts + h * p.out_hs;
    float x[2 * V], y[2 * V];
    load_values<DT, V>(p.x, e + a, x);
    load_values<DT, V>(p.x, e + b, x + V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int i0 = ADJACENT ? 2 * i : i, i1 = ADJACENT ? 2 * i + 1 : V + i;
      y[i0] = turned ? x[i0] * c[i] - x[i1] * s[i] : x[i0];
      y[i1] = turned ? x[i1] * c[i] + x[i0] * s[i] : x[i1];
    }
    store_values<DT, V>(p.out, o + a, y);
    store_values<DT, V>(p.out, o + b, y + V);
  }
}

template <int DT, int V, bool ADJACENT>
__global__ void __launch_bounds__(256) k_rotate(Rotate p) {
  const int lanes = p.head_dim / (2 * V), rows = 256 / lanes;
  const int row = threadIdx.x / lanes, u = threadIdx.x - row * lanes;
  const int64_t t = (int64_t)blockIdx.x * rows + row;
  if (row >= rows || t >= p.tokens) return;
  rotate_rows<DT, V, ADJACENT>(p, t, u, 0, p.heads);
}

int launch_rotate(const Turn &turn, bool adjacent, bool transpose, const RowSpan &x,
                  const RowSpan &out, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                  hipStream_t st) {
  const Rotate p = {turn,   x.x,    const_cast<void *>(out.x), x.ts,          x.hs,
                    out.ts, out.hs, tokens,                    (int)heads, (int)head_dim, transpose};
  const int v = turn.pairs % 8 || head_dim % 16 ? 4 : 8;
  const int64_t rows = 256 / (head_dim / (2 * v));
  const dim3 g((unsigned)((tokens + rows - 1) / rows)), b(256);
  const auto go = [&](auto dt, auto vv) {
    if (adjacent) hipLaunchKernelGGL((k_rotate<dt.value, vv.value, true>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_rotate<dt.value, vv.value, false>), g, b, 0, st, p);
  };
  const auto with = [&](auto dt) {
    if (v == 8) go(dt, std::integral_constant<int, 8>{});
    else go(dt, std::integral_constant<int, 4>{});
  };
  if (dtype == NVFP4_DTYPE_BF16) with(std::integral_constant<int, NVFP4_DTYPE_BF16>{});
  else with(std::integral_constant<int, NVFP4_DTYPE_F32>{});
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- append

struct Append {
  Rotate q;
  Turn turn;
  const void *x[2];
  int64_t ts[2], hs[2];
  uint8_t *codes[2], *scales[2];
  const float *S[2];
  const int64_t *slots;
  int64_t n_slots, tokens;
  int kv_heads, head_dim, page_shift;
};

// The block of 16 channels from ch of key row e, turned: y = x c - other s, with the block's own
// cosines and signed sines.
template <int DT, bool ADJACENT>
__device__ __forceinline__ void load_turned(const Append &p, int64_t e, int ch, const float *c,
                                            const float *s, float *y) {
  float x[16], other[16];
  load8<DT>(p.x[0], e + ch, x);
  load8<DT>(p.x[0], e + ch + 8, x + 8);
#pragma unroll
  for (int j = 0; j < 16; j += 8) {
    if (ADJACENT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) other[j + i] = ch + j < 2 * p.turn.pairs ? x[j + (i ^ 1)] : 0.0f;
    } else if (ch + j < 2 * p.turn.pairs) {
      load8<DT>(p.x[0], e + ch + j + (ch + j < p.turn.pairs ? p.turn.pairs : -p.turn.pairs), other + j);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) other[j + i] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i] * c[i] - other[i] * s[i];
}

template <int DT, bool ADJACENT>
__global__ void __launch_bounds__(256) k_kv_append(Append p) {
  const int lanes = p.head_dim >> 4, rows = 256 / lanes;
  const int row = threadIdx.x / lanes, part = threadIdx.x - row * lanes;
  const int64_t t = (int64_t)blockIdx.x * rows + row;
  if (row >= rows || t >= p.tokens) return;
  if (blockIdx.y == 2) {
    rotate_rows<DT, 8, ADJACENT>(p.q, t, part, 0, p.q.heads);
    return;
  }
  const int kv = blockIdx.y, ch = part * 16;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) return;
  float c[16], s[16];
  if (kv == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int P = p.turn.pairs, d = ch + i;
      const int pair = ADJACENT ? d >> 1 : d < P ? d : d - P;
      c[i] = 1.0f, s[i] = 0.0f;
      if (d < 2 * P) turn_of(position_of(p.turn, pair, t), p.turn.inv_freq[pair], p.turn.factor, c[i], s[i]);
      if (ADJACENT ? d & 1 : d >= P) s[i] = -s[i];
    }
  }
  const int64_t page = slot >> p.page_shift, offset = slot & (((int64_t)1 << p.page_shift) - 1);
  for (int h = 0; h < p.kv_heads; ++h) {
    const float S = p.S[kv][h];
    const int64_t e = t * p.ts[kv] + h * p.hs[kv];
    float v[16];
    if (kv == 0) {
      load_turned<DT, ADJACENT>(p, e, ch, c, s, v);
    } else {
      load8<DT>(p.x[1], e + ch, v);
      load8<DT>(p.x[1], e + ch + 8, v + 8);
    }
    float lo6, hi6;
    recip_bracket(6.0 * (double)S, lo6, hi6);
    uint2 codes;
    const int byte = quantise16(v, lo6, hi6, S, codes);
    const int64_t at = ((page * p.kv_heads + h) << p.page_shift) + offset;
    reinterpret_cast<uint2 *>(p.codes[kv])[at * lanes + part] = codes;
    p.scales[kv][at * lanes + part] = (uint8_t)byte;
  }
}

int launch_kv_append(const nvfp4_kv_cache &c, const Turn &turn, bool adjacent, const RowSpan &q,
                     const RowSpan &q_out, const RowSpan &k, const RowSpan &v, int dtype,
                     int64_t tokens, int64_t heads, const int64_t *slots, hipStream_t st) {
  Append p;
  p.q = {turn,     q.x,      const_cast<void *>(q_out.x), q.ts,       q.hs,
         q_out.ts, q_out.hs, tokens,                      (int)heads, (int)c.head_dim, 0};
  p.turn = turn;
  p.x[0] = k.x, p.x[1] = v.x, p.ts[0] = k.ts, p.ts[1] = v.ts, p.hs[0] = k.hs, p.hs[1] = v.hs;
  p.codes[0] = c.k_codes, p.codes[1] = c.v_codes;
  p.scales[0] = c.k_scales, p.scales[1] = c.v_scales;
  p.S[0] = c.S_k, p.S[1] = c.S_v;
  p.slots = slots, p.tokens = tokens, p.n_slots = c.pages * c.page_size;
  p.kv_heads = (int)c.kv_heads, p.head_dim = (int)c.head_dim;
  p.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  const int64_t rows = 256 / (c.head_dim / 16);
  const dim3 g((unsigned)((tokens + rows - 1) / rows), heads ? 3 : 2), b(256);
  if (dtype == NVFP4_DTYPE_BF16) {
    if (adjacent) hipLaunchKernelGGL((k_kv_append<NVFP4_DTYPE_BF16, true>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_kv_append<NVFP4_DTYPE_BF16, false>), g, b, 0, st, p);
  } else {
    if (adjacent) hipLaunchKernelGGL((k_kv_append<NVFP4_DTYPE_F32, true>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_kv_append<NVFP4_DTYPE_F32, false>), g, b, 0, st, p);
  }
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
