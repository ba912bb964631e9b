// Key/value cache in NVFP4: quantise rows into cache slots, and read slots back.
//
// Both kernels take (token, head) rows of head_dim values, eight values per lane (half a
// block), so a row is head_dim / 8 lanes and a workgroup of 256 takes 256 / (head_dim / 8) rows
// of one head: its tensor scale is uniform, and consecutive tokens of a page are contiguous
// in the cache, so a workgroup's stores join into whole lines. They are bound by memory: write
// moves 2 or 4 bytes in and 9/16 out per value, read the reverse.
#include "nvfp4_device.h"
#include "nvfp4_kv.h"

namespace nvfp4 {

// maximum with the other lane of a pair (lanes 2i, 2i + 1)
__device__ __forceinline__ float pair_max(float x) {
  const int o = __builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xF, 0xF, true);
  return fmaxf(x, __int_as_float(o));
}

template <int DT>
__device__ __forceinline__ void load8(const void *x, int64_t e, float v[8]) {
  if (DT == NVFP4_DTYPE_BF16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + e);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + e);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

struct KvWrite {
  const void *x[2];
  int64_t ts[2], hs[2];
  uint8_t *codes[2], *scales[2];
  const float *S[2];
  const int64_t *slots;
  int64_t tokens, n_slots;
  int heads, head_dim, page_shift;
};

template <int DT>
__global__ void __launch_bounds__(256) k_kv_write(KvWrite p) {
  const int kv = blockIdx.z, h = blockIdx.y;
  const int lanes = p.head_dim >> 3, rows = 256 / lanes;
  const int row = threadIdx.x / lanes, part = threadIdx.x - row * lanes;
  if (row >= rows) return;  // whole lane pairs: lanes is even
  const float S = p.S[kv][h];
  float lo6, hi6;
  recip_bracket(6.0 * (double)S, lo6, hi6);
  const int64_t mask = ((int64_t)1 << p.page_shift) - 1;
  for (int64_t t = (int64_t)blockIdx.x * rows + row; t < p.tokens; t += (int64_t)gridDim.x * rows) {
    const int64_t slot = p.slots[t];
    if (slot < 0 || slot >= p.n_slots) continue;  // the same for the whole row
    float v[8];
    load8<DT>(p.x[kv], t * p.ts[kv] + h * p.hs[kv] + part * 8, v);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = pair_max(amax);
    const int b = max_scale_byte_fast(amax, lo6, hi6, S);
    unsigned c = 0u;
    if (b) {
      const double sS = e4m3_value_d(b) * (double)S;
      float lo, hi;
      recip_bracket(sS, lo, hi);
      c = fp4_clear_neg_zero(fp4_exact_codes8(v, lo, hi, sS));
    }
    const int64_t at = ((((slot >> p.page_shift) * p.heads + h) << p.page_shift) + (slot & mask));
    reinterpret_cast<unsigned *>(p.codes[kv])[at * lanes + part] = c;
    if (!(part & 1)) p.scales[kv][at * (lanes >> 1) + (part >> 1)] = (uint8_t)b;
  }
}

static int page_shift_of(const nvfp4_kv_cache &c) { return __builtin_ctzll((unsigned long long)c.page_size); }

static dim3 row_grid(int64_t tokens, int64_t heads, int64_t head_dim, int z) {
  const int64_t rows = 256 / (head_dim / 8);
  int64_t g = (tokens + rows - 1) / rows;
  int64_t cap = 65536 / (heads * z);  // rows beyond are taken in a loop
  if (cap < 64) cap = 64;
  return dim3((unsigned)(g < cap ? g : cap), (unsigned)heads, (unsigned)z);
}

int launch_kv_write(const nvfp4_kv_cache &c, const void *k, const void *v, int dtype,
                    int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                    const int64_t *slots, hipStream_t st) {
  KvWrite p;
  p.x[0] = k, p.x[1] = v;
  p.ts[0] = k_ts, p.ts[1] = v_ts, p.hs[0] = k_hs, p.hs[1] = v_hs;
  p.codes[0] = c.k_codes, p.codes[1] = c.v_codes;
  p.scales[0] = c.k_scales, p.scales[1] = c.v_scales;
  p.S[0] = c.S_k, p.S[1] = c.S_v;
  p.slots = slots, p.tokens = tokens, p.n_slots = c.pages * c.page_size;
  p.heads = (int)c.kv_heads, p.head_dim = (int)c.head_dim, p.page_shift = page_shift_of(c);
  const dim3 g = row_grid(tokens, c.kv_heads, c.head_dim, 2);
  if (dtype == NVFP4_DTYPE_BF16)
    hipLaunchKernelGGL(k_kv_write<NVFP4_DTYPE_BF16>, g, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(k_kv_write<NVFP4_DTYPE_F32>, g, dim3(256), 0, st, p);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

struct KvRead {
  const uint8_t *codes[2], *scales[2];
  const float *S[2];
  void *y[2];
  const int64_t *slots;
  int64_t n, n_slots;
  int heads, head_dim, page_shift;
};

template <int DT>
__global__ void __launch_bounds__(256) k_kv_read(KvRead p) {
  const int kv = blockIdx.z, h = blockIdx.y;
  const int lanes = p.head_dim >> 3, rows = 256 / lanes;
  const int row = threadIdx.x / lanes, part = threadIdx.x - row * lanes;
  if (row >= rows) return;
  const float S = p.S[kv][h];
  const int64_t mask = ((int64_t)1 << p.page_shift) - 1;
  for (int64_t t = (int64_t)blockIdx.x * rows + row; t < p.n; t += (int64_t)gridDim.x * rows) {
    const int64_t slot = p.slots[t];
    float y[8] = {};
    if (slot >= 0 && slot < p.n_slots) {
      const int64_t at = ((((slot >> p.page_shift) * p.heads + h) << p.page_shift) + (slot & mask));
      const unsigned c = reinterpret_cast<const unsigned *>(p.codes[kv])[at * lanes + part];
      const float s = e4m3_value(given_byte(p.scales[kv][at * (lanes >> 1) + (part >> 1)]));
      float g[8];
      fp4_decode8(c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = g[i] * s * S;  // g s is exact
    }
    const int64_t e = (t * p.heads + h) * p.head_dim + part * 8;
    if (DT == NVFP4_DTYPE_BF16) {
      uint4 w;
      w.x = bf16x2_bits(y[0], y[1]), w.y = bf16x2_bits(y[2], y[3]);
      w.z = bf16x2_bits(y[4], y[5]), w.w = bf16x2_bits(y[6], y[7]);
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y[kv]) + e) = w;
    } else {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.y[kv]) + e);
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
}

int launch_kv_read(const nvfp4_kv_cache &c, const int64_t *slots, int64_t n, void *k, void *v,
                   int out_dtype, hipStream_t st) {
  KvRead p;
  int z = 0;
  if (k) p.codes[z] = c.k_codes, p.scales[z] = c.k_scales, p.S[z] = c.S_k, p.y[z++] = k;
  if (v) p.codes[z] = c.v_codes, p.scales[z] = c.v_scales, p.S[z] = c.S_v, p.y[z++] = v;
  if (z == 0) return NVFP4_OK;
  p.slots = slots, p.n = n, p.n_slots = c.pages * c.page_size;
  p.heads = (int)c.kv_heads, p.head_dim = (int)c.head_dim, p.page_shift = page_shift_of(c);
  const dim3 g = row_grid(n, c.kv_heads, c.head_dim, z);
  if (out_dtype == NVFP4_DTYPE_BF16)
    hipLaunchKernelGGL(k_kv_read<NVFP4_DTYPE_BF16>, g, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(k_kv_read<NVFP4_DTYPE_F32>, g, dim3(256), 0, st, p);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
