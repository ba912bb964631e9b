// Rows of bf16 or fp32 values in registers, and the quantiser of a block of 16 held by one lane.
#pragma once

#include "../../include/nvfp4.h"
#include "nvfp4_device.h"

namespace nvfp4 {

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

// A block of 16 values at tensor scale S: returns the max-scaling byte b, c the packed codes
// (nvfp4_quantize's); lo6 < 1 / (6 S) < hi6.
__device__ __forceinline__ int quantise16(const float *v, float lo6, float hi6, float S, uint2 &c) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
  const int b = max_scale_byte_fast(amax, lo6, hi6, S);
  c = make_uint2(0u, 0u);
  if (b) {
    const double sS = e4m3_value_d(b) * (double)S;
    float lo, hi;
    recip_bracket(sS, lo, hi);
    c.x = fp4_clear_neg_zero(fp4_exact_codes8(v, lo, hi, sS));
    c.y = fp4_clear_neg_zero(fp4_exact_codes8(v + 8, lo, hi, sS));
  }
  return b;
}

}  // namespace nvfp4
