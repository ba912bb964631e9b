// Internal launchers of the rotation (not exported). Arguments are validated by the entry points in
// nvfp4_rotary_api.hip before any of these run.
#pragma once

#include "../../include/nvfp4_kv.h"
#include "../../include/nvfp4_rotary.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

// Rows of a strided [tokens][heads][..] tensor.
struct RowSpan {
  const void *x;
  int64_t ts, hs;
};

// positions by pair: what a kernel needs of nvfp4_rotary
struct Turn {
  const double *inv_freq;
  const int32_t *axis;
  const int64_t *positions;
  int64_t stride;
  double factor;
  int pairs, axes;
};

int launch_rotate(const Turn &turn, bool adjacent, bool transpose, const RowSpan &x,
                  const RowSpan &out, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                  hipStream_t st);
int launch_kv_append(const nvfp4_kv_cache &c, const Turn &turn, bool adjacent, const RowSpan &q,
                     const RowSpan &q_out, const RowSpan &k, const RowSpan &v, int dtype,
                     int64_t tokens, int64_t heads, const int64_t *slots, hipStream_t st);

}  // namespace nvfp4
