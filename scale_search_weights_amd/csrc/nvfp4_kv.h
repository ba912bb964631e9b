// Internal launchers of the key/value cache (not exported). Arguments are validated by the
// entry points in nvfp4_kv_api.hip before any of these run.
#pragma once

#include "../../include/nvfp4_kv.h"
#include "nvfp4_internal.h"
#include "nvfp4_kv_plan.h"

namespace nvfp4 {

int launch_kv_write(const nvfp4_kv_cache &c, const void *k, const void *v, int dtype,
                    int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                    const int64_t *slots, hipStream_t st);
int launch_kv_read(const nvfp4_kv_cache &c, const int64_t *slots, int64_t n, void *k, void *v,
                   int out_dtype, hipStream_t st);

int launch_kv_attention(const KvAttention &a, hipStream_t st);
int launch_kv_window_attention(const KvAttention &a, int64_t window, int64_t sinks, hipStream_t st);

// NVFP4_DEBUG_CHECKS: scan a strided [tokens][heads][head_dim] tensor for NaN and infinities.
void debug_check_finite_rows(const void *x, int dtype, int64_t tokens, int64_t heads,
                             int64_t head_dim, int64_t token_stride, int64_t head_stride,
                             hipStream_t st);

}  // namespace nvfp4
