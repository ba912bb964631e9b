// Key/value cache in NVFP4: quantise rows into cache slots, and read slots back.
//
// Both kernels take (token, head) rows of head_dim values, one head to a workgroup: its tensor
// scale is uniform, and consecutive tokens of a page are contiguous in the cache, so a
// workgroup's stores join into whole lines. A lane of write takes a block of 16: its maximum
// needs no exchange, and the fp64 work on its scale, which costs as much as its values, is done
// once (with half a block a lane 16384 tokens of 8 heads of 128 took 4 us more). A lane of read
// takes the values of 16 bytes of output, so the lanes of a store are contiguous.
//
// They are bound by memory: write moves 2 or 4 bytes in and 9/16 out per value, read the reverse.
// 131072 tokens of 8 heads of 128 are read in 134 us, 5.1 TB/s, what a 1 GiB copy reaches; 16384
// tokens are written and read in 35 us, 5.0 TB/s; 30000 in fp32 in 100 us, 5.6 TB/s (eight
// values a lane of read, two strided stores, cost 74 us more). Values that are read back are stored
// non-temporally (134 us, 141 with ordinary stores), except in rows of no whole 64 bytes (19103
// tokens of 11 heads of 112: 21 us, 29 non-temporally; 101071 of 12 heads of 80: 130 and 158); codes
// are not, the attention that follows finds them in the caches.
#include "nvfp4_device.h"
#include "nvfp4_kv.h"
#include "nvfp4_rows.h"

namespace nvfp4 {

// Rows a lane takes at once, their loads issued together: without it a wave waits for one row's
// slot and then its codes, and read runs at 3.5 TB/s (131072 tokens, 8 heads of 128: 198 us;
// with 4 rows 134 us, 2 or 8 rows 3 to 8% slower). Write: 16384 tokens written and read 35.4 us
// with 1 row, 34.2 with 2, 35.6 with 4. Calls of fewer rows times lanes than these fill the chip
// with one row a lane only (48 tokens written and read: 5.5 us, 6.5 us with several; 4000 tokens of
// 5 heads of 64 read in fp32, 640 Ki: 5.4 us with 1, 5.3 with 4; 3000, 480 Ki: 4.7 and 4.5).
constexpr int kReadRows = 4, kWriteRows = 2;
constexpr int64_t kReadFew = 512 << 10, kWriteFew = 256 << 10;

// Slots of this lane's U rows: a workgroup takes U x 256 / lanes; -1 past the end
// and for tokens without a slot in the cache.
template <int U>
__device__ __forceinline__ void load_slots(const int64_t *slots, int64_t n, int64_t n_slots,
                                           int64_t t0, int rows, int64_t *slot) {
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = t0 + u * rows < n ? slots[t0 + u * rows] : -1;
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = slot[u] < n_slots ? slot[u] : -1;
}

// The (head, first token, token step) of a workgroup. Large calls (DIES): workgroups go to the 8
// dies in turn, and those of one chunk of tokens follow each other on one die, so that lines shared
// by neighbouring heads meet in its L2. (With heads far apart in the grid: rows of 160 bytes, 101071
// tokens of 12 heads, 213 us read, 130 so; rows of 512, 30000 tokens written and read, 116 and 100.
// In small calls that order costs 0.3 to 1 us.)
struct Place {
  int h;
  int64_t t, step;
};
template <bool DIES>
__device__ __forceinline__ Place place_of(int heads, int per) {
  if (!DIES) return {(int)blockIdx.z, (int64_t)blockIdx.x * per, (int64_t)gridDim.x * per};
  const int die = blockIdx.x & 7, j = blockIdx.x >> 3, chunk = j / heads;
  return {j - chunk * heads, (int64_t)(chunk * 8 + die) * per, (int64_t)(gridDim.x / heads) * per};
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

template <int DT, int U>
__global__ void __launch_bounds__(256) k_kv_write(KvWrite p) {
  const int lanes = p.head_dim >> 4, rows = 256 / lanes;
  const Place at0 = place_of<(U > 1)>(p.heads, U * rows);
  const int kv = blockIdx.y, h = at0.h;
  const int row = threadIdx.x / lanes, part = threadIdx.x - row * lanes;
  if (row >= rows) return;
  const float S = p.S[kv][h];
  float lo6, hi6;
  recip_bracket(6.0 * (double)S, lo6, hi6);
  const int64_t mask = ((int64_t)1 << p.page_shift) - 1;
  for (int64_t t = at0.t + row; t < p.tokens; t += at0.step) {
    int64_t slot[U];
    float v[U][16];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // loads of all rows first, also of tokens that are skipped
      const int64_t e = min(t + u * rows, p.tokens - 1) * p.ts[kv] + h * p.hs[kv] + part * 16;
      load8<DT>(p.x[kv], e, v[u]);
      load8<DT>(p.x[kv], e + 8, v[u] + 8);
    }
    load_slots<U>(p.slots, p.tokens, p.n_slots, t, rows, slot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (slot[u] < 0) continue;
      uint2 c;
      const int b = quantise16(v[u], lo6, hi6, S, c);
      const int64_t at = (((slot[u] >> p.page_shift) * p.heads + h) << p.page_shift) + (slot[u] & mask);
      reinterpret_cast<uint2 *>(p.codes[kv])[at * lanes + part] = c;
      p.scales[kv][at * lanes + part] = (uint8_t)b;
    }
  }
}

static int page_shift_of(const nvfp4_kv_cache &c) { return __builtin_ctzll((unsigned long long)c.page_size); }

// Grid for `tokens` rows of `lanes` lanes, u rows a lane, as place_of reads it.
static dim3 row_grid(int64_t tokens, int64_t heads, int64_t lanes, int z, int u) {
  const int64_t rows = 256 / lanes * u;
  int64_t g = (tokens + rows - 1) / rows, cap = 65536 / (heads * z);  // the rest in a loop
  if (cap < 64) cap = 64;
  if (g > cap) g = cap;
  if (u == 1) return dim3((unsigned)g, (unsigned)z, (unsigned)heads);
  return dim3((unsigned)((g + 7) / 8 * 8 * heads), (unsigned)z);
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
  const int64_t lanes = c.head_dim / 16;
  const int u = tokens * c.kv_heads * lanes * 2 < kWriteFew ? 1 : kWriteRows;
  const dim3 g = row_grid(tokens, c.kv_heads, lanes, 2, u), b(256);
  if (dtype == NVFP4_DTYPE_BF16) {
    if (u == 1) hipLaunchKernelGGL((k_kv_write<NVFP4_DTYPE_BF16, 1>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_kv_write<NVFP4_DTYPE_BF16, kWriteRows>), g, b, 0, st, p);
  } else {
    if (u == 1) hipLaunchKernelGGL((k_kv_write<NVFP4_DTYPE_F32, 1>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_kv_write<NVFP4_DTYPE_F32, kWriteRows>), g, b, 0, st, p);
  }
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

typedef unsigned kv_u4 __attribute__((ext_vector_type(4)));
typedef float kv_f4 __attribute__((ext_vector_type(4)));

// Values a lane of read takes: 16 bytes of output, so that the lanes of a store are contiguous.
constexpr int read_values(int dt) { return dt == NVFP4_DTYPE_BF16 ? 8 : 4; }

template <int DT, int U, bool STREAM>  // STREAM: rows are whole pieces of 64 bytes
__global__ void __launch_bounds__(256) k_kv_read(KvRead p) {
  constexpr int V = read_values(DT);
  const int lanes = p.head_dim / V, rows = 256 / lanes;
  const Place at0 = place_of<(U > 1)>(p.heads, U * rows);
  const int kv = blockIdx.y, h = at0.h;
  const int row = threadIdx.x / lanes, part = threadIdx.x - row * lanes;
  if (row >= rows) return;
  const float S = p.S[kv][h];
  const int64_t mask = ((int64_t)1 << p.page_shift) - 1;
  for (int64_t t = at0.t + row; t < p.n; t += at0.step) {
    int64_t slot[U];
    unsigned c[U], b[U];
    load_slots<U>(p.slots, p.n, p.n_slots, t, rows, slot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c[u] = b[u] = 0u;  // no slot: zeros
      if (slot[u] >= 0) {
        const int64_t at = (((slot[u] >> p.page_shift) * p.heads + h) << p.page_shift) + (slot[u] & mask);
        if (V == 8) c[u] = reinterpret_cast<const unsigned *>(p.codes[kv])[at * lanes + part];
        else c[u] = reinterpret_cast<const uint16_t *>(p.codes[kv])[at * lanes + part];
        b[u] = p.scales[kv][at * (lanes * V / 16) + part * V / 16];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * rows >= p.n) continue;
      const float s = e4m3_value(given_byte(b[u]));
      float y[8];
      fp4_decode8(c[u], y);
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = y[i] * s * S;  // g s is exact
      const int64_t e = ((t + u * rows) * p.heads + h) * p.head_dim + part * V;
      if (DT == NVFP4_DTYPE_BF16) {
        const kv_u4 w = {bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]), bf16x2_bits(y[4], y[5]),
                         bf16x2_bits(y[6], y[7])};
        kv_u4 *o = reinterpret_cast<kv_u4 *>(static_cast<uint16_t *>(p.y[kv]) + e);
        if (STREAM) __builtin_nontemporal_store(w, o);
        else *o = w;  // the caches join the pieces
      } else {
        const kv_f4 w = {y[0], y[1], y[2], y[3]};
        __builtin_nontemporal_store(w, reinterpret_cast<kv_f4 *>(static_cast<float *>(p.y[kv]) + e));
      }
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
  const int64_t lanes = c.head_dim / read_values(out_dtype);
  const int u = n * c.kv_heads * lanes * z < kReadFew ? 1 : kReadRows;
  const dim3 g = row_grid(n, c.kv_heads, lanes, z, u), b(256);
  if (out_dtype == NVFP4_DTYPE_F32) {
    if (u == 1) hipLaunchKernelGGL((k_kv_read<NVFP4_DTYPE_F32, 1, true>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_kv_read<NVFP4_DTYPE_F32, kReadRows, true>), g, b, 0, st, p);
  } else if (u == 1) {  // small: what is stored stays in the caches either way
    hipLaunchKernelGGL((k_kv_read<NVFP4_DTYPE_BF16, 1, false>), g, b, 0, st, p);
  } else if (c.head_dim % 32) {
    hipLaunchKernelGGL((k_kv_read<NVFP4_DTYPE_BF16, kReadRows, false>), g, b, 0, st, p);
  } else {
    hipLaunchKernelGGL((k_kv_read<NVFP4_DTYPE_BF16, kReadRows, true>), g, b, 0, st, p);
  }
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
