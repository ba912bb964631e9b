/*
 * libnvfp4, key/value cache — the keys and values of an attention layer held in NVFP4, and
 * the attention that reads them, on AMD Instinct MI355X (gfx950).
 *
 * A cached vector (one token, one key/value head) is a row of head_dim values in the format
 * of nvfp4.h: E2M1 codes, one E4M3 scale for every 16 values, and one fp32 tensor scale for
 * each head, S_k[h] for keys and S_v[h] for values. A cached value stands for G * s * S (G the
 * code's grid value, s its block's scale). The cache is paged:
 *   k_codes, v_codes    [pages][kv_heads][page_size][head_dim / 2]   uint8, 16-byte aligned
 *   k_scales, v_scales  [pages][kv_heads][page_size][head_dim / 16]  uint8, 16-byte aligned
 *   S_k, S_v            [kv_heads]                                   fp32
 * A slot is page * page_size + offset. Which pages belong to which sequence is the caller's
 * (a block table); cache memory need not be initialised: bytes of tokens beyond a sequence's
 * length never reach a result, whatever they hold. Scale bytes are read as E4M3 magnitudes
 * with 0x7F coded as zero, as everywhere in the library. A cache without pages may leave the codes
 * and block scales NULL; S_k and S_v are needed by every call that has something to do, except that
 * write has nothing to do then, and append only queries to turn.
 *
 * Conventions (pointers, streams, status codes, rounding) are those of nvfp4.h, except that
 * k, v and q may be strided: the last dimension is contiguous, the strides of the token and the
 * head dimension are given in elements, and every row (one token, one head) starts at a
 * multiple of 16 bytes. page_size is a power of two from 16 to 32768; head_dim is a multiple
 * of 16, up to 1024 for write and read and up to 256 for attention.
 */
#ifndef NVFP4_KV_H
#define NVFP4_KV_H

#include "nvfp4.h"
#include "nvfp4_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache of one layer: device pointers and sizes as above. The library reads the struct
 * during the call and keeps nothing of it. */
typedef struct nvfp4_kv_cache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float *S_k, *S_v;
  int64_t pages, page_size, kv_heads, head_dim;
} nvfp4_kv_cache;

/*
 * Quantise new keys and values as they are written: for every token t with
 * 0 <= slots[t] < pages * page_size, k[t][h] and v[t][h] go to slot slots[t] of head h, with
 * max-scaling block bytes and exact nearest-even decisions (the results of nvfp4_quantize at
 * S_k[h], S_v[h]). Tokens with any other slot (padding) are skipped. Two tokens of one call
 * must not share a slot. k, v: [tokens][kv_heads][head_dim] of `dtype`, strided; slots:
 * [tokens] int64.
 */
NVFP4_API int nvfp4_kv_write(const nvfp4_kv_cache *cache, const void *k, const void *v, int dtype,
                             int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                             void *stream);

/*
 * Append: nvfp4_kv_write with the rotation of nvfp4_rotate on the way. For every token t with
 * 0 <= slots[t] < pages * page_size, k[t][h] turned by the token's positions and v[t][h] as it is go
 * to slot slots[t] of head h; a turned key is quantised from its fp32 value, without a rounding to
 * bf16 in between. Tokens with any other slot are skipped. Two tokens of one call must not share a
 * slot. q_out[t][j] = q[t][j] turned, for every token, skipped ones too: q, q_out
 * [tokens][heads][head_dim] of `dtype`, strided; q_out may be q itself, with the same strides, and
 * must not overlap anything else that the call reads. heads 0 for none (q, q_out may then be NULL).
 * k, v: [tokens][kv_heads][head_dim] of `dtype`, strided; slots: [tokens] int64; positions as in
 * nvfp4_rotate. The rotation's pairs are a multiple of 8. All of it in one launch.
 */
NVFP4_API int nvfp4_kv_append(const nvfp4_kv_cache *cache, const nvfp4_rotary *rotary,
                              const int64_t *positions, int64_t position_stride, const void *q,
                              const void *k, const void *v, int dtype, int64_t tokens,
                              int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                              int64_t k_token_stride, int64_t k_head_stride,
                              int64_t v_token_stride, int64_t v_head_stride, void *q_out,
                              int64_t q_out_token_stride, int64_t q_out_head_stride,
                              const int64_t *slots, void *stream);

/*
 * Read cached keys and values back: k[n][h], v[n][h] = the values of slot slots[n], dequantised
 * as nvfp4_dequantize does (fp32(G s S), one rounding; bf16 from that). A slot outside the
 * cache gives zeros. k, v: [n][kv_heads][head_dim] contiguous, of out_dtype; either may be
 * NULL, and is then not read.
 */
NVFP4_API int nvfp4_kv_read(const nvfp4_kv_cache *cache, const int64_t *slots, int64_t n, void *k,
                            void *v, int out_dtype, void *stream);

/*
 * Softmax attention of new queries over cached tokens. q: [tokens][heads][head_dim], strided;
 * query head j reads key/value head j / (heads / kv_heads). The batch's tokens are packed:
 * sequence b owns rows q_offsets[b] .. q_offsets[b+1] (device int32 [batch + 1],
 * non-decreasing, at most max_q each); q_offsets == NULL means max_q rows each, and then
 * tokens == batch * max_q.
 *
 * A query of sequence b sees
 *  - every token of the shared prefix: prefix_len tokens in the pages prefix_pages
 *    [ceil(prefix_len / page_size)] (device int32; prefix_len 0 for none), read once for the
 *    whole batch, and
 *  - tokens of its own: kv_lens[b] (device int32, at most max_kv) in the pages
 *    block_table[b][0..] (device int32 [batch][table_width]). With n query rows, row i
 *    sees own tokens j <= kv_lens[b] - n + i if `causal` is non-zero (the new tokens are the
 *    last n of the sequence) and all of them if it is zero (an encoder's states).
 * max_kv is at most table_width * page_size; max_kv 0 means no sequence has tokens of its own
 * (block_table and kv_lens are then not read and may be NULL).
 *   out[i][j] = sum_t p_t v_t,  p = softmax over the seen tokens of scale * (q[i][j] . k_t);
 *   lse[i][j] (nullable, fp32) = ln sum_t exp(scale * (q[i][j] . k_t)).
 * A row that sees nothing gets out = 0 and lse = -inf; any other row whose query is not finite gets
 * NaN in both, and other rows stay right. Rows of out and lse that belong to no
 * sequence hold unspecified values. Page ids outside [0, pages) hide the page's tokens; kv_lens
 * is cut to [0, max_kv].
 *
 * Products take fp16 operands (cached values without S are exact in fp16; bf16 queries are
 * scaled by a power of two per row, probabilities are rounded to 11 bits, and to multiples of
 * 2^-31 of the row's largest) with fp32 sums; for fp32 q, queries and probabilities are split
 * in two fp16 halves (22 bits, multiples of 2^-37). Softmax statistics are fp32.
 * out: [tokens][heads][head_dim] contiguous, of `dtype`. Partial sums are joined in a fixed
 * order: results are bitwise reproducible for the same arguments and device.
 *
 * tokens * heads is at most 2^31 - 1025. max_q may be loose, but the call then launches a workgroup
 * for every 16 to 256 rows that it allows each sequence and key/value head, with rows or without;
 * more than 2^31 - 1 of them are refused (NVFP4_ERR_SHAPE).
 *
 * workspace: 16-byte aligned, at least nvfp4_kv_attention_workspace_size() bytes (may be 0),
 * no initialisation needed; calls that share it must not overlap.
 */
NVFP4_API size_t nvfp4_kv_attention_workspace_size(const nvfp4_kv_cache *cache, int dtype,
                                                   int64_t tokens, int64_t heads, int64_t batch,
                                                   int64_t max_q, int64_t max_kv,
                                                   int64_t prefix_len);
NVFP4_API int nvfp4_kv_attention(const nvfp4_kv_cache *cache, const void *q, int dtype,
                                 int64_t tokens, int64_t heads, int64_t q_token_stride,
                                 int64_t q_head_stride, int64_t batch, const int32_t *q_offsets,
                                 int64_t max_q, const int32_t *block_table, int64_t table_width,
                                 const int32_t *kv_lens, int64_t max_kv,
                                 const int32_t *prefix_pages, int64_t prefix_len, float scale,
                                 int causal, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * Attention over a sliding window and the first tokens, which stay visible (sinks): as
 * nvfp4_kv_attention without a prefix, except that row i of a sequence's n, at position P = kv_lens[b] -
 * n + i, sees the tokens t <= P with t > P - window or t < sinks. window is 1 to 2^30, sinks 0 to 2^30.
 * Only tokens that some row of a tile of at most 256 rows sees are read (in groups of 16): the work and
 * the workspace do not grow with the context, and the pages of tokens between the sinks' and the
 * windows' groups may be gone from the block table (any ids there). Results are reproducible as
 * there; a window that covers the context sees what nvfp4_kv_attention sees.
 */
NVFP4_API size_t nvfp4_kv_window_attention_workspace_size(const nvfp4_kv_cache *cache, int dtype,
                                                          int64_t tokens, int64_t heads,
                                                          int64_t batch, int64_t max_q,
                                                          int64_t max_kv, int64_t window,
                                                          int64_t sinks);
NVFP4_API int nvfp4_kv_window_attention(const nvfp4_kv_cache *cache, const void *q, int dtype,
                                        int64_t tokens, int64_t heads, int64_t q_token_stride,
                                        int64_t q_head_stride, int64_t batch,
                                        const int32_t *q_offsets, int64_t max_q,
                                        const int32_t *block_table, int64_t table_width,
                                        const int32_t *kv_lens, int64_t max_kv, int64_t window,
                                        int64_t sinks, float scale, void *out, float *lse,
                                        void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_H */
