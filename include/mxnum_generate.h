/*
 * mxnum_generate.h -- C ABI of libmxnum.so, second part: one generation step of a model whose weights and
 * key/value cache are held in NVFP4.  The conventions of mxnum.h hold for every entry point (device pointers,
 * caller-owned buffers, host-side checks, asynchronous launches on the caller's stream); index and FP32 arrays
 * must be 4-byte aligned.
 * The kernels of these calls are launched so that the device may set one up while the one before it in the stream still
 * runs; each waits for the earlier work before it touches memory, so the order of a stream holds as ever.
 *
 * Source: Miles page -- NVFP4 rollout engines; NVIDIA NeMo RL FP8 page, "FP8 KV cache" -- a key/value cache in
 * few bits, its scales calibrated ahead of the step (the pages give no layout: this one is the library's).
 *
 * The cache is uint8 [pages, kv_heads, page_size / 16, 18 * head_dim]: records of 16 tokens of one head, each
 *   K codes   16 rows of head_dim / 2 bytes (E2M1, the even element in the low nibble)
 *   K scales  16 rows of head_dim / 16 E4M3 bytes
 *   V codes   16 rows of head_dim / 2 bytes
 *   V scales  [head_dim / 16][16] E4M3 bytes, token i of the record at position i ^ ((i >> 1) & 1)
 * with value = val(code) * val(block scale) * S, S one FP32 per kv head for K (s_k) and one for V (s_v), given by the
 * caller.  page_size is a multiple of 16 (at most 2^20), kv_heads at most 65535, head_dim 64, 128 or 256, pages * page_size < 2^31.
 * Slot number of a cached token: page * page_size + its offset inside the page.
 */
#ifndef MXNUM_GENERATE_H
#define MXNUM_GENERATE_H

#include "mxnum.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page, page_size / 16 * kv_heads * 18 * head_dim (0 for sizes the cache does not take). */
int64_t mx_kv_page_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim);

/* Largest number of requests of a step. */
#define MX_KV_MAX_REQUESTS 4096

/* Page and slot maps of a step, from the requests' lengths (negative lengths count as zero).
 *   seq_lens, new_lens [requests]  tokens already cached, tokens to add in this step
 *   block_table [requests, table_width], rows table_stride apart: page of each page_size positions.  The columns
 *            from ceil(seq / page_size) to ceil((seq + new) / page_size) - 1 (below table_width) are written: the new
 *            pages, in request order, are popped from the free stack, -1 once it is empty.
 *   free_pages [free_capacity], *free_count  the stack (its top at *free_count - 1; clamped to the capacity)
 * Outputs:
 *   q_start [requests + 1]  exclusive sums of new_lens;  total_lens [requests] = seq + new
 *   slots, positions [max_tokens]  slot (or -1 where the token has no page) and position in its request of
 *            each new token, requests in order; -1 from the number of new tokens on
 *   *free_left  pages left on the stack;  *unplaced  new tokens without a slot (those beyond max_tokens too)
 * total_lens may be seq_lens and free_left may be free_count; the other arrays must not overlap.  The new tokens and
 * requests * table_width must stay below 2^31.  requests <= MX_KV_MAX_REQUESTS. */
mx_status mx_kv_slots(const int32_t* seq_lens, const int32_t* new_lens, int64_t requests, int64_t page_size,
                      int32_t* block_table, int64_t table_width, int64_t table_stride, const int32_t* free_pages,
                      int64_t free_capacity, const int32_t* free_count, int32_t* q_start, int32_t* total_lens,
                      int32_t* slots, int32_t* positions, int64_t max_tokens, int32_t* free_left, int32_t* unplaced,
                      cudaStream_t stream);

/* Quantize new keys and values into the cache.  Per 16-block, with S the head's second-level scale: block scale
 * and codes as in mx_nvfp4_quantize_per_token (bs = E4M3(amax_b / 6 / S), saturating: a block whose maximum
 * exceeds 2688 S is clipped).  A NaN makes its block NaN; an infinity saturates.
 *   k, v [T, kv_heads, head_dim] BF16, token and head strides in elements (multiples of 8; unit element stride)
 *   slots [T] distinct slot numbers; a token whose slot lies outside the cache (-1) is skipped. */
mx_status mx_nvfp4_kv_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                             int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots, int64_t T,
                             const float* s_k, const float* s_v, uint8_t* cache, int64_t pages, int64_t page_size,
                             int64_t kv_heads, int64_t head_dim, cudaStream_t stream);

/* Read cached tokens back: k, v = BF16 RNE of fp32(val(code) * val(block scale)) * S, for prompt passes that attend in BF16
 * to what later steps will read from the cache.  Arguments as in mx_nvfp4_kv_append; slots need not be distinct, and
 * a slot outside the cache gives zeros. */
mx_status mx_nvfp4_kv_gather(const uint8_t* cache, int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim,
                             const int32_t* slots, int64_t T, const float* s_k, const float* s_v, void* k,
                             int64_t k_token_stride, int64_t k_head_stride, void* v, int64_t v_token_stride,
                             int64_t v_head_stride, cudaStream_t stream);

/* Attention of a step's new tokens over the cache, which holds them already:
 *   out[t, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q[t, h] . k_j),  lse[t, h] = log sum_j p_j
 * over the positions j of the token's request with max(0, pos - window + 1) <= j <= pos (window = 0: all from 0), where
 * pos = seq_len - n + i for token i of the request's n.  q head h reads kv head h / (heads / kv_heads).  A token
 * with nothing to attend to gives zeros and lse = -inf.  Positions whose page number lies outside the cache are
 * skipped.
 *   q [T, heads, head_dim] BF16 and out alike, with token and head strides in elements (multiples of 8)
 *   q_start [requests + 1]  first token of each request (nondecreasing, at most T; rows of out and lse that belong to
 *            no request are not written)
 *   seq_lens [requests]  cached tokens, the new ones included
 *   max_q  rows of a request: at least the largest n (of a request with more the first max_q are written, the others left as
 *            they are).  The work of all requests is laid out for it, so the largest n itself is fastest.
 *   block_table [requests, table_width] as written by mx_kv_slots;  s_k, s_v [kv_heads]
 *   lse [T, heads] FP32 or NULL
 *   workspace: mx_kv_attention_workspace_bytes(head_dim) bytes, 16-byte aligned, need not be cleared.
 * Scores, softmax statistics and sums are FP32; the probabilities enter the second product as FP16.  A NaN among the keys
 * makes the rows that attend to it NaN, one among the values their 16 dimensions of that block; a masked one reaches
 * nothing.  The result does not depend on what runs beside it: the split of the work, which the order of the sums follows, goes by
 * the lengths, the table's width, max_q and the number of SMs.  A table no wider than the step's longest context is fastest for
 * short ones: one request of 777 tokens takes 6.8 us under its own and 8.5 under one of 131072 positions. */
size_t mx_kv_attention_workspace_bytes(int64_t head_dim);
mx_status mx_nvfp4_kv_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t T, int64_t heads,
                                const int32_t* q_start, const int32_t* seq_lens, int64_t requests, int64_t max_q,
                                const int32_t* block_table, int64_t table_width, int64_t table_stride,
                                const uint8_t* cache, int64_t pages, int64_t page_size, int64_t kv_heads,
                                int64_t head_dim, const float* s_k, const float* s_v, float scale, int64_t window,
                                void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Products of a few tokens with NVFP4 weights (the linear layers of a step), sixteen tokens a pass over the weights; beyond
 * 32 tokens mx_gemm_bf16_dq_nvfp4 is quicker for wide N (12288 x 4096: 41 to 44 us at any M up to 64, here 11 at 5 tokens, 35 at 32,
 * 70 at 64), if weights rounded to BF16 will do:
 *   y[m, n] = s2[n or 0] * sum_k x[m, k] * val(q[n, k]) * val(bs[n, k / 16])
 *   x [M, ldx] BF16;  q [N, K/2] E2M1 codes, s mx_scale_bytes(N, K, 16) E4M3 scales in the GEMM layout, s2 one FP32
 *   (MX_SCOPE_TENSOR) or N (MX_SCOPE_ROW): a weight as the row-wise NVFP4 quantizers write it
 *   y [M, ldy] BF16 (y_fp32 = 0) or FP32 (y_fp32 = 1)
 * The weights enter the products exactly, sums are FP32.  Requires M <= MX_MATVEC_MAX_TOKENS, K % 16 == 0, ldx % 8 == 0;
 * x, q, s, y 16-byte aligned; any N. */
#define MX_MATVEC_MAX_TOKENS 64
mx_status mx_nvfp4_matvec(const void* x, int64_t ldx, const uint8_t* q, const uint8_t* s, const float* s2,
                          mx_scope s2_scope, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int y_fp32,
                          cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXNUM_GENERATE_H */
