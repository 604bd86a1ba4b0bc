/*
 * mxnum_layer.h -- C ABI of libmxnum.so, third part: what lies between the products of a layer with routed experts.  The
 * norm before a product with the residual's addition and its output in MXFP8, the router's choice of experts, the tokens
 * sorted by expert for the grouped products and back, and the gradients.  The conventions of mxnum.h hold for every entry
 * point (device pointers, caller-owned buffers, host-side checks, asynchronous launches on the caller's stream).  BF16
 * tensors, codes, scales, group offsets and workspaces must be 16-byte aligned, 32-bit arrays 4-byte aligned.
 * Calls that may overlap on the GPU (other streams, other captured graphs) need workspaces of their own.
 * The kernels of these calls may be set up while the one before in the stream still runs; each waits for the earlier work
 * before it touches memory, so the order of a stream holds as ever.
 *
 * Source: Miles page -- the quantizer fused with what produces its input, NVFP4 on the routed experts only; E2E page Table 2
 * (128 experts, top-8) and Table 6 (the time of separate quantize and rearrange passes).  The pages give no formulas for
 * norm, routing or sorting: these are the usual ones, written out below.
 */
#ifndef MXNUM_LAYER_H
#define MXNUM_LAYER_H

#include "mxnum.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of a tensor that may be BF16 or FP32. */
typedef enum { MX_DTYPE_BF16 = 0, MX_DTYPE_FP32 = 1 } mx_dtype;

/* Widest row of the norm, and most experts of a token. */
#define MX_RMSNORM_MAX_COLS 16384
#define MX_MOE_MAX_TOP_K 32

/* Root-mean-square norm with the residual's addition, and its output in MXFP8.  Per row:
 *   h = BF16(x + residual)                            (h = x without a residual)
 *   y = BF16(h * weight / sqrt(mean(h^2) + eps))      (FP32: the product with weight, exact where that is BF16 and
 *                                                      the product a normal number, times 1 / sqrt)
 *   codes and scales: those of mx_quantize_mxfp8(y), byte for byte, in either orientation
 *   x, residual [rows, cols] BF16, rows ldx and ldr elements apart;  residual NULL: none
 *   weight   [cols], BF16 or FP32 by weight_type
 *   sum      [rows, lds] BF16: h (NULL: not written; without a residual it must be NULL).  It may be x or residual itself.
 *   y        [rows, ldy] BF16 (NULL: not written)
 *   q_row, s_row, q_col, s_col as in mx_quantize_mxfp8 (NULL: skip)
 * At least one of y, q_row and q_col.  No other two buffers may overlap.  Requires cols % 8 == 0, for row-wise codes cols % 32
 * == 0, for column-wise ones rows % 32 == 0; cols <= MX_RMSNORM_MAX_COLS; eps >= 0 and finite; weights below 2^60.  A row's values do not
 * depend on the other rows, their number or which outputs are asked for.  Rows whose squares leave FP32's range are summed in
 * FP64.  A NaN makes its row NaN; an infinity too where it stands, and zeros elsewhere. */
mx_status mx_rmsnorm_mxfp8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                           mx_dtype weight_type, float eps, int64_t rows, int64_t cols, void* sum, int64_t lds, void* y,
                           int64_t ldy, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                           cudaStream_t stream);

/* Its gradient.  With h the norm's input (the sum where there was a residual), r = 1 / sqrt(mean(h^2) + eps), n = h r and
 * dn = dy * weight:
 *   dx = BF16(r (dn - n mean(dn n)) + dsum),   dweight = sum over rows of dy * n
 *   dy, h, dsum, dx [rows, cols] BF16 with their row strides; dsum: what reaches h by the residual path (NULL: nothing).  dx is
 *            the gradient of x and of the residual alike, and may be dsum or dy itself.
 *   dweight  [cols] FP32 (written), the sums in FP32 in an order that depends on the sizes and the GPU only
 *   workspace: mx_rmsnorm_workspace_bytes(rows, cols) bytes, need not be cleared
 * The rounding of the output to MXFP8 counts as the identity.  Sizes as above. */
size_t mx_rmsnorm_workspace_bytes(int64_t rows, int64_t cols);
mx_status mx_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                              mx_dtype weight_type, float eps, int64_t rows, int64_t cols, const void* dsum, int64_t ldds,
                              void* dx, int64_t lddx, float* dweight, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream);

/* The experts of each token: the top_k largest logits, largest first, of equal ones the lowest index first.
 *   weights = softmax over the chosen logits (normalize = 1) or the chosen entries of the softmax over all (0)
 *   logits [tokens, ldl], BF16 or FP32 by logits_type, 4-byte aligned;  ids [tokens, top_k] int32, weights [tokens, top_k] FP32
 * A logit of -inf is never chosen: where fewer than top_k are left the others' ids are -1 and their weights zero.  A NaN counts
 * as the largest and makes the row's weights NaN, as +inf does.  experts <= MX_MAX_GROUPS, top_k <= experts and
 * <= MX_MOE_MAX_TOP_K. */
mx_status mx_moe_route(const void* logits, mx_dtype logits_type, int64_t ldl, int64_t tokens, int64_t experts, int64_t top_k,
                       int normalize, int32_t* ids, float* weights, cudaStream_t stream);

/* Gradient of the logits from that of the weights, with w recomputed from logits and ids (ids outside [0, experts) are skipped):
 *   normalize = 1: dlogits[id_j] = w_j (dw_j - sum_i w_i dw_i), zero elsewhere
 *   normalize = 0: dlogits[e] = p_e (dw_j where e = id_j - sum_i w_i dw_i), p the softmax over all
 * dlogits [tokens, ldd] of the logits' type.  Where w or p is NaN (a NaN or +inf among the logits that it is made of) these are NaN:
 * the chosen ones' (1) or the whole row (0). */
mx_status mx_moe_route_backward(const void* logits, mx_dtype logits_type, int64_t ldl, int64_t tokens, int64_t experts,
                                int64_t top_k, int normalize, const int32_t* ids, const float* dweights, void* dlogits,
                                int64_t ldd, cudaStream_t stream);

/* Tokens sorted by expert.  ids [tokens, top_k]; choice number t * top_k + j; choices of one expert keep their order.
 *   group_offsets [experts + 1] int64: first row of each expert, as the grouped calls take it
 *   rows   [tokens, top_k]: row of each choice; -1 where its id lies outside [0, experts), which leaves it out
 *   source [tokens * top_k]: choice of each row, -1 from row group_offsets[experts] on (NULL: not written)
 *   workspace: mx_moe_sort_workspace_bytes(tokens * top_k, experts) bytes, need not be cleared
 * tokens * top_k < 2^31, experts <= MX_MAX_GROUPS; ids must not overlap the outputs. */
size_t mx_moe_sort_workspace_bytes(int64_t choices, int64_t experts);
mx_status mx_moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int64_t* group_offsets,
                      int32_t* rows, int32_t* source, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Rows to their experts: y[rows[t, j]] = x[t].  x [tokens, ldx], y [total_rows, ldy] BF16, hidden % 8 == 0.  rows [tokens,
 * top_k] distinct row numbers; those outside [0, total_rows) are skipped, rows of y that none names are left as they were. */
mx_status mx_moe_dispatch(const void* x, int64_t ldx, int64_t tokens, int64_t hidden, const int32_t* rows, int64_t top_k,
                          void* y, int64_t ldy, int64_t total_rows, cudaStream_t stream);

/* The same for rows that are quantized already, each token once: the codes and scales that the grouped quantizer would
 * write for the dispatched BF16 rows.
 *   q [tokens, hidden (/2 for NVFP4)], s mx_scale_bytes(tokens, hidden, 32 or 16) as the row-wise quantizers write them
 *   s2, s2_out [tokens], [total_rows] FP32 second-level scales (NVFP4; both NULL for MXFP8)
 *   rows [tokens, top_k], group_offsets [G + 1] as written by mx_moe_sort
 *   q_out [total_rows, hidden (/2)], s_out mx_grouped_scale_bytes(total_rows, G, hidden, 32 or 16), its padding zeroed
 * hidden % 32 == 0, G <= MX_MAX_GROUPS. */
mx_status mx_moe_dispatch_quantized(mx_format fmt, const uint8_t* q, const uint8_t* s, const float* s2, int64_t tokens,
                                    int64_t hidden, const int32_t* rows, int64_t top_k, int64_t G,
                                    const int64_t* group_offsets, uint8_t* q_out, uint8_t* s_out, float* s2_out,
                                    int64_t total_rows, cudaStream_t stream);

/* The experts' rows back to their tokens: y[t] = BF16(sum_j weights[t, j] z[rows[t, j]] + residual[t]), in FP32, j ascending.
 *   z [total_rows, ldz], y [tokens, ldy], residual [tokens, ldr] BF16 (residual NULL: none; y may be residual itself)
 *   weights [tokens, top_k] FP32 (NULL: all 1; the call is then the gradient of mx_moe_dispatch)
 * Rows outside [0, total_rows) are skipped, so a token without any gives its residual or zeros.  hidden % 8 == 0. */
mx_status mx_moe_combine(const void* z, int64_t ldz, int64_t total_rows, int64_t hidden, const int32_t* rows,
                         const float* weights, int64_t tokens, int64_t top_k, const void* residual, int64_t ldr, void* y,
                         int64_t ldy, cudaStream_t stream);

/* Its gradients: dz[rows[t, j]] = BF16(weights[t, j] dy[t]), dweights[t, j] = dy[t] . z[rows[t, j]] (FP32; 0 where the row is
 * skipped).  rows distinct; rows of dz that none names are left as they were; dz may be z itself.  The residual's gradient is
 * dy. */
mx_status mx_moe_combine_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, int64_t total_rows, int64_t hidden,
                                  const int32_t* rows, const float* weights, int64_t tokens, int64_t top_k, void* dz,
                                  int64_t lddz, float* dweights, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXNUM_LAYER_H */
