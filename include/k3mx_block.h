/*
 * k3mx_block.h - the steps between the products of an expert block of any
 * shape, and their gradients: pairs sorted by expert, rows taken to their
 * experts and back with the routing weights, the gated activation between the
 * two products, and the backward passes that read activations saved in 8 bits.
 *
 * The contract is k3mx.h's: device pointers and sizes, status codes, no device
 * memory allocated, calls asynchronous on `stream`, arguments refused and
 * never defaulted.  Every argument may come from the kernel launched right
 * before on the stream.  Calls that share a workspace must be ordered by the
 * caller.  All results are deterministic.
 *
 * A pair is a token and one of its `topk` choices: pair t * topk + k.  What
 * the library calls MXFP8 here is K3MX_MXFP8 of k3mx_mx.h: e4m3 codes
 * [rows][cols] and a ue8m0 byte for 32 columns [rows][cols/32].  An activation
 * saved in 8 bits is an MXFP8 matrix, made by k3mx_mx_quantize or by
 * k3mx_situ_mx itself.
 */
#ifndef K3MX_BLOCK_H_
#define K3MX_BLOCK_H_

#include "k3mx_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { K3MX_E4M3 = 2 };              /* dtype of k3mx_dispatch: MXFP8 codes, beside K3MX_F32, K3MX_BF16 */

#define K3MX_BLOCK_MAX_PAIRS (1 << 24)                  /* n_tokens * topk */
#define K3MX_BLOCK_MAX_ELEMENTS (INT64_C(1) << 38)      /* rows x columns of k3mx_dispatch and k3mx_combine */

/*
 * Pairs in the order of their experts, pairs of one expert in pair order.
 *   idx     [n_tokens][topk]: the pair's expert in 0..n_experts-1, or -1: dropped
 *           (another value: dropped too, and k3mx_device_status reports
 *           K3MX_EINVAL with the pair).  An expert may come twice.
 *   offsets [n_experts + 1]: expert e has rows offsets[e]..offsets[e + 1] - 1
 *   perm    [n_tokens][topk] or NULL: the pair of each row; entries from
 *           offsets[n_experts] on are left as they are
 *   place   [n_tokens][topk]: the row of each pair, -1 where it was dropped
 *   workspace: device, 16-byte aligned, >= k3mx_sort_workspace_size(...) bytes
 *   (0 for few pairs: then it may be NULL)
 *   n_tokens, topk >= 1, n_tokens * topk <= K3MX_BLOCK_MAX_PAIRS,
 *   1 <= n_experts <= K3MX_MX_MAX_GROUPS.  Arrays 4-byte aligned.
 */
size_t k3mx_sort_workspace_size(int n_tokens, int topk, int n_experts);
k3mx_status k3mx_sort(int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, int n_tokens,
                      int topk, int n_experts, void *workspace, size_t ws_bytes, k3mx_stream_t stream);

/*
 * rows[place[t][k]] = x[t]: a token's row to each of its pairs.
 *   x      [n_tokens] rows of width values, ldx elements apart (width <= ldx
 *          <= 2^32), dtype K3MX_F32, K3MX_BF16 or K3MX_E4M3 (bytes)
 *   x_scales [n_tokens][width/32], scales [n_rows][width/32]: moved likewise;
 *          for K3MX_E4M3 (width a multiple of 32), else both NULL
 *   place  [n_tokens][topk] as k3mx_sort writes it: -1 is skipped, another
 *          value outside 0..n_rows-1 too, and k3mx_device_status reports
 *          K3MX_EINVAL with the pair; a row that two tokens' pairs name holds
 *          parts of either
 *   rows   [n_rows][width] and scales: rows that no pair names are left as
 *          they are
 *   n_tokens * topk <= K3MX_BLOCK_MAX_PAIRS, 1 <= n_rows <= K3MX_MX_MAX_ROWS,
 *   1 <= width <= K3MX_MX_MAX_COLS, n_rows * width and n_tokens * width
 *   <= K3MX_BLOCK_MAX_ELEMENTS.  Pointers aligned to their elements; where all
 *   rows begin at multiples of 16 bytes they are moved with wide accesses.
 * Its gradient is k3mx_combine without weights.
 */
k3mx_status k3mx_dispatch(void *rows, uint8_t *scales, const void *x, const uint8_t *x_scales, int64_t ldx,
                          int dtype, const int32_t *place, int n_tokens, int topk, int n_rows, int width,
                          k3mx_stream_t stream);

/*
 * y[t] = base[t] + sum_k w[t][k] rows[place[t][k]], in fp32, k rising, base
 * last, one rounding to y's type: a token's bits do not depend on the others of
 * the call.
 *   rows  [n_rows][width], rows_dtype K3MX_F32 or K3MX_BF16
 *   place [n_tokens][topk] as for k3mx_dispatch; skipped pairs add nothing
 *   w     [n_tokens][topk] fp32, or NULL: all 1
 *   base  [n_tokens][width] of y's type, or NULL: 0; may be y itself
 *   y     [n_tokens][width], y_dtype K3MX_F32 or K3MX_BF16, written whole
 *   sizes and alignment as for k3mx_dispatch
 */
k3mx_status k3mx_combine(void *y, int y_dtype, const void *rows, int rows_dtype, const int32_t *place,
                         const float *w, const void *base, int n_tokens, int topk, int n_rows, int width,
                         k3mx_stream_t stream);

/*
 * The gradients of k3mx_combine (base's is dy itself): for each pair
 *   drows[place] = w dy[t] (one rounding to rows' type),
 *   dw = sum_c dy[t][c] rows[place][c] (fp32; 0 for a skipped pair).
 *   dy    [n_tokens] rows, lddy elements apart (width <= lddy <= 2^32)
 *   drows [n_rows][width] of rows' type; rows that no pair names are left as
 *         they are (one that two pairs name holds parts of either's); may be
 *         rows itself where no two pairs name one row
 *   dw    [n_tokens][topk]
 *   otherwise as k3mx_combine
 */
k3mx_status k3mx_combine_backward(void *drows, float *dw, const void *dy, int64_t lddy, int dy_dtype,
                                  const void *rows, int rows_dtype, const int32_t *place, const float *w,
                                  int n_tokens, int topk, int n_rows, int width, k3mx_stream_t stream);

/*
 * SiTU-GLU of gate | up rows (the activation of k3mx_expert_ffn):
 *   h = 4 tanh(g/4) sigma(g) * 25 tanh(u/25), g = gu[r][0..inter-1],
 *   u = gu[r][inter..2 inter-1],
 * in MXFP8, as the next product reads it, and g | u in MXFP8 for the backward
 * pass.
 *   gu     [rows] rows of 2 inter values, ldgu elements apart (2 inter <= ldgu
 *          <= 2^32), dtype K3MX_F32 or K3MX_BF16
 *   codes  [rows][inter], scales [rows][inter/32]: written
 *   saved  [rows][2 inter], saved_scales [rows][2 inter/32]: written, or both
 *          NULL: nothing saved
 *   1 <= rows <= K3MX_MX_MAX_ROWS, inter a multiple of 32, 2 inter <=
 *   K3MX_MX_MAX_COLS.  Pointers 16-byte aligned (scales: any), ldgu a multiple
 *   of 16 bytes.
 * What is saved is exactly k3mx_mx_quantize's.  The codes and scales of h are
 * those that k3mx_mx_quantize's definition gives for h itself, formed within
 * 2^-29 where |h| > 2^-96; but where g < -16 they are those of a value within
 * 2^-15 of h, and where g < -87 h may be taken for 0.  Infinite g and u have
 * their limits; a NaN makes its block NaN.
 */
k3mx_status k3mx_situ_mx(uint8_t *codes, uint8_t *scales, uint8_t *saved, uint8_t *saved_scales,
                         const void *gu, int64_t ldgu, int dtype, int rows, int inter, k3mx_stream_t stream);

/*
 * The gradient of k3mx_situ_mx at the g and u that were saved:
 *   dg = dh (dh/dg), du = dh (dh/du), one rounding to dgu's type.
 *   dh  [rows] rows of inter values, lddh elements apart, dtype K3MX_F32 or
 *       K3MX_BF16
 *   dgu [rows][2 inter] of the same type, written: dg | du
 *   sizes and alignment as for k3mx_situ_mx
 * The derivatives are within 2^-18 (1 + (|g| + |u|)/16) of themselves (dh/dg:
 * of its two terms' magnitudes) and within 2^-119.  A saved block of scale 255
 * (it held Inf or NaN) makes its columns' dg and du NaN.
 */
k3mx_status k3mx_situ_mx_backward(void *dgu, const void *dh, int64_t lddh, int dtype, const uint8_t *saved,
                                  const uint8_t *saved_scales, int rows, int inter, k3mx_stream_t stream);

/*
 * The gradient of n = s g / sqrt(mean(s^2) + eps) (k3mx_rmsnorm_mx) at the s
 * that was saved, per row t, with k = 1 / sqrt(mean(s^2) + eps), a = g dn:
 *   dx = dres + k (a - s k^2 mean(a s)) (one rounding to its type),
 *   dweight = sum_t dn s k (fp32).
 *   dn   [n_tokens] rows of width values, lddn elements apart (width <= lddn
 *        <= 2^32), dtype K3MX_F32 or K3MX_BF16
 *   dres [n_tokens][width] of the same type: the gradient that s has from
 *        elsewhere (the residual stream's); NULL: 0; may be dx itself
 *   saved [n_tokens][width], saved_scales [n_tokens][width/32]: s in MXFP8
 *   g    [width] bf16; eps finite, >= 0
 *   dx   [n_tokens][width] of dn's type, dweight [width]: written
 *   workspace: device, 16-byte aligned,
 *        >= k3mx_rmsnorm_mx_backward_workspace_size(...) bytes
 *   sizes as for k3mx_rmsnorm_mx.  Pointers 16-byte aligned (saved_scales:
 *   any), lddn a multiple of 16 bytes.
 * Rows are added in fp32, at most 1024 by one thread, then the parts.  Sums of
 * a row that leave fp32, or its normal numbers, are formed of scaled values:
 * where sqrt(mean(s^2) + eps) >= 2^-126 and g dn, normal or 0, and what dx adds
 * up are finite, dx is within (width / 1024 + 62) 2^-24 of the magnitudes it
 * adds up, and within 2^-117, before its rounding.  A row of zeros with eps = 0
 * has no gradient: NaN.
 */
size_t k3mx_rmsnorm_mx_backward_workspace_size(int n_tokens, int width);
k3mx_status k3mx_rmsnorm_mx_backward(void *dx, float *dweight, const void *dn, int64_t lddn, const void *dres,
                                     int dtype, const uint8_t *saved, const uint8_t *saved_scales,
                                     const uint16_t *g, float eps, int n_tokens, int width, void *workspace,
                                     size_t ws_bytes, k3mx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* K3MX_BLOCK_H_ */
