/*
 * k3mx_mx.h - microscaled operators of any shape around the MXFP4 routed-
 * expert layer (k3mx.h): making the two microscaled formats, the norm that
 * writes one of them, and the products that read both.
 *
 * The contract is k3mx.h's: device pointers and sizes, status codes, no
 * device memory allocated, calls asynchronous on `stream`, arguments refused
 * and never defaulted.  None of these calls needs a workspace, and every
 * argument may come from the kernel launched right before on the stream.
 *
 * Formats.  A matrix of `rows` x `cols` (cols a multiple of 32) is two
 * row-major arrays, codes and scales [rows][cols/32]; the 32 columns of a
 * block share one ue8m0 byte s, value = code value * 2^(s - 127).
 *   K3MX_MXFP4  codes [rows][cols/2], e2m1, two per byte, the low nibble the
 *               even column: the library's weight format.  s = 255: the block
 *               contributes nothing.
 *   K3MX_MXFP8  codes [rows][cols], e4m3, one per byte: the format of the
 *               activations that the products below read.  s = 255: the
 *               block is NaN.
 */
#ifndef K3MX_MX_H_
#define K3MX_MX_H_

#include "k3mx.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { K3MX_MXFP4 = 0, K3MX_MXFP8 = 1 };

#define K3MX_MX_MAX_ROWS   (1 << 24)   /* rows of a microscaled matrix       */
#define K3MX_MX_MAX_COLS   (1 << 20)   /* its columns                        */
#define K3MX_MX_MAX_ELEMENTS (INT64_C(1) << 40)  /* rows x columns           */
#define K3MX_NORM_MAX_WIDTH 32768      /* columns of k3mx_rmsnorm_mx         */
#define K3MX_MX_MAX_IN     65536       /* inner width of the products        */
#define K3MX_MX_MAX_GROUPS 1024        /* weight matrices of k3mx_mx_grouped */

/*
 * x -> codes and scales.  Per block of 32 columns, m = max |x|: the scale is
 * 2^e with the smallest e >= -127 for which m <= top * 2^e (top = 6 for
 * e2m1, 448 for e4m3), so nothing saturates (a quantiser that takes the
 * exponent of m less that of the top, as the OCP microscaling specification
 * suggests, gives a smaller scale where m's mantissa is above the top's, and
 * saturates there); code = x / 2^e rounded to the
 * nearest code value, ties to the even code; byte e + 127.  An all-zero
 * block has byte 0.  A block that holds Inf or NaN gets byte 255 and zero
 * codes; for K3MX_MXFP4, where products skip such a block, that is also
 * reported by k3mx_device_status (K3MX_EINVAL, detail = the row).
 *   x [rows] rows of cols values, ldx elements apart (cols <= ldx <= 2^32), x_dtype
 *   K3MX_F32 or K3MX_BF16, aligned to its element; rows whose address and
 *   pitch are multiples of 16 bytes are read with wide loads
 *   codes, scales: written, contiguous, codes 16-byte aligned
 *   1 <= rows <= K3MX_MX_MAX_ROWS; cols a multiple of 32 up to
 *   K3MX_MX_MAX_COLS
 * Exact: every code and scale is the one the definition gives.
 */
k3mx_status k3mx_mx_quantize(uint8_t *codes, uint8_t *scales, const void *x, int x_dtype,
                             int rows, int cols, int64_t ldx, int format, k3mx_stream_t stream);

/*
 * codes and scales -> y [rows][cols] (contiguous, written; y_dtype K3MX_F32:
 * exact, K3MX_BF16: rounded to nearest even where bf16 has no such value).
 * Blocks of scale 255 give 0 (K3MX_MXFP4) or NaN (K3MX_MXFP8).  y and codes
 * 16-byte aligned.
 */
k3mx_status k3mx_mx_dequantize(void *y, int y_dtype, const uint8_t *codes, const uint8_t *scales,
                               int rows, int cols, int format, k3mx_stream_t stream);

/*
 * Residual addition, RMSNorm and quantisation to K3MX_MXFP8, per row t:
 *   s = x + residual (fp32), n = s * g / sqrt(mean(s^2) + eps) (fp32),
 *   codes, scales = k3mx_mx_quantize of n,
 *   sum = s and normed = n, each rounded to its type once.
 *   x [n_tokens] rows ldx elements apart (width <= ldx <= 2^32), dtype K3MX_F32
 *   or K3MX_BF16
 *   residual [n_tokens][width], the same type; NULL: s = x and sum is not
 *   written (pass NULL)
 *   sum [n_tokens][width], x's type, written; may be residual itself, or x
 *   where ldx = width
 *   normed [n_tokens][width] bf16, written, or NULL
 *   g [width] bf16; eps finite, >= 0
 *   codes [n_tokens][width], scales [n_tokens][width/32]: written
 *   1 <= n_tokens <= K3MX_MX_MAX_ROWS, width a multiple of 32 up to
 *   K3MX_NORM_MAX_WIDTH.  All pointers 16-byte aligned (scales: any), ldx a
 *   multiple of 16 bytes.
 * |n - exact| <= 2^-20 |exact| for finite rows s whose root mean square lies
 * in 2^-63 .. 2^120 (squares may leave fp32), where n and the factor
 * g / sqrt(mean + eps) are normal fp32 numbers.
 */
k3mx_status k3mx_rmsnorm_mx(uint8_t *codes, uint8_t *scales, void *sum, uint16_t *normed,
                            const void *x, int64_t ldx, const void *residual, int dtype,
                            const uint16_t *g, float eps, int n_tokens, int width,
                            k3mx_stream_t stream);

/*
 * y[t][n] = sum_c x[t][c] w[n][c] with x in K3MX_MXFP8 and w in K3MX_MXFP4:
 *   codes [n_tokens][in], scales [n_tokens][in/32]
 *   packed [out][in/2], wscales [out][in/32]
 *   y [n_tokens][out] (written), y_dtype K3MX_F32 or K3MX_BF16 (one rounding)
 *   1 <= n_tokens, out <= K3MX_MX_MAX_ROWS; in a multiple of 128 up to
 *   K3MX_MX_MAX_IN
 * y, codes 16-byte, packed 32-byte, scales and wscales 4-byte aligned.  The
 * tensor cores multiply the codes exactly and add in fp32 with cut, not
 * rounded, addends, 1024 columns at a time for K3MX_F32 and 8192 for
 * K3MX_BF16; these sums are added in fp32.  |error| <= 4e-5 * sum_c |x w| for
 * K3MX_F32 and 3e-4 * sum_c |x w| for K3MX_BF16 (before y's rounding),
 * reached where a large term is followed by many that are 2^-26 of it; for
 * terms of mixed signs and sizes it is below 1e-5.  A weight block
 * of scale 255 adds exactly 0 (they are taken to be rare: one in every 128
 * outputs x 512 columns makes a call three to four times slower); a NaN code
 * or scale of x makes its whole row
 * of y NaN.  Deterministic.
 */
k3mx_status k3mx_mx_linear(void *y, int y_dtype, const uint8_t *codes, const uint8_t *scales,
                           const uint8_t *packed, const uint8_t *wscales, int n_tokens, int in,
                           int out, k3mx_stream_t stream);

/*
 * k3mx_mx_linear by groups of rows, each with a weight matrix of its own:
 * rows offsets[g] <= r < offsets[g + 1] use packed[g], wscales[g].
 *   codes [n_rows][in], scales [n_rows][in/32], y [n_rows][out]
 *   packed [n_groups][out][in/2], wscales [n_groups][out][in/32]
 *   offsets [n_groups + 1] int32, DEVICE, rising from >= 0 to <= n_rows
 *   (as k3mx_group writes it).  A group may be empty; rows of no group are
 *   left as they are.  A group whose offsets fall, or leave 0..n_rows, is
 *   skipped and k3mx_device_status reports K3MX_EINVAL with its index.
 *   1 <= n_rows <= K3MX_MX_MAX_ROWS, 1 <= n_groups <= K3MX_MX_MAX_GROUPS,
 *   n_groups * out <= 2^30; otherwise as k3mx_mx_linear; offsets 4-byte
 *   aligned.
 */
k3mx_status k3mx_mx_grouped(void *y, int y_dtype, const uint8_t *codes, const uint8_t *scales,
                            const uint8_t *packed, const uint8_t *wscales, const int32_t *offsets,
                            int n_groups, int n_rows, int in, int out, k3mx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* K3MX_MX_H_ */
