/*
 * qat_mx.h -- C ABI of microscaled 4-bit floating point (MXFP4) on gfx950:
 * quantisation, and the linear layer's product on the matrix cores' 4-bit
 * rate, for any token count.
 *
 * The format (OCP Microscaling Formats specification 1.0, MXFP4): blocks of
 * 32 consecutive elements of a row share one scale 2^e, stored as the byte
 * e + 127 (E8M0); each element is an E2M1 code c: sign bit 3, magnitude
 * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[c & 7]. The value is magnitude * 2^e.
 *   codes  [rows][in / 2] uint8, element 2i in the low half of byte i
 *   scales [rows][in / 32] uint8
 * The byte 255 is a scale that is not a number: all 32 values are NaN.
 *
 * Conventions: those of qat.h (device pointers owned by the caller, 16-byte
 * aligned; checks before anything is enqueued; asynchronous on `stream`; a
 * QAT_* status returned; nothing allocated or kept), and
 * - dtype is QAT_F32, QAT_BF16 or QAT_F16 (16-bit patterns);
 * - in is a multiple of 32; rows and out are any positive counts; a row
 *   count M of 0 is a valid call that does nothing;
 * - ldx, ldy: elements from one row to the next, at least the row's length;
 *   rows of X start 16-byte aligned (ldx * element size a multiple of 16);
 *   ldy is free;
 * - a product's in is at most 2^20 and every operand smaller than 2 GiB.
 * Calls that share a workspace must not overlap in time.
 */
#ifndef QAT_MX_H
#define QAT_MX_H

#include "qat.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QAT_F32 = 0, QAT_BF16 = 1, QAT_F16 = 2 };

/*
 * Quantisation (the conversion of the specification's section 6.3): for a
 * block with largest magnitude a > 0,
 *   e = max(floor(log2 a) - 2, -127),  code = E2M1(x 2^-e),
 * rounded to nearest, ties to the even code, magnitudes above 6 saturating at
 * 6; the sign of zero is kept. A block of zeros has e = -127. A block that
 * holds an infinity or a NaN gets the scale byte 255 and zero codes.
 * X [rows][cols] of `dtype`, ldx apart, cols a multiple of 32. Outputs:
 * codes and scales (both or neither), X_hat [rows][cols] contiguous, the
 * values in X's type (exact: every value is representable there); either the
 * pair or X_hat may be NULL.
 */
int32_t qat_mx_quant(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, void* X_hat, hipStream_t stream);

/* Workspace bytes that serve both qat_mx_gemm and qat_mx_linear at these sizes;
 * 0 where neither needs one (a few tokens) and for invalid sizes. ws may be NULL
 * then. */
size_t qat_mx_ws_bytes(int64_t M, int64_t out, int64_t in);

/*
 * Y[m][o] = sum_k X_hat[m][k] W_hat[o][k] with both operands in MXFP4: exact
 * products, fp32 accumulation, one rounding to dtype (QAT_BF16 or QAT_F16).
 * X codes [M][in / 2], scales [M][in / 32]; W codes [out][in / 2], scales
 * [out][in / 32]; Y [M][out], ldy apart. An output whose row of X or W holds
 * a block of scale 255 is NaN.
 */
int32_t qat_mx_gemm(const uint8_t* X_codes, const uint8_t* X_scales, const uint8_t* W_codes,
                    const uint8_t* W_scales, int64_t M, int64_t out, int64_t in, int32_t dtype, void* Y,
                    int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * The linear layer on 16-bit activations: qat_mx_quant of X [M][in] (dtype
 * QAT_BF16 or QAT_F16, ldx apart), then the product of qat_mx_gemm; the
 * result is the same bit for bit.
 */
int32_t qat_mx_linear(const void* X, int64_t ldx, const uint8_t* W_codes, const uint8_t* W_scales, int64_t M,
                      int64_t out, int64_t in, int32_t dtype, void* Y, int64_t ldy, void* ws, size_t ws_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QAT_MX_H */
