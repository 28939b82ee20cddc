/*
 * signrot.h -- C ABI of libsignrot, SignRot's online activation path on
 * AMD Instinct MI355X (gfx950).
 *
 * The method (pages: the SignRot abstract, arXiv 2611.16502, and the explainer
 * "SignRot for 4-bit LLM quantization -- Sign-adjusted Hadamard rotation"):
 * at the input of an LLM down-projection every token x (a row of n bf16
 * values) is rotated by an orthonormal Hadamard matrix, y = x.H / sqrt(n)
 * (explainer, paragraph on rotation: every entry of H is +-1/sqrt(n), applied
 * with a fast Walsh-Hadamard transform, paragraph on the down-projection); the
 * columns of H are sign-flipped by a calibrated vector d so that the one
 * massive-outlier channel reaches every output with the same sign
 * (explainer, paragraph on the sign adjustment; abstract); and the result is
 * quantized per token to 16 evenly spaced levels between the token's minimum
 * and maximum, an asymmetric INT4 code with a zero-point (explainer,
 * paragraphs on the quantizer and on symmetric versus asymmetric quantizers).
 *
 * Hadamard order (n <= 32768).  n = 2^k (k >= 1) uses the Sylvester matrix in
 * natural order, H[i][j] = (-1)^popcount(i & j).  Any other n = o * 2^v (o
 * odd) uses H = H_m (x) H_{2^k} with index i = a * 2^k + b (a < m, b < 2^k),
 * where m = o * 2^j for the smallest j >= 2 for which Paley's construction I
 * (q = m - 1 a prime power = 3 mod 4: H_m = I + S, S the Jacobsthal matrix of
 * the quadratic character of GF(q) bordered by a row of +1 and a column of -1)
 * or, failing that, construction II (q = m/2 - 1 a prime power = 1 mod 4:
 * H_m = C (x) [[1,1],[1,-1]] + I (x) [[1,-1],[-1,-1]], C the symmetric
 * conference matrix) exists with m <= 512.  GF(p^e) is GF(p)[t] modulo the
 * first monic irreducible polynomial in lexicographic order of its
 * coefficients.  So 28 * 2^k uses H28 over GF(27) = GF(3)[t]/(t^3 + 2t + 1),
 * 13824 = 108 * 2^7 uses construction I over GF(107), and 11008 = 344 * 2^5
 * uses construction I over GF(7^3) (172 * 2^6 has no Paley factor).  The
 * pages only ask for some Hadamard matrix; these are the library's choices.
 * Orientation: y_j = sum_i x_i H[i][j] (x is a row vector; the outlier at
 * channel c reaches the outputs through row c of H).
 *
 * Conventions shared by every call:
 *   - All sizes are element counts.  Device pointers are plain HIP device
 *     addresses (e.g. from torch).  `stream` is a hipStream_t passed as
 *     void*; NULL means the default stream.  Every tensor is owned by the
 *     caller; the library keeps no pointer after a call returns.
 *   - Activations are bf16 bit patterns, row-major [tokens][ld], ld >= n,
 *     with the base pointer 16-byte aligned and ld a multiple of 8 (so each
 *     row starts 16-byte aligned).
 *   - Calls return a signrot_status.  Argument errors are detected on the
 *     host before any HIP call and leave every output untouched.  A HIP
 *     error returns SIGNROT_EHIP; outputs are then unspecified and
 *     signrot_last_error() holds the HIP message.  Nothing throws.
 *   - tokens == 0 is a successful no-op (null pointers are then allowed).
 *   - Non-finite inputs, or inputs so large that the rotated values overflow
 *     binary32, give unspecified outputs (no checks on the hot path).
 *   - Calls are reentrant; concurrent calls on different streams are allowed.
 *   - Device memory the library itself allocates: (1) per device, the sign
 *     table of an outer factor H_m with m != 28 (and the transposed table for
 *     the outer-order MFMA kernel), at most 32 KiB each, copied there by the
 *     first call that needs it (hipMalloc + hipMemcpy) and kept until the
 *     process ends; a first call made while `stream` is being captured into
 *     a graph returns SIGNROT_EHIP instead and leaves the capture intact.
 *     H28 (every width 28 * 2^k) and the Sylvester-only widths with their own
 *     kernel need no table: H28 travels by value in the kernel arguments.
 *     (2) Stream-ordered scratch (hipMallocAsync / hipFreeAsync on `stream`),
 *     named at each call that uses it.  Nothing else.
 */
#ifndef SIGNROT_H
#define SIGNROT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SIGNROT_OK = 0,
  SIGNROT_EINVAL = -1,          /* bad pointer, size, stride or alignment   */
  SIGNROT_EUNSUPPORTED_N = -2,  /* n has no factorisation of the rule above  */
  SIGNROT_EHIP = -3             /* a HIP runtime call or launch failed       */
} signrot_status;

/* 1 if n factors by the rule above (n <= 32768), else 0. */
int signrot_supported_n(int64_t n);

/* The outer order m of n by that rule (1 for n = 2^k), or 0 when n is
 * unsupported. */
int signrot_outer_order(int64_t n);

/*
 * Calibration (abstract: one calibration forward pass; explainer, paragraph
 * on the sign adjustment: the channel with the largest absolute activation,
 * and a flip of each column j of H by the sign of that row's entry).
 *
 *   x_bf16  device, [tokens][ld] bf16 calibration batch (tokens < 2^28).
 *   d_out   device, [n] int8: d_j = sign(M_c) * H[c][j], values +1/-1, where
 *           c is the channel of the largest |x| over the batch and M_c the
 *           signed value there.  Ties: smallest channel, then smallest token.
 *           sign(+0) = sign(-0) = +1.
 *   c_out   host, may be NULL: the channel c.
 *   t_out   host, may be NULL: the token t holding M_c.
 *   mc_out  host, may be NULL: M_c widened to float.
 *
 * Enqueues its kernels on `stream`, then synchronizes that stream (the host
 * outputs need the result).  Uses a 16-byte stream-ordered scratch buffer
 * (hipMallocAsync / hipFreeAsync).  Unlike the other calls, tokens == 0 ->
 * SIGNROT_EINVAL: an empty batch has no largest activation, so there is no
 * channel to find.  t_out is reported in addition to c and M_c so that a
 * caller can check the argmax against its own data.
 */
int signrot_calibrate(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld,
                      int8_t* d_out, int32_t* c_out, int64_t* t_out, float* mc_out,
                      void* stream);

/*
 * signrot_calibrate without any allocation, for callers that cannot allocate
 * device memory (tight serving loops, harnesses that forbid hipMalloc).  Same
 * arguments, outputs and argument errors as signrot_calibrate.  The 16-byte
 * argmax record lives in a static device array of the library (one per GPU,
 * kept until the process ends; its address is looked up once per device)
 * instead of a stream-ordered allocation; each call clears it first.  The
 * record's size does not depend on the input, so no input is too large for
 * it.  Only widths whose Hadamard factors need no device table are taken,
 * n = 2^k and n = 28 * 2^k; any other supported n -> SIGNROT_EUNSUPPORTED_N
 * (use signrot_calibrate).  Calls that overlap on one GPU (several streams or
 * threads) race on the shared record: serialize them.  Synchronizes `stream`
 * before returning, as signrot_calibrate does.
 */
int signrot_calibrate_noalloc(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld,
                              int8_t* d_out, int32_t* c_out, int64_t* t_out, float* mc_out,
                              void* stream);

/*
 * The online path: y = (x . H / sqrt(n)) (.) d, then per-token asymmetric
 * INT4 (explainer, paragraphs on rotation, on the sign adjustment and on the
 * quantizer).  Per token, with mn = min_j y_j and mx = max_j y_j:
 *   scale = (mx - mn) / 15, or 1 when mx == mn;
 *   zero  = -mn / scale, in code units, neither rounded nor clamped;
 *   q_j   = clamp(round((y_j - mn) / scale), 0, 15), round to nearest.
 *
 *   x_bf16  device, [tokens][ld] bf16.
 *   d       device, [n] int8, 16-byte aligned, every entry +1 or -1 (any
 *           other value gives unspecified output).  When d = sigma * (row c of H) -- the form
 *           signrot_calibrate produces -- the library recognises it and
 *           evaluates the identical quantity as ((x - x_c e_c) . H) (.) d plus
 *           the constant sigma * x_c / sqrt(n), so the outlier is added once
 *           instead of being rounded through every butterfly stage.
 *   codes   device, [tokens][n/2] uint8, 16-byte aligned: code of channel 2m
 *           in the low nibble of byte m, channel 2m+1 in the high nibble.
 *   scale   device, [tokens] float.
 *   zero    device, [tokens] float.
 *   y_out   device, [tokens][n] float, 16-byte aligned, or NULL: the
 *           rotated, flipped values in binary32 (a debugging output; the
 *           codes do not depend on it).
 *
 * A misaligned x, d, codes or y_out, ld < n or ld not a multiple of 8, a null
 * pointer (tokens > 0) or tokens < 0 -> SIGNROT_EINVAL; an unsupported n ->
 * SIGNROT_EUNSUPPORTED_N.
 *
 * Asynchronous: returns once the kernel is enqueued on `stream`.  Arithmetic
 * is binary32 throughout.
 */
int signrot_rotate_quant_int4(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld,
                              const int8_t* d, uint8_t* codes, float* scale, float* zero,
                              float* y_out, void* stream);

/*
 * The online path for the sign vector in its calibrated form, given by the
 * outlier channel c and sigma = sign(M_c) instead of as the vector d
 * (explainer, paragraph on the sign adjustment: each column j of H is
 * multiplied by the sign of the outlier row's entry, so d_j = sigma * H[c][j]
 * with H the library's unnormalised +-1 matrix).  Computes exactly what
 * signrot_rotate_quant_int4 computes for that d, without reading d or
 * deciding its form on the device: about 1.7 us less per decode-sized call at
 * n = 14336, and under 1 us on a batch of 8192 tokens.
 *
 *   c       the channel signrot_calibrate returns in c_out, 0 <= c < n.
 *   sigma   +1 or -1: the sign of M_c (mc_out), with sign(+-0) = +1.
 *   the other arguments as for signrot_rotate_quant_int4.
 *
 * c outside [0, n) or sigma not +-1 -> SIGNROT_EINVAL; the other errors as
 * for signrot_rotate_quant_int4.  For the widths without a fast kernel, d is
 * built in a stream-ordered n-byte scratch (hipMallocAsync / hipFreeAsync).
 * Asynchronous.
 */
int signrot_rotate_quant_int4_outlier(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld, int64_t c,
                                      int sigma, uint8_t* codes, float* scale, float* zero, float* y_out,
                                      void* stream);

/*
 * A variant with an integer zero-point (the GyRot abstract, on the pages as a
 * related paper: asymmetric quantization reformulated with a rounded
 * zero-point so that dequantization is integer arithmetic times one scale).
 * With the same scale s = (mx - mn) / 15 (1 when mx == mn):
 *   zero = rint(-mn / s), an integer (stored exactly in the float output);
 *   q_j  = clamp(rint(y_j / s) + zero, 0, 15),
 * so y_hat = s * (q - zero) with (q - zero) an integer.  Rounding the
 * zero-point moves the window of 16 levels by at most half a step, so
 * y / s + zero stays in [-0.5, 15.5] and every value is still within s/2 of
 * its level.
 *
 * The sign vector is given as (c, sigma) as for
 * signrot_rotate_quant_int4_outlier; there is no y_out.  Same arguments,
 * alignment and errors as that call.  Asynchronous.
 */
int signrot_rotate_quant_int4_zint(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld, int64_t c, int sigma,
                                   uint8_t* codes, float* scale, float* zero, void* stream);

/*
 * The online path with its producer fused in (explainer, paragraph on the
 * down-projection: the gated nonlinearity between the up/gate projections and
 * the down-projection is why the rotation has to run online).  The
 * down-projection input is computed from the producer's two operands,
 *   x = bf16(SiLU(gate) * up),  SiLU(z) = z / (1 + e^-z),
 * in binary32 and rounded once to bf16 (nearest, ties to even), and then goes
 * through exactly what signrot_rotate_quant_int4_outlier computes for that x;
 * x itself never reaches memory.  (SwiGLU as the gated unit is a reading: the
 * pages name the nonlinearity, not its formula.)  The binary32 SiLU is within
 * about 2e-6 relative of the exact value for |gate| <= 16, so x equals the
 * exactly rounded bf16 value except where that value lies that close to a
 * point halfway between two bf16 numbers.
 *
 *   gate_bf16, up_bf16  device, [tokens][ld] bf16 each, same ld, 16-byte
 *                       aligned; ld >= n, ld % 8 == 0.
 *   c, sigma            the calibrated sign vector, as for
 *                       signrot_rotate_quant_int4_outlier (calibrated on x).
 *   codes, scale, zero, y_out   as for signrot_rotate_quant_int4.
 *
 * Only the widths with a fast kernel: n = 3584, 7168, 14336, 28672, 4096,
 * 8192, 16384; any other supported n -> SIGNROT_EUNSUPPORTED_N.  Other errors
 * as for signrot_rotate_quant_int4_outlier (a null or misaligned up ->
 * SIGNROT_EINVAL).  No allocation.  Asynchronous.
 */
int signrot_swiglu_rotate_quant_int4(const void* gate_bf16, const void* up_bf16, int64_t tokens, int64_t n, int64_t ld,
                                     int64_t c, int sigma, uint8_t* codes, float* scale, float* zero, float* y_out,
                                     void* stream);

/*
 * Dequantization (explainer, paragraph on the 4-bit quantizer: a token's 16
 * levels are spread evenly from its smallest to its largest value, so code q
 * stands for the level mn + q * scale; paragraph on symmetric versus
 * asymmetric quantizers: the asymmetric form carries a zero-point):
 * y_hat[t][j] = scale[t] * (q_j - zero[t]).
 *
 *   codes   device, [tokens][n/2] uint8, as signrot_rotate_quant_int4 or
 *           signrot_rotate_quant_int4_zint writes them.
 *   scale   device, [tokens] float; zero device, [tokens] float.
 *   y_hat   device, [tokens][n] float, 8-byte aligned.
 *
 * n must be supported (SIGNROT_EUNSUPPORTED_N otherwise); a null pointer or a
 * misaligned y_hat (tokens > 0) or tokens < 0 -> SIGNROT_EINVAL.  No
 * allocation.  Asynchronous.
 */
int signrot_dequant(const uint8_t* codes, const float* scale, const float* zero,
                    int64_t tokens, int64_t n, float* y_hat, void* stream);

/*
 * Offline weight fold (explainer, paragraph on the sign adjustment: the same
 * flip is folded into the weights offline; paragraph on rotation: H / sqrt(n)
 * is orthogonal, so rotating both factors of a product leaves it unchanged).
 * For a down-projection out = x . W^T with W [rows][n] (one row per output
 * feature), W' = W . H . D / sqrt(n): every row w of W becomes
 * (w . H / sqrt(n)) (.) d, the very transform applied to the activations, so
 * that out = x' . W'^T with x' = (x . H / sqrt(n)) (.) d.
 *
 *   w_bf16  device, [rows][ld] bf16, 16-byte aligned, ld >= n, ld % 8 == 0.
 *   d       device, [n] int8, 16-byte aligned, entries +1/-1 (the vector
 *           signrot_calibrate produced for the activations).
 *   w_out   device, [rows][n] float, 16-byte aligned.
 *
 * Runs the rotation kernels of signrot_rotate_quant_int4, whose INT4 codes
 * go to a stream-ordered scratch of rows * (n/2 + 8) bytes (hipMallocAsync /
 * hipFreeAsync on `stream`) and are discarded.  Asynchronous.  rows == 0 is a
 * no-op; argument errors as for signrot_rotate_quant_int4.
 */
int signrot_fold_weights(const void* w_bf16, int64_t rows, int64_t n, int64_t ld, const int8_t* d, float* w_out,
                         void* stream);

/*
 * Row sums of a folded weight, rowsum[k] = sum_j w[k][j] (explainer,
 * paragraph on symmetric versus asymmetric quantizers: the zero-point's share
 * of the product is the zero-point times a precomputed sum of the weights).
 * Computed once per weight, offline.
 *
 *   w_bf16  device, [rows][ld] bf16 (W' = W . H . D / sqrt(n) rounded to
 *           bf16), ld >= n; no alignment requirement.
 *   rowsum  device, [rows] float: the exact sum of the bf16 values,
 *           accumulated in binary64 and rounded once.
 *
 * rows == 0 is a no-op; rows < 0, n < 0, ld < n or a null pointer ->
 * SIGNROT_EINVAL.  Any n (the sum does not depend on the Hadamard order).
 * Asynchronous.
 */
int signrot_weight_rowsum(const void* w_bf16, int64_t rows, int64_t n, int64_t ld, float* rowsum, void* stream);

/*
 * The consumer of the INT4 activations: the down-projection on the folded
 * weight, out = yhat . W'^T with yhat = scale * (q - zero), evaluated as
 * (explainer, paragraph on symmetric versus asymmetric quantizers)
 *
 *   out[t][k] = scale[t] * (sum_j q[t][j] * w[k][j] - zero[t] * rowsum[k]),
 *
 * so the product itself runs on the unsigned integer codes.
 *
 *   codes   device, [tokens][n/2] uint8, as signrot_rotate_quant_int4 writes
 *           them (channel 2m in the low nibble of byte m).
 *   scale   device, [tokens] float; zero device, [tokens] float.
 *   w_bf16  device, [rows][ldw] bf16: row k is output feature k of W'.
 *   rowsum  device, [rows] float, from signrot_weight_rowsum.
 *   out     device, [tokens][rows] float.
 *
 * n even and >= 2 (any Hadamard order), ldw >= n.  The MFMA kernel runs when
 * n % 64 == 0, ldw % 8 == 0, rows * ldw < 2^31 and codes and w are 16-byte
 * aligned; other shapes take a plain one-thread-per-output kernel.  The
 * integer-by-bf16 products are exact; they are summed in binary32 (in an
 * order that differs between the two kernels).  tokens == 0 or rows == 0 is a
 * no-op; negative sizes, odd n, ldw < n, tokens or rows >= 2^31 or a null
 * pointer -> SIGNROT_EINVAL.  Asynchronous.
 */
int signrot_int4_linear(const uint8_t* codes, const float* scale, const float* zero, int64_t tokens, int64_t n,
                        const void* w_bf16, int64_t ldw, const float* rowsum, int64_t rows, float* out,
                        void* stream);

/* Which kernel signrot_int4_linear would launch for these operands (a static
 * string), or NULL when the arguments are invalid. */
const char* signrot_int4_linear_kernel_name(const uint8_t* codes, int64_t tokens, int64_t n, const void* w_bf16,
                                            int64_t ldw, int64_t rows);

/*
 * ---- 8-bit integer products and the norms around a block ------------------
 *
 * The projections of a block whose inputs need no online rotation run on
 * 8-bit integers (one scale per token, one per output channel), the
 * down-projection runs on the rotated INT4 codes with 8-bit weights, and the
 * norms around the block hand their result to the product as integer codes.
 */

/* Element types of the calls below. */
typedef enum { SIGNROT_F32 = 0, SIGNROT_BF16 = 1 } signrot_type;

/*
 * Symmetric per-token INT8 quantizer.  Per row, with a = max_j |x_j|:
 *   scale = a / 127, or 1 when a == 0;
 *   q_j   = rint(127 x_j / a) (ties to even; 0 when a == 0), -127 .. 127.
 * The scale is the binary32 quotient correctly rounded; the codes are the
 * exact rint of the rational 127 x_j / a (a bf16 row makes it decidable in
 * binary32), so they do not depend on the order of anything.  Run on the rows
 * of a weight [rows][n] it is the per-output-channel weight quantizer.  A row
 * that holds an infinity or NaN gets a non-finite scale (and unspecified
 * codes), so every product with it is non-finite too.
 *
 *   x_bf16  device, [tokens][ld] bf16, ld >= n.
 *   codes   device, [tokens][ldc] int8, ldc >= n.
 *   scale   device, [tokens] float.
 *   sum     device, [tokens] int32, or NULL: sum_j q_j.
 *
 * 1 <= n <= 131071; any alignment and stride (16-byte aligned rows are the
 * fast case).  tokens < 0 or >= 2^31, n out of range, ld < n, ldc < n or a
 * null pointer -> SIGNROT_EINVAL.  No allocation.  Asynchronous.
 */
int signrot_quant_int8(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld, int8_t* codes, int64_t ldc,
                       float* scale, int32_t* sum, void* stream);

/*
 * The 8-bit product (W8A8):
 *   out[t][k] = scale[t] * w_scale[k] * sum_j q[t][j] * w[k][j] + bias[k].
 * The sum is a whole number in int32 (exact, whatever the order); it is
 * widened to binary32, scaled, and rounded once to the output type.
 *
 *   codes    device, [tokens][ldc] int8, ldc >= n.
 *   scale    device, [tokens] float.
 *   w        device, [rows][ldw] int8, ldw >= n: row k is output channel k.
 *   w_scale  device, [rows] float.
 *   bias     device, [rows] float, or NULL.
 *   out      device, [tokens][ldo] of out_type, ldo >= rows.
 *   workspace, workspace_bytes
 *            device scratch of at least signrot_int8_linear_workspace bytes
 *            (for the same operands), 16-byte aligned; NULL when that is 0.
 *            Its contents are unspecified before and after the call; it must
 *            not be used by anything else until the call's work has ended.
 *
 * 1 <= n <= 131071 (an int32 sum cannot overflow); any alignment and stride
 * of codes, w and out.  Rows that are not 16-byte aligned with n a multiple of
 * 16 (32 of packed INT4 codes) cost more; large ones are laid out anew in the
 * workspace first.  Rows of codes and w are read in words: bytes before and after a row
 * that lie in one aligned 16-byte chunk with a byte of it may be read too (so no
 * page but the row's own); their values do not matter.  tokens == 0 or rows == 0 is a no-op.  Negative
 * sizes, tokens or rows >= 2^30, a leading dimension below its row, an unknown
 * out_type, a workspace that is too small or a null pointer ->
 * SIGNROT_EINVAL.  No allocation.  Asynchronous.
 */
int signrot_int8_linear(const int8_t* codes, int64_t ldc, const float* scale, int64_t tokens, int64_t n,
                        const int8_t* w, int64_t ldw, const float* w_scale, const float* bias, int64_t rows,
                        void* out, int64_t ldo, int out_type, void* workspace, int64_t workspace_bytes,
                        void* stream);

/*
 * The consumer of the rotated INT4 activations with 8-bit weights (W8A4):
 *   out[t][k] = scale[t] * w_scale[k]
 *               * (sum_j q[t][j] * w[k][j] - zero[t] * w_sum[k]) + bias[k],
 * which is sum_j yhat[t][j] * (w_scale[k] w[k][j]) with yhat = scale * (q -
 * zero); the product runs on the unsigned integer codes.
 *
 *   codes    device, [tokens][n/2] uint8, as signrot_rotate_quant_int4 writes
 *            them (channel 2m in the low nibble of byte m).
 *   scale, zero  device, [tokens] float each.
 *   w_sum    device, [rows] int32: sum_j w[k][j] (signrot_quant_int8's sum).
 *   workspace  as above, signrot_int4_w8_linear_workspace bytes.
 *   the other arguments as for signrot_int8_linear.
 *
 * n even, 2 <= n <= 131070; the other errors as for signrot_int8_linear.  No
 * allocation.  Asynchronous.
 */
int signrot_int4_w8_linear(const uint8_t* codes, const float* scale, const float* zero, int64_t tokens, int64_t n,
                           const int8_t* w, int64_t ldw, const float* w_scale, const int32_t* w_sum,
                           const float* bias, int64_t rows, void* out, int64_t ldo, int out_type, void* workspace,
                           int64_t workspace_bytes, void* stream);

/* Scratch bytes the two products need for these operands (0: none, the pointer
 * may be NULL), or -1 when the sizes are invalid.  They depend on the sizes and
 * on the alignment of the pointers and strides.  Host-only. */
int64_t signrot_int8_linear_workspace(const int8_t* codes, int64_t ldc, int64_t tokens, int64_t n, const int8_t* w,
                                      int64_t ldw, int64_t rows);
int64_t signrot_int4_w8_linear_workspace(const uint8_t* codes, int64_t tokens, int64_t n, const int8_t* w, int64_t ldw,
                                         int64_t rows);

/* Which kernel the two products would launch for these operands (a static
 * string), or NULL when the sizes are invalid.  Host-only. */
const char* signrot_int8_linear_kernel_name(const int8_t* codes, int64_t ldc, int64_t tokens, int64_t n,
                                            const int8_t* w, int64_t ldw, int64_t rows);
const char* signrot_int4_w8_linear_kernel_name(const uint8_t* codes, int64_t tokens, int64_t n, const int8_t* w,
                                               int64_t ldw, int64_t rows);

/* Norms of signrot_residual_norm, of a row x with weight w and bias b:
 *   RMS    x / sqrt(mean_j x_j^2 + eps) * w + b
 *   LAYER  (x - mean x) / sqrt(mean_j (x_j - mean x)^2 + eps) * w + b
 *   NONE   x (weight and bias are not applied) */
typedef enum { SIGNROT_NORM_NONE = 0, SIGNROT_NORM_RMS = 1, SIGNROT_NORM_LAYER = 2 } signrot_norm;

/*
 * The norm after a block, the block's gate and residual scale, the residual
 * sum and the norm before the next block, in one pass over the rows:
 *   h'[t] = beta * h[t] + alpha * gate[r] * Norm_post(y[t])
 *   u[t]  = Norm_pre(h'[t]) * (1 + mod_scale[r]) + mod_shift[r]
 * with r the modulation row of token t: 0 where the stride (ldg, ldm) is 0,
 * else mod_index[t] (clamped into [0, mod_rows)), or t when mod_index is
 * NULL.  u leaves as bf16, or as the symmetric per-token INT8 codes and
 * scales of signrot_quant_int8 (of the binary32 u), or both.  Norm_pre reads
 * h' before it is rounded to the stream's type.  All arithmetic is binary32;
 * each output is rounded once.  A row that holds an infinity or NaN gives
 * unspecified outputs in that row only; its code scale is non-finite.
 * So does a row whose h' or, for LAYER, whose sum passes binary32's range (its
 * squares may).
 *
 *   tokens, n     rows, and channels of a row: 0 <= tokens < 2^31,
 *                 1 <= n <= 131071.
 *   h, ldh        device, [tokens][ldh] of h_type: the residual stream.
 *   y, ldy        device, [tokens][ldy] bf16: the block's output, or NULL: no
 *                 branch, h' = beta * h.
 *   h_out, ldho   device, [tokens][ldho] of h_type, or NULL: h' is not stored.
 *                 May be h itself (same pointer and stride); may not overlap
 *                 h in another way.
 *   u, ldu        device, [tokens][ldu] bf16, or NULL.
 *   codes, ldc, code_scale   device, [tokens][ldc] int8 and [tokens] float,
 *                 or both NULL.
 *   post_weight, post_bias, pre_weight, pre_bias   device, [n] of param_type,
 *                 each may be NULL (weight 1, bias 0).
 *   gate, ldg     device, [n] (ldg == 0) or [mod_rows][ldg], or NULL (1).
 *   mod_scale, mod_shift, ldm   device, the same two layouts, each may be NULL.
 *   mod_index, mod_rows  device, [tokens] int32 or NULL; the number of rows of
 *                 gate, mod_scale and mod_shift where their stride is not 0
 *                 (at least tokens when mod_index is NULL).
 *
 * Any alignment and stride (16-byte aligned rows are the fast case).  A null
 * h, a leading dimension below n (0 for a shared modulation row), no output
 * at all, codes without code_scale or the reverse, an unknown norm or type,
 * a non-finite or negative eps or non-finite alpha or beta, sizes out of
 * range -> SIGNROT_EINVAL.  tokens == 0 is a no-op.  No allocation.
 * Asynchronous.  The order of a row's sums is fixed for a number of tokens, and
 * may be another one for another number.
 */
typedef struct {
  int64_t tokens, n;
  const void* h;
  int64_t ldh;
  const void* y;
  int64_t ldy;
  void* h_out;
  int64_t ldho;
  void* u;
  int64_t ldu;
  int8_t* codes;
  int64_t ldc;
  float* code_scale;
  const void* post_weight;
  const void* post_bias;
  const void* gate;
  int64_t ldg;
  const void* pre_weight;
  const void* pre_bias;
  const void* mod_scale;
  const void* mod_shift;
  int64_t ldm;
  const int32_t* mod_index;
  int64_t mod_rows;
  float alpha, beta, eps_post, eps_pre;
  int32_t post_norm, pre_norm;  /* signrot_norm */
  int32_t h_type, param_type;   /* signrot_type */
} signrot_residual_norm_args;

int signrot_residual_norm(const signrot_residual_norm_args* args, void* stream);

/*
 * Microscaled 4-bit floating point (MXFP4, the OCP microscaling formats' E2M1
 * elements with E8M0 scales).  A row is cut into blocks of 32 channels.  A
 * block's scale byte b stands for 2^(b - 127) (255: NaN); a code stands for
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6 (its low three bits) with the sign of its high
 * bit, times the scale.  A row of n channels has nb = ceil(n / 32) blocks: 16
 * bytes of codes a block (channel 2m in the low nibble of byte m) and one scale
 * byte.  Channels beyond n in the last block have code 0.
 *
 * Choice of a block's scale 2^e, a = max |x| of the block:
 *   FLOOR   e = floor(log2 a) - 2: a / 2^e in [4, 8), values over 6 saturate.
 *   NOCLIP  the same, and one more where a > 6 2^e: the least e of which no
 *           value saturates.
 * e is kept within [-127, 127]; an all-zero block has e = -127.
 */
typedef enum { SIGNROT_MX_FLOOR = 0, SIGNROT_MX_NOCLIP = 1 } signrot_mx_rule;

/*
 * MXFP4 quantizer: code = x / 2^e rounded to the nearest level, to the even
 * code at a tie, the sign kept (also of zero).  Exact: the same codes and
 * scales as the definition in real numbers.  A block that holds an infinity or
 * NaN gets scale byte 255 and codes 0.
 *
 *   x       device, [tokens][ld] of x_type, ld >= n.
 *   codes   device, [tokens][ldc] uint8, ldc >= 16 nb.
 *   scale   device, [tokens][lds] uint8, lds >= nb.
 *
 * 0 <= tokens < 2^31, 1 <= n <= 131072; any alignment and stride (16-byte
 * aligned rows with n a multiple of 8 are the fast case).  tokens == 0 is a
 * no-op.  Sizes out of range, a leading dimension below its row, an unknown
 * type or rule, a null pointer -> SIGNROT_EINVAL.  No allocation.  Asynchronous.
 */
int signrot_quant_mxfp4(const void* x, int x_type, int64_t tokens, int64_t n, int64_t ld, int rule, uint8_t* codes,
                        int64_t ldc, uint8_t* scale, int64_t lds, void* stream);

/*
 * The values MXFP4 codes stand for: y [tokens][ldy] of y_type, ldy >= n, the
 * first n channels of every row.  Exact in either type (2^e level passes
 * binary32's range, and becomes an infinity, for scale bytes above 252 only).
 * The other arguments and errors as for signrot_quant_mxfp4.
 */
int signrot_dequant_mxfp4(const uint8_t* codes, int64_t ldc, const uint8_t* scale, int64_t lds, int64_t tokens,
                          int64_t n, void* y, int y_type, int64_t ldy, void* stream);

/*
 * The product of MXFP4 operands:
 *   out[t][k] = sum_j x[t][j] * w[k][j] + bias[k],
 * x and w the values the codes stand for, both in blocks along j.  The matrix
 * cores multiply the codes and apply both scales; sums are binary32, and the
 * result is rounded once to the output type.  The order of the sums is fixed
 * for given sizes and alignments.  A NaN scale makes the results of its row (of
 * tokens or weights) NaN.
 *
 *   codes, scale      device, [tokens][ldc] and [tokens][lds] uint8.
 *   w, w_scale        device, [rows][ldw] and [rows][ldws] uint8: row k is
 *                     output channel k.
 *   bias              device, [rows] float, or NULL.
 *   out               device, [tokens][ldo] of out_type, ldo >= rows.
 *   workspace, workspace_bytes
 *                     device scratch of at least signrot_mxfp4_linear_workspace
 *                     bytes (for the same operands), 16-byte aligned; NULL when
 *                     that is 0.  Its contents are unspecified before and after
 *                     the call; it must not be used by anything else until the
 *                     call's work has ended.
 *
 * n a multiple of 32 (whole blocks), 32 <= n <= 131072; tokens and rows below
 * 2^30; any alignment and stride (code rows that do not start on 16-byte
 * boundaries are laid out anew in the workspace, and so are rows of fewer than
 * four scales that do not start on 4-byte ones).  Scales may be read in aligned
 * words of four: bytes beside a row's in the words that hold its ends may be
 * read too; their values do not matter.  tokens == 0 or
 * rows == 0 is a no-op.  Negative sizes, a leading dimension below its row, an
 * unknown out_type, a workspace that is too small or a null pointer ->
 * SIGNROT_EINVAL.  No allocation.  Asynchronous.
 */
int signrot_mxfp4_linear(const uint8_t* codes, int64_t ldc, const uint8_t* scale, int64_t lds, int64_t tokens,
                         int64_t n, const uint8_t* w, int64_t ldw, const uint8_t* w_scale, int64_t ldws,
                         const float* bias, int64_t rows, void* out, int64_t ldo, int out_type, void* workspace,
                         int64_t workspace_bytes, void* stream);

/* Scratch bytes of the product for these operands (0: none, the pointer may be
 * NULL), or -1 when the sizes are invalid, and the kernel it would launch (a
 * static string; NULL when the sizes are invalid).  They depend on the sizes
 * and on the alignment of the pointers and strides.  Host-only. */
int64_t signrot_mxfp4_linear_workspace(const uint8_t* codes, int64_t ldc, const uint8_t* scale, int64_t lds,
                                       int64_t tokens, int64_t n, const uint8_t* w, int64_t ldw,
                                       const uint8_t* w_scale, int64_t ldws, int64_t rows);
const char* signrot_mxfp4_linear_kernel_name(const uint8_t* codes, int64_t ldc, const uint8_t* scale, int64_t lds,
                                             int64_t tokens, int64_t n, const uint8_t* w, int64_t ldw,
                                             const uint8_t* w_scale, int64_t ldws, int64_t rows);

/*
 * The rotation and sign flip of signrot_rotate_quant_int4_outlier (d = sigma *
 * row c of H) with MXFP4 output: the codes and scales that signrot_quant_mxfp4
 * gives of y = (x.H / sqrt(n)) * d in binary32 (the y_out of that call).
 *
 *   x_bf16, tokens, n, ld, c, sigma   as for signrot_rotate_quant_int4_outlier.
 *   rule, codes, ldc, scale, lds      as for signrot_quant_mxfp4; codes 16-byte
 *                     aligned and ldc a multiple of 16.
 *   workspace, workspace_bytes        device scratch of at least
 *                     signrot_rotate_quant_mxfp4_workspace(tokens, n) bytes,
 *                     16-byte aligned (as for the product): 0 at the widths of
 *                     the fused kernels (signrot_kernel_name "rq_mfma..."), the
 *                     rotated rows at the others.
 *
 * Any supported n; errors as for the two calls.  Asynchronous.  No allocation
 * beyond signrot_rotate_quant_int4_outlier's own.
 */
int signrot_rotate_quant_mxfp4(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld, int64_t c, int sigma,
                               int rule, uint8_t* codes, int64_t ldc, uint8_t* scale, int64_t lds, void* workspace,
                               int64_t workspace_bytes, void* stream);
int64_t signrot_rotate_quant_mxfp4_workspace(int64_t tokens, int64_t n);

/*
 * The same on x = bf16(SiLU(gate) * up), the producer fused in, as
 * signrot_swiglu_rotate_quant_int4 (gate and up with one stride ld; the widths
 * of the fused kernels only).
 */
int signrot_swiglu_rotate_quant_mxfp4(const void* gate_bf16, const void* up_bf16, int64_t tokens, int64_t n, int64_t ld,
                                      int64_t c, int sigma, int rule, uint8_t* codes, int64_t ldc, uint8_t* scale,
                                      int64_t lds, void* stream);

/*
 * The norm of each head of the queries and keys and their rotation by the
 * token's position, in one pass.  Per token t and head, v = Norm(x) over the
 * head's channels (signrot_norm, with weight and bias; the same norm for
 * queries and keys), then for each pair p < rotary / 2 of its first `rotary`
 * channels, (a, b) = channels (p, p + rotary / 2), or (2p, 2p + 1) when
 * interleaved:
 *   a' = a cos[r][p] - b sin[r][p],   b' = b cos[r][p] + a sin[r][p],
 * r = positions[t] (clamped into [0, places)), or t when positions is NULL.
 * Channels from `rotary` on are normed only; with NORM_NONE their values come
 * through as they are, signs of zeros too.  All arithmetic is binary32; each
 * result is rounded once.  A head that holds an infinity or NaN gives
 * unspecified results in that head only, with NORM_NONE in its pair only.  Sums
 * and squares may pass binary32's range, or fall below it with an eps that does
 * not hide them: such a head is normed on scaled values.  (With eps 0 a head of
 * zeros, or of equal values with NORM_LAYER, gives NaN.)
 *
 *   tokens, head, rotary   0 <= tokens < 2^31; channels of a head, even, in
 *                 [8, 512]; rotated channels, even, in [0, head].
 *   q, ldq, hsq   device, in_type: channel j of head h of token t at
 *                 q[t * ldq + h * hsq + j]; strides in elements, any sign-free
 *                 order of tokens and heads (each >= 0).
 *   q_out, ldqo, hsqo   device, out_type, the same; may be q itself (same
 *                 pointer, strides and type); may not overlap q or k otherwise,
 *                 and its rows may not overlap each other.
 *   k, k_out, ... the same for the keys; NULL with k_heads 0: no keys.
 *   q_heads, k_heads   heads of a token, in [1, 65536] and [0, 65536].
 *   cos, sin, ldt, places   device, [places][ldt] float, ldt >= rotary / 2;
 *                 may be NULL when rotary is 0.
 *   positions     device, [tokens] int32 (positions_64 0) or int64 (1), or NULL
 *                 (places >= tokens then).
 *   q_weight, k_weight, q_bias, k_bias   device, [head] of param_type, each may
 *                 be NULL (weight 1, bias 0); not applied with NORM_NONE.
 *
 * Any alignment (16-byte aligned heads of a multiple of 8 channels are the fast
 * case).  tokens == 0 is a no-op.  Sizes out of range, an unknown norm or type,
 * a negative or non-finite eps, a null pointer -> SIGNROT_EINVAL.  No
 * allocation.  Asynchronous.
 */
typedef struct {
  int64_t tokens, head, rotary;
  const void* q;
  int64_t ldq, hsq;
  void* q_out;
  int64_t ldqo, hsqo;
  const void* k;
  int64_t ldk, hsk;
  void* k_out;
  int64_t ldko, hsko;
  const float* cos;
  const float* sin;
  int64_t ldt, places;
  const void* positions;
  const void* q_weight;
  const void* k_weight;
  const void* q_bias;
  const void* k_bias;
  int32_t q_heads, k_heads;
  float eps;
  int32_t norm;                             /* signrot_norm */
  int32_t interleaved, positions_64;        /* 0 or 1 */
  int32_t in_type, out_type, param_type;    /* signrot_type */
} signrot_qk_norm_rope_args;

int signrot_qk_norm_rope(const signrot_qk_norm_rope_args* args, void* stream);

/*
 * Measurement aid, not part of the method: a kernel that moves the bytes the
 * online path moves per token -- reads the bf16 row (2n bytes), writes n/2
 * bytes to out [tokens][n/2] and one float each to s0 [tokens] and
 * s1 [tokens] -- with no arithmetic (each 16-byte input chunk becomes the XOR
 * of its four words).  Its time is the memory system's ceiling for that
 * read/write mix at the shape.  n a multiple of 8 in [8, 32768], ld >= n and
 * a multiple of 8, tokens * n / 8 < 2^32, x 16-byte and out 4-byte aligned.
 * Asynchronous.
 */
int signrot_stream_ceiling(const void* x_bf16, int64_t tokens, int64_t n, int64_t ld, uint8_t* out, float* s0,
                           float* s1, void* stream);

/* Static text for a status code. */
const char* signrot_strerror(int status);

/* Detail of the last failure on the calling thread ("" if none). */
const char* signrot_last_error(void);

/*
 * The library's own H28, row-major, entries +1/-1, written to host memory
 * out[784].  Lets a test compare it with an independently built table.
 */
int signrot_debug_h28(int8_t* out);

/*
 * The library's outer factor H_m (m = 28 or any Paley order of the rule above,
 * m <= 512), row-major, entries +1/-1, written to host memory out[m * m].
 * Host-only (no GPU needed).  SIGNROT_EINVAL when m has no construction.
 */
int signrot_debug_outer(int m, int8_t* out);

/*
 * The outer factor the rotate kernel uses when it reads n = m * 2^k as
 * (m 2^fold) * 2^(k - fold): H_m (x) Syl_{2^fold}, entry
 * (a 2^fold + u, a' 2^fold + v) = H_m[a][a'] (-1)^popcount(u & v), with
 * m = 1 (the Sylvester matrix alone), 28, or a Paley order.  Written
 * row-major to host memory out[(m 2^fold)^2].  Host-only.  SIGNROT_EINVAL
 * when m 2^fold > 512 or m has no construction.
 */
int signrot_debug_outer_folded(int m, int fold, int8_t* out);

/* How many Sylvester index bits the rotate kernel for n moves into its outer
 * factor (0: none), or -1 when n is unsupported.  Host-only. */
int signrot_outer_fold(int64_t n);

/* Which kernel variant signrot_rotate_quant_int4 would launch for n (a
 * static string naming it), or NULL when n is unsupported:
 *   "rq_mfma32_w8"   n = 4096, 8192, 16384 (Sylvester);
 *   "rq_mfma28_w7"   n = 28 * 2^k, k = 7, 8, 9;
 *   "rq_mfma28x2_w7" n = 28672 (two halves of the 14336 transform);
 *   "rq_outer_mfma"  n = m * 2^k with 16 <= 2^k <= 256 and ceil(m / 32)
 *                    at most 12, 12, 8, 6, 4 for 2^k = 16, 32, 64, 128, 256
 *                    (11008, 13824, 18944, 8960, 27648, 5120, 5504, 896,
 *                    1792 among them), and widths that reach such a shape
 *                    with Sylvester bits moved into the outer factor (24576,
 *                    20480, 12288, 10240, 6144, 64 .. 2048, 32768; most
 *                    2^k = 256 widths, e.g. 5120 and 17408, run as
 *                    (2 m) * 128);
 *   "rq_generic"     every other supported n.
 * Host-only (no GPU needed). */
const char* signrot_kernel_name(int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* SIGNROT_H */
