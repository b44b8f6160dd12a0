/*
 * qw_mx.h -- the part of libqw's C ABI for the feed-forward half of a layer whose
 * weights are held in microscaled 4-bit floating point: codes, products, RMS norm
 * with the residual's addition and quantized output, the gated feed-forward block,
 * and the gradients.  Conventions (device pointers, streams, statuses, limits, no
 * allocation, nothing enqueued by a call that returns a validation error) are
 * those of qw.h.
 *
 * Microscaled 4-bit floating point (OCP Microscaling Formats 1.0, "MXFP4"):
 *
 *   code      4 bits per value: e2m1, bit 3 the sign, the others 0, 0.5, 1, 1.5,
 *             2, 3, 4, 6.  Two to a byte, the value of even index in the low half.
 *   blocks    QW_MX_BLOCK = 32 consecutive values of a row (the reduction axis k).
 *   scale     one byte s per block, it stands for 2^(s - 127): the exponent of the
 *             block's largest magnitude less 2, 2^(floor(log2 max|w|) - 2), at least
 *             2^-127; 1 (s = 127) where all values are zero.
 *   value     code = e2m1(w / scale), rounded to nearest, ties to the even code; a
 *             magnitude above 6 scales (less than 8 by construction) is 6.  The sign
 *             of zeros is kept.  The value it stands for is code * scale.
 *   NaN       a block with a NaN or an infinity has s = 255 and codes 0: all its
 *             values, and so every sum that it enters, are NaN.
 *   layout    rows of kp = qw_mx_pitch(k) values, k rounded up to a multiple of 512:
 *             codes [n][kp / 2] and scales [n][kp / 32] bytes.  Behind k the codes are
 *             0 and the scales of whole blocks 127.  A row of codes starts a 256-byte
 *             and a row of scales a 16-byte unit, so no k needs a kernel of its own.
 *   `codes` and `scales` pointers are 16-byte aligned (QW_EARG otherwise); all
 *   others may have the alignment of their type.
 *   Types are QW_F32 or QW_BF16, QW_EARG otherwise; a result is rounded once, to
 *   nearest even, from fp32.
 */
#ifndef QW_MX_H
#define QW_MX_H

#include "qw.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QW_MX_BLOCK 32

/* Values in a row of codes (-1 if k is invalid). */
int64_t qw_mx_pitch(int64_t k);

/*
 * Quantize w [n][k] (read):
 *   transpose 0: codes [n][qw_mx_pitch(k) / 2], scales [n][qw_mx_pitch(k) / 32]
 *   transpose 1: the codes of w's columns, as rows: codes [k][qw_mx_pitch(n) / 2],
 *                scales [k][qw_mx_pitch(n) / 32] (written)
 * (QW_EARG for another transpose).  One pass over w.  The second form makes the
 * operands of a weight gradient, whose sums run over the rows (tokens), and of an
 * input gradient, whose sums run over the weight's rows.  Blocks lie along the sum,
 * so a transposed weight has codes of its own.
 */
int qw_mx_quantize(int transpose, int64_t n, int64_t k, int type, const void* w,
                   uint8_t* codes, uint8_t* scales, void* stream);

/* Values of codes: out fp32 [n][k], exact (written). */
int qw_mx_unpack(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales,
                 float* out, void* stream);

/*
 * Product of two quantized matrices on the 4-bit matrix cores:
 *   y[r][i] = sum_j x[r][j] w[i][j]
 *   codes, scales       the weight, n x k      (read)
 *   x_codes, x_scales   m rows of k values     (read)
 *   y                   [m][n]                 (written), m >= 0
 * k <= QW_BLOCK_MAX_K and n <= 2^27 (QW_ESHAPE), m <= 2^27 (QW_EM), also for k = 0, where
 * y is zeros.  Sums are held in fp32: error <= (4 + k/64) *
 * 2^-23 * sum_j |x[r][j] w[i][j]| and y's rounding, where no block's two scales
 * have a product below 2^-149 (a smaller one counts as zero).  Deterministic: the
 * same call gives the same bits, and rows of x do not influence each other.
 */
int qw_mx_gemm(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
               const uint8_t* x_codes, const uint8_t* x_scales, int y_type, void* y,
               void* stream);

/*
 * The same with float activations, quantized on the way: the codes are those of
 * qw_mx_quantize.
 *   x [m][k] (read),  y [m][n] (written),
 *   work: qw_mx_matmul_work_bytes(m, k) bytes, 16-byte aligned (QW_EWORK); a buffer
 *   for the largest call is enough for all smaller ones.
 */
int64_t qw_mx_matmul_work_bytes(int64_t m, int64_t k);
int qw_mx_matmul(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
                 int x_type, const void* x, int y_type, void* y, void* work,
                 int64_t work_bytes, void* stream);

/*
 * RMS norm of the sum of x and a residual:
 *   s = x + residual, rounded to `type` (x itself without a residual)
 *   y = s / sqrt(mean(s^2) + eps) * weight, in fp32, rounded once
 *   x [rows][d], residual [rows][d] or NULL  (read)
 *   sum [rows][d]: s (written; NULL: not; with a residual it is what the next layer's
 *        residual and the gradient start from).  It may be x or residual itself.
 *   weight [d] of weight_type, or NULL (all 1)   (read)
 *   y [rows][d] of y_type (written)
 * eps is finite and >= 0 (QW_EARG).  x, residual and sum have `type`.  Squares
 * and their sum are held in 64 bits; y is rounded to fp32 and then to its type, for
 * rows with sqrt(mean(s^2) + eps) from 2^-126 to 2^100.  (Beyond 2^100 the factor of a
 * row has fewer bits, y is off by 2^-21 of itself at most; below 2^-128, which takes
 * subnormal values and such an eps, the factor and y are infinite.)
 */
int qw_rms_norm(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                void* sum, int weight_type, const void* weight, float eps, int y_type, void* y,
                void* stream);

/* The same with y (in fp32) quantized on the way: as e4m3 codes with 1 x 128 blocks,
 * as qw_block_quantize writes them: codes [rows][qw_block_pitch(d)] (16-byte aligned),
 * scales [rows][qw_block_pitch(d) / 128]. */
int qw_rms_norm_block(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                      void* sum, int weight_type, const void* weight, float eps,
                      uint8_t* codes, float* scales, void* stream);

/* The same as 4-bit codes, as qw_mx_quantize writes them. */
int qw_rms_norm_mx(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                   void* sum, int weight_type, const void* weight, float eps, uint8_t* codes,
                   uint8_t* scales, void* stream);

/*
 * Gradients of qw_rms_norm (and, as if y were not rounded, of the other two) for the
 * output gradient dy: with r = 1 / sqrt(mean(s^2) + eps),
 *   ds = r (dy weight - s r^2 mean(dy weight s)) + dsum    (of x and of the residual)
 *   dweight[j] = sum over the rows of dy s r
 *   dy, s [rows][d] (read); dsum [rows][d]: the gradient that reaches s past the
 *   norm, or NULL (none);  all of `type`
 *   ds [rows][d] of `type` (written; NULL: not).  It may be dy or dsum itself.
 *   dweight fp32 [d] (written; NULL: not)
 *   work: qw_rms_norm_backward_work_bytes(rows, d) bytes, 16-byte aligned (QW_EWORK),
 *   needed for dweight only; a buffer for the largest call is enough for all smaller.
 * A row's sums are held in fp32, of s by a power of two where its squares would leave
 * it, so that rows of any magnitude with sqrt(mean(s^2) + eps) from 2^-126 on have their
 * gradients (below that r is infinite).  The rows' sum has a fixed order: the same call
 * gives the same bits.
 */
int64_t qw_rms_norm_backward_work_bytes(int64_t rows, int64_t d);
int qw_rms_norm_backward(int64_t rows, int64_t d, int type, const void* dy, const void* s,
                         int weight_type, const void* weight, float eps, const void* dsum,
                         void* ds, float* dweight, void* work, int64_t work_bytes,
                         void* stream);

/*
 * The gated half of a feed-forward block, both projections and the gating in one
 * product:
 *   gate = x G^T, up = x U^T,  h = silu(gate) * up = gate / (1 + exp(-gate)) * up
 *   codes, scales      2 f x k: the rows of G, then those of U   (read)
 *   x_codes, x_scales  m rows of k values                        (read)
 * as floats h [m][f] of h_type, or (from fp32) as 4-bit codes and scales of m rows of
 * f values.  gate and up have qw_mx_gemm's error.
 */
int qw_mx_gated(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
                const uint8_t* x_codes, const uint8_t* x_scales, int h_type, void* h,
                void* stream);
int qw_mx_gated_codes(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales,
                      int64_t m, const uint8_t* x_codes, const uint8_t* x_scales,
                      uint8_t* h_codes, uint8_t* h_scales, void* stream);

/*
 * Its gradients with regard to gate and up, which are computed again, not kept: with
 * t = 1 / (1 + exp(-gate)),
 *   dgate = dh up t (1 + gate (1 - t)),  dup = dh gate t
 *   dh [m][f] (read); dgate_up [m][2 f]: dgate | dup (written); h [m][f]: the gated
 *   values again, for the gradient of the next weight (written; NULL: not);
 *   all of `type`
 * The gradients of the block follow with qw_mx_quantize and qw_mx_gemm: of x with the
 * transposed weight, of the weight with transposed dgate_up and x.
 */
int qw_mx_gated_backward(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales,
                         int64_t m, const uint8_t* x_codes, const uint8_t* x_scales, int type,
                         const void* dh, void* dgate_up, void* h, void* stream);

/*
 * The whole block, the calls above in one:
 *   y = D Q(h),  h = silu(gate) * up of Q(x),  Q the quantizer
 *   gate_up 2 f x d (gate rows, then up rows), down d x f;  x, y [m][d]
 *   work: qw_mx_mlp_work_bytes(m, d, f) bytes, 16-byte aligned (QW_EWORK); it grows
 *   with every argument.
 * For few rows h is summed in another order than for many: where a value lies within
 * the sums' error of the border between two codes, its code may be either.
 */
int64_t qw_mx_mlp_work_bytes(int64_t m, int64_t d, int64_t f);
int qw_mx_mlp(int64_t d, int64_t f, const uint8_t* gate_up, const uint8_t* gate_up_scales,
              const uint8_t* down, const uint8_t* down_scales, int64_t m, int x_type,
              const void* x, int y_type, void* y, void* work, int64_t work_bytes,
              void* stream);

/*
 * Diagnostic: which kernel a call of these sizes would take, or a negative status;
 * `op`: 0 qw_mx_gemm, 1 qw_mx_gated, 2 qw_mx_gated_codes, 3 qw_mx_gated_backward (n = f):
 *     100 t + u = the kernel whose waves share k, with 16 t rows of x and u units of 512
 *     values of k a wave (105: run by the kernel of 6 units, with the last one empty);
 *     2 = tiles of 64 x 64 whose waves share every step of k;
 *     otherwise 1000 * weight rows + tokens of a tile
 *   4 qw_mx_matmul: 1 = the product quantizes x, 2 = a kernel before it does
 * Enqueues nothing.
 */
int qw_mx_debug_path(int op, int64_t m, int64_t n, int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* QW_MX_H */
