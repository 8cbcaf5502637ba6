/*
 * gemm_s8.h -- 8-bit integer operands of the GB300 (sm_103a) GEMM library: rows
 * quantised to int8 with one scale each, and products of two such operands.
 *
 * An operand is a matrix of type GEMM_S8 (two's complement, all of -128 .. 127)
 * and an array of fp32 scales on the device: one per row of A (token), one per
 * column of B (output channel).  x-hat = code * scale.
 *
 * Conventions (status codes, streams, ownership, alignment checks) are those of
 * gemm.h.  Host-side checks are made before anything is enqueued; no call
 * allocates device memory or needs a workspace.
 */
#ifndef QGEMM_GEMM_S8_H_
#define QGEMM_GEMM_S8_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantise X (row-major, f32 / f16 / bf16, any ld >= cols, num matrices) row by
 * row: with amax the row's largest magnitude and every step rounded to fp32,
 *   S[r] = max(amax / 127, 2^-126),   Q[r][c] = RN(X[r][c] * (127 / amax)),
 * RN to nearest, ties to even (for amax / 127 < 2^-126 the factor is 2^126).  A row with a NaN
 * or an infinity gets a NaN scale and zero codes, so it shows in every product
 * it takes part in.  Q: row-major, GEMM_S8, any ld >= cols (gemm_run_s8 wants a
 * multiple of 16), as many matrices as X; it must not overlap X.  S: num * rows floats, matrix after
 * matrix.  Weights [N, K] quantised like this are operand B: one scale per
 * output channel.
 */
int gemm_s8_quantize(gemm_handle_t h, const void* X, const gemm_layout_t* Xdesc, void* Q, const gemm_layout_t* Qdesc,
                     float* S, gemm_stream_t stream);

/*
 * D = act(alpha * SA[i] * SB[j] * (sum over k of A[i][k] * B[k][j]) + beta * C + bias).
 *   A : M x K, row-major, GEMM_S8, SA its M scales (NULL: 1);
 *   B : K x N, col-major, GEMM_S8 (rows of K codes, one per column), SB its N
 *       scales (NULL: 1);
 *   C, D as in gemm_run (f32 / f16 / bf16).
 * A's and B's base addresses are 16-byte aligned and their ld a multiple of 16;
 * K need not be.  The sum is exact, as in 32-bit integers (K at most 131071, above it
 * GEMM_ERR_UNSUPPORTED); it is converted to fp32, multiplied by alpha * SA[i] and
 * by SB[j], and finished as in gemm_run: fp32 steps, one rounding to D's type.
 * Of op, epilogue / bias / bias_type apply; GELU is x Phi(x) as in gemm_run_mx: for an
 * f32 D in gemm.h's form, off by up to 1.5 * 2^-22 |x| (at x = -5 some parts in a hundred
 * of the result, which is small there), for a 16-bit D within 2e-5, relative; splitk
 * forces that many K slices (1, 2, 4 or 8, as far as K has 128-wide steps for
 * them; 0 chooses) where a kernel that slices K serves the call; dispatch is
 * accepted and the built-in choice used.  U / V groups, streamk = 1, zero points,
 * batches and an int8 D are GEMM_ERR_UNSUPPORTED.  Results do not depend on the
 * run, nor on the kernel that was chosen.
 */
int gemm_run_s8(gemm_handle_t h, const gemm_op_t* op, float alpha, const void* A, const gemm_layout_t* Adesc,
                const float* SA, const void* B, const gemm_layout_t* Bdesc, const float* SB, float beta, const void* C,
                const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc, gemm_stream_t stream);

/*
 * The grouped form: rows of A (and of C, D) sorted by expert as in
 * gemm_run_grouped, B with num = num_experts matrices, SB num_experts * N scales,
 * expert after expert.  Rows that no expert holds keep what D had.
 */
int gemm_run_s8_grouped(gemm_handle_t h, const gemm_op_t* op, float alpha, const void* A, const gemm_layout_t* Adesc,
                        const float* SA, const void* B, const gemm_layout_t* Bdesc, const float* SB, float beta,
                        const void* C, const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc,
                        const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMM_GEMM_S8_H_ */
