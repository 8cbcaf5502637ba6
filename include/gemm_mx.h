/*
 * gemm_mx.h -- 4-bit microscaled operators of the GB300 (sm_103a) GEMM library.
 *
 * An operand is a rows x cols matrix of E2M1 codes (sign, two exponent bits,
 * one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with one
 * scale per block of consecutive columns in a row:
 *
 *   GEMM_NVFP4  blocks of 16, E4M3 scales (s >= 0), and one fp32 scale g for
 *               the whole tensor: x = code * s * g;
 *   GEMM_MXFP4  blocks of 32, E8M0 scales (byte e stands for 2^(e - 127),
 *               255 for NaN): x = code * s.
 *
 * Codes: two per byte, column 2t in bits 3:0 and 2t+1 in bits 7:4 of byte t of
 * a row; type GEMM_E2M1, ld in codes, a multiple of 32 (16 bytes), the base
 * 16-byte aligned.  When cols is odd the last byte's high half is zero.
 *
 * Scales: bytes in 512-byte atoms of 128 rows x 4 blocks; the scale of row r
 * and block b is byte (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4 of atom
 * (r / 128) * ceil(blocks / 4) + b / 4.  Blocks past the last one, up to the
 * end of an atom, are zero; rows past the last one may hold anything.  The
 * base is 16-byte aligned.  A GEMM_E2M1 matrix with num > 1 (the experts'
 * weights) has its matrices' scales one after another, each
 * gemm_mx_scale_size(format, rows, cols, 0) bytes.  Rows sorted by expert
 * (expert_offsets_dev of gemm_run_grouped) start every expert on an atom row
 * of its own: expert e's row i has the scale row
 * 128 * sum over e' < e of ceil(m_e' / 128) + i.
 *
 * Conventions (status codes, streams, ownership, alignment checks) are those
 * of gemm.h.  Host-side checks are made before anything is enqueued; no call
 * allocates device memory or needs a workspace.
 */
#ifndef QGEMM_GEMM_MX_H_
#define QGEMM_GEMM_MX_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_MXFP4 = 1, GEMM_NVFP4 = 2 } gemm_mx_format_t;

/*
 * Bytes of the scales of a rows x cols operand.  num_experts == 0: one matrix.
 * num_experts > 0: rows sorted by that many experts, for any split of the
 * rows (rows / 128 + num_experts atom rows).
 */
int gemm_mx_scale_size(int32_t format, int64_t rows, int64_t cols, int32_t num_experts, size_t* bytes);

/*
 * Quantise X (row-major, f32 / f16 / bf16, any ld >= cols, num matrices) to
 * codes and scales.  With amax the block's largest magnitude and every step
 * rounded to fp32:
 *   GEMM_NVFP4  s = RN_E4M3(min(amax / (6 g), 448)),
 *               code = RN_E2M1(x / (s g)), 0 where s is 0;
 *   GEMM_MXFP4  s = 2^(floor(log2 amax) - 2), at least 2^-127,
 *               code = RN_E2M1(x / s);
 * RN to nearest, ties to even, magnitudes above 6 to 6.  A block with a NaN or
 * an infinity gets a NaN scale and zero codes, so it shows in every product it
 * takes part in.  tensor_scale is g: within [2^-64, 2^64], and 1 for MXFP4.
 * expert_offsets_dev (with num_experts > 0, else NULL and 0): X's rows are
 * sorted by expert; rows outside every expert are left out.
 */
int gemm_mx_quantize(gemm_handle_t h, int32_t format, float tensor_scale, const void* X, const gemm_layout_t* Xdesc,
                     void* Q, const gemm_layout_t* Qdesc, void* S, size_t S_size,
                     const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream);

/*
 * The values of a quantised matrix: D = RN_D(code * s * g) for a D of type
 * f32 / f16 / bf16; for a D of type GEMM_E4M3 the codes' own values (exact in
 * 8 bits), scales left out and tensor_scale not used.
 */
int gemm_mx_dequantize(gemm_handle_t h, int32_t format, float tensor_scale, const void* Q,
                       const gemm_layout_t* Qdesc, const void* S, size_t S_size, void* D,
                       const gemm_layout_t* Ddesc, const int32_t* expert_offsets_dev, int32_t num_experts,
                       gemm_stream_t stream);

/*
 * D = act(alpha * (A-hat @ B-hat) + beta * C + bias): both operands in 4 bits,
 * fp32 accumulation, one rounding to D's type (f32 / f16 / bf16).
 *   A : M x K, row-major, GEMM_E2M1, scales SA;
 *   B : K x N, col-major, GEMM_E2M1 (rows of K codes, one per column), scales
 *       SB over its N rows;
 *   C, D as in gemm_run.
 * Tensor scales go into alpha (alpha * g_a * g_b).  Of op, epilogue / bias /
 * bias_type apply; GELU is x Phi(x), for an f32 D in gemm.h's form
 * 0.5 x (1 + erf(x / sqrt 2)), for a 16-bit D within 2e-5 of it, relative, before
 * the rounding (negative x included, where gemm.h's form cancels); splitk forces
 * that many K slices (1, 2, 4 or 8, as far as there are 256-wide K-steps and the
 * partial tiles fit shared memory; 0 chooses), dispatch is accepted and the
 * built-in choice used (nothing is measured or cached); U / V groups, streamk = 1
 * and zero points have no meaning here and are GEMM_ERR_UNSUPPORTED, as are
 * batches and an int8 D.
 * Results do not depend on the run (slices are added in a fixed order).
 */
int gemm_run_mx(gemm_handle_t h, const gemm_op_t* op, int32_t format, float alpha, const void* A,
                const gemm_layout_t* Adesc, const void* SA, size_t SA_size, const void* B,
                const gemm_layout_t* Bdesc, const void* SB, size_t SB_size, float beta, const void* C,
                const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc, gemm_stream_t stream);

/*
 * The grouped form: rows of A (and of C, D) sorted by expert as in
 * gemm_run_grouped, B with num = num_experts matrices.  expert_alpha (device,
 * num_experts floats, or NULL) multiplies alpha expert by expert: the tensor
 * scales of the experts' weights.  Rows that no expert holds keep what D had, also
 * with K = 0 (D = act(beta C + bias)).
 */
int gemm_run_mx_grouped(gemm_handle_t h, const gemm_op_t* op, int32_t format, float alpha,
                        const float* expert_alpha, const void* A, const gemm_layout_t* Adesc, const void* SA,
                        size_t SA_size, const void* B, const gemm_layout_t* Bdesc, const void* SB, size_t SB_size,
                        float beta, const void* C, const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc,
                        const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream);

/*
 * What lies between two blocks of a network, in one pass over a row: the norm
 * after a block with its gate and residual scale, the residual sum, the norm
 * before the next block, and that block's 4-bit operand.  For every row:
 *   u  = F, or F * rsqrt(mean(F^2) + eps) * post_weight with a post_weight;
 *   u *= gate                      (a value per column, or per element);
 *   r' = RN(R + residual_scale * u)   in R's type, written to O;
 *   y  = r' * rsqrt(mean(r'^2) + eps) * pre_weight;
 *   Q, S = y quantised as gemm_mx_quantize does (its tensor_scale included).
 * F NULL: r' = R, and O may be NULL.  F, R, O: row-major, one of f32 / f16 /
 * bf16, any ld; O may be R or F.  pre_weight NULL: 1.  cols at most 32768.
 * Rows that no expert of expert_offsets holds get their r', but no Q and S.
 */
typedef struct {
    int32_t format;         /* gemm_mx_format_t                                 */
    float tensor_scale;     /* g of the quantised result                        */
    float eps;
    float residual_scale;
    const void* post_weight; /* cols values, or NULL: no norm of F              */
    const void* pre_weight;  /* cols values, or NULL                            */
    int32_t weight_type;     /* of both weights: GEMM_F32 / GEMM_F16 / GEMM_BF16 */
    int32_t gate_type;       /* GEMM_F32 / GEMM_F16 / GEMM_BF16                  */
    const void* gate;        /* or NULL                                          */
    int64_t gate_ld;         /* elements between rows of the gate; 0: one row for all */
    const int32_t* expert_offsets; /* device int32[num_experts + 1]: rows sorted by expert, whose
                                scales then start every expert on an atom row; or NULL */
    int32_t num_experts;     /* 0 without expert_offsets                         */
} gemm_mx_norm_t;

int gemm_mx_norm_quantize(gemm_handle_t h, const gemm_mx_norm_t* op, const void* F, const gemm_layout_t* Fdesc,
                          const void* R, const gemm_layout_t* Rdesc, void* O, const gemm_layout_t* Odesc, void* Q,
                          const gemm_layout_t* Qdesc, void* S, size_t S_size, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMM_GEMM_MX_H_ */
