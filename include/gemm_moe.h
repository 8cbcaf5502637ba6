/*
 * gemm_moe.h -- what lies around the grouped products of a mixture of experts:
 * choosing every token's experts, placing the tokens' rows by expert, and
 * bringing the experts' rows back to their tokens.
 *
 *   gemm_moe_route      logits -> experts, weights, and where each (token, slot)
 *                       has its row among the rows sorted by expert
 *   gemm_moe_dispatch   token rows -> rows sorted by expert (copied, or in int8)
 *   gemm_run_grouped / gemm_run_mx_grouped / gemm_run_s8_grouped
 *   gemm_moe_combine    rows sorted by expert -> weighted sum per token
 *
 * Conventions are those of gemm.h.
 */
#ifndef QGEMM_GEMM_MOE_H_
#define QGEMM_GEMM_MOE_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_ROUTE_SOFTMAX = 0, GEMM_ROUTE_SIGMOID = 1 } gemm_route_score_t;

typedef struct {
    int32_t score;       /* gemm_route_score_t: s = softmax(l) over the experts, or sigmoid(l)      */
    int32_t topk;        /* slots per token: 1 .. 32, at most the experts                            */
    int32_t groups;      /* 0 or 1: none; else 2 .. 32 groups of consecutive experts, equally large  */
    int32_t group_topk;  /* groups kept (1 .. groups)                                                */
    int32_t group_best;  /* a group's score is the sum of its 1 or 2 best choice scores              */
    int32_t renormalize; /* divide a token's weights by their sum                                    */
    float scale;         /* factor on the weights, finite                                            */
    const float* bias;   /* device, one per expert, or NULL                                          */
} gemm_route_t;

/*
 * Choose `topk` experts for each of L's rows (tokens x experts, row-major,
 * f32 / f16 / bf16; at most 1024 experts and 2^23 tokens).
 *   Choice scores  c = s + bias.  An expert whose logit or bias is -inf is never
 *     chosen.  With groups, only experts of the group_topk groups with the best
 *     group scores are.  Slots hold the experts with the largest c (without a
 *     bias: the largest logits), best first, ties to the lowest index (of groups
 *     too).  The choice is that of c in 64-bit arithmetic.
 *   Weights  s of the chosen expert (without the bias), with renormalize divided
 *     by the token's sum over its slots, times scale; fp32.
 *   A slot for which no expert is left: id -1, weight 0, row -1.  A token whose
 *     scores are undefined (a NaN logit, +inf under softmax, a NaN bias): ids and
 *     rows -1, weights NaN.
 * ids, weights (and rows): tokens x topk, contiguous.  rows[t * topk + j]: the row
 * of token t's slot j among the rows sorted by expert, then by token, then by
 * slot; expert_offsets: int32[experts + 1], as the grouped products take it (the
 * last one is the number of rows in use).  rows and expert_offsets may both be
 * NULL.  With them, more than 64 tokens need workspace partials of
 * GEMM_ROUTE_SCRATCH(experts) bytes (GEMM_ERR_WORKSPACE); barriers are not used.
 */
#define GEMM_ROUTE_SCRATCH(experts) ((size_t)304 * 16 * (((size_t)(experts) + 7) / 8))
int gemm_moe_route(gemm_handle_t h, const gemm_route_t* op, const void* L, const gemm_layout_t* Ldesc, int32_t* ids,
                   float* weights, int32_t* rows, int32_t* expert_offsets, const gemm_workspace_t* workspace,
                   gemm_stream_t stream);

/*
 * Place row t of X at rows rows[t * topk + j] of Y, j < topk.  Y has X's type
 * (f32, f16, bf16, GEMM_S8, GEMM_E4M3, GEMM_E5M2), or is GEMM_S8 with X f32 / f16 / bf16: its
 * rows are quantised as gemm_s8_quantize does and S[row] is the scale.  Rows that are
 * copied have no S: it is NULL (else GEMM_ERR_INVALID_ARG).  The scales of rows that are
 * int8 already are placed by a second call, as f32 rows of one column.  Entries
 * outside 0 .. Y's rows - 1 are left out, rows of Y that no entry names keep
 * what they held.  No row may be named twice.  X and Y: row-major, any ld; they
 * must not overlap.
 */
int gemm_moe_dispatch(gemm_handle_t h, const void* X, const gemm_layout_t* Xdesc, const int32_t* rows, int32_t topk,
                      void* Y, const gemm_layout_t* Ydesc, float* S, gemm_stream_t stream);

/*
 * D[t] = beta * C[t] + sum over j < topk of weights[t * topk + j] * Y[rows[t * topk + j]],
 * summed in fp32 in slot order, rounded once.  Y, C, D: row-major, one of
 * f32 / f16 / bf16, any ld.  A slot whose row lies outside Y counts as a row of
 * zeros (so a NaN weight shows).  C is not read when beta == 0 and may then be
 * NULL; D may be C, and must not overlap Y.
 */
int gemm_moe_combine(gemm_handle_t h, const void* Y, const gemm_layout_t* Ydesc, const int32_t* rows,
                     const float* weights, int32_t topk, float beta, const void* C, const gemm_layout_t* Cdesc, void* D,
                     const gemm_layout_t* Ddesc, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMM_GEMM_MOE_H_ */
