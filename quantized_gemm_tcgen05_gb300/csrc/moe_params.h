// Parameter blocks and launchers of the operators around the grouped products
// (include/gemm_moe.h) and of row quantisation (include/gemm_s8.h).
#pragma once
#include "kparams.h"

namespace qg {

constexpr int MOE_MAX_EXPERTS = 1024;
constexpr int MOE_MAX_TOPK = 32;
// Routing: blocks of the launch that counts, at most (the workspace holds their
// counts), and tokens that one block handles alone.
constexpr int ROUTE_MAX_BLOCKS = 304;
constexpr int ROUTE_ONE_BLOCK = 64;
// Threads of a block (a token a warp): with more experts a lane holds more keys.
QG_HD int route_threads(int experts) { return experts <= 256 ? 1024 : 512; }
constexpr int ROUTE_FEW = 16;    // tokens for which a single block is the quickest

// A block's counts are 16-bit numbers, and rows 32-bit ones.
constexpr int64_t ROUTE_MAX_TOKENS = 1 << 23;

enum RouteScore : int32_t { ROUTE_SOFTMAX = 0, ROUTE_SIGMOID = 1 };

struct RouteParams {
    const void* L;
    int64_t ld;
    int32_t type;
    int32_t tokens, experts, topk;
    int32_t groups, group_topk, group_best;  // groups 1: none
    int32_t score, renormalize;
    float scale;
    const float* bias;
    int32_t* ids;
    float* weights;
    int32_t* rows;      // with offsets, or null
    int32_t* offsets;
    uint16_t* counts;   // workspace: [blocks][pitch]
    int32_t pitch;      // experts, rounded up to 8
    int32_t blocks, tokens_per_block;
};

// Rows to rows: quantised (to int8 with a scale per row) or copied.
struct RowsParams {
    const void* X;
    const void* x_end;      // past the last value
    int64_t ldx, x_bstride; // elements
    void* Y;
    int64_t ldy, y_bstride; // elements
    float* S;
    int64_t rows;           // of X, per matrix
    int32_t cols, num;
    int32_t type;           // of X
    int32_t vec;            // X: base and rows 32-byte (2) or 16-byte (1) aligned, or neither (0)
    int32_t yvec;           // int8 Y: rows 16-byte aligned
    int32_t copy_unit;      // copy: bytes an access may have (16, 8, 4, 2 or 1)
    int32_t element;        // copy: bytes of an element
    const int32_t* map;     // rows[t * topk + j], or null: row t to row t
    int32_t topk;
    int64_t y_rows;
};

struct CombineParams {
    const void *Y, *C;
    const void *y_end, *c_end;
    void* D;
    int64_t ldy, ldc, ldd;
    int64_t tokens, y_rows;
    int32_t cols, type, topk, vec;  // vec: of Y, C and D
    float beta;
    const int32_t* map;
    const float* weights;
};

cudaError_t launch_route(const RouteParams& p, cudaStream_t st);
cudaError_t launch_row_quantize(const RowsParams& p, cudaStream_t st);
cudaError_t launch_row_copy(const RowsParams& p, cudaStream_t st);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t st);

}  // namespace qg
