// Parameters and launchers of the int8 products (include/gemm_s8.h).
#pragma once
#include "kparams.h"

namespace qg {

// Largest K whose sums of int8 products (at most 2^14 each) fit 32-bit integers.
constexpr int64_t S8_MAX_K = 131071;

struct S8GemmParams {
    EpiParams epi;             // M, N, D, C, alpha, beta, flags, bias
    const int8_t *A, *B;
    int64_t lda, ldb, b_bs;    // bytes
    const float *sa, *sb;      // or null
    int64_t K;
    const int32_t* offsets;    // grouped: device int32[num_experts + 1], else null
    int32_t num_experts;
    int32_t tiles_m;           // token tiles (grouped: an upper bound)
    int32_t tile_rows;         // tokens of a tile
    int32_t kslices;           // streaming kernel: warps that share a row's K
};

// The streaming kernel on the CUDA cores: any M, meant for a few rows per expert.
constexpr int S8_GEMV_ROWS = 8;  // tokens of a tile, at most
cudaError_t launch_s8_gemv(const S8GemmParams& p, int sm_count, cudaStream_t st);
int s8_gemv_slices(int64_t n, int64_t k, int64_t tiles, int sm_count);

}  // namespace qg
