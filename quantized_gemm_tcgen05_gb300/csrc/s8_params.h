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
    // the tensor-core kernels
    int32_t tiles_n;           // tiles of channels
    int32_t k_steps;           // 128-wide K-steps
    int32_t splits;            // CTAs of a cluster, each a share of the K-steps
    int32_t programs;          // persistent programs (pair kernel)
    int32_t b3d;               // B's map takes an expert coordinate
    uint32_t idesc;
    int32_t vec4;              // D (and C): four columns of a row at once
    uint32_t* status;
    uint64_t timeout_ns;
};

struct S8Maps {
    CUtensorMap a, b;
};

constexpr int S8_KSTEP = 128;   // codes of one 128-byte swizzle row
constexpr int S8_CHUNK = 8;     // K-steps whose sums fp32 holds exactly: 1024 products of at most 2^14

// The streaming kernel on the CUDA cores: a token a tile, up to 65535 of them.
cudaError_t launch_s8_gemv(const S8GemmParams& p, cudaStream_t st);
int s8_gemv_slices(int64_t n, int64_t k, int64_t tokens, int sm_count);

// The tensor-core kernel, one tile of 128 channels x up to `width` tokens per
// cluster (width 32 or 128).
cudaError_t launch_s8_gemm(int width, const S8Maps& m, const S8GemmParams& p, int grid, cudaStream_t st);
// Whether the kernel was built with the registers that its warps share out.
bool s8_gemm_usable(int width);

// The CTA-pair kernel: 256 channels x up to S8_PAIR_TOKENS tokens, persistent
// clusters of two.
constexpr int S8_PAIR_TOKENS = 192;
cudaError_t launch_s8_pair(const S8Maps& m, const S8GemmParams& p, int clusters, cudaStream_t st);
// Clusters that can be resident at once.
int s8_pair_max_clusters();

}  // namespace qg
