// Parameters and launchers of the 4-bit microscaled products.
#pragma once
#include "mx_params.h"

namespace qg {

struct MxGemmParams {
    EpiParams epi;               // M, N, D, C, alpha, beta, flags, bias
    const float* expert_alpha;   // grouped: factor on alpha per expert, or null
    const int32_t* offsets;      // grouped: device int32[num_experts + 1], else null
    int32_t num_experts;
    int32_t tiles_m, tiles_n;    // output tiles (grouped: tiles_m is an upper bound)
    int32_t k_steps;             // 256-wide K-steps
    int32_t splits;              // CTAs of a cluster, each a share of the K-steps (single-CTA kernel)
    int32_t programs;            // persistent programs (pair kernel)
    int32_t a_rows;              // rows of A a stage holds (a multiple of 8, at most 128)
    int32_t stages;
    int32_t b3d;                 // B's maps take an expert coordinate
    uint32_t idesc;
    int32_t vec32;               // D (and C) rows: 32-byte accesses
    uint32_t* status;
    uint64_t timeout_ns;
};

struct MxMaps {
    CUtensorMap a, b, sa, sb;
};

// Instruction descriptor of tcgen05.mma.kind::mxf4 / mxf4nvf4: A / B format
// E2M1 = 1 (bits 7-9, 10-11), N >> 3 (bits 17-22), scale type (bit 23: E4M3 = 0,
// E8M0 = 1), M >> 4 (bits 24-28), K = 64 (bit 31 = 0).  The byte of a scale
// column that holds the instruction's first scale goes into bits 29-30 (A) and
// 4-5 (B).
QG_HD uint32_t make_idesc_mx(int nvf4, int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((nvf4 ? 0u : 1u) << 23) | ((uint32_t)(m >> 4) << 24);
}

cudaError_t launch_mx_gemm(int bn, int format, const MxMaps& m, const MxGemmParams& p, int grid, cudaStream_t st);
// K = 0: D = act(beta C + bias), of the rows that an expert holds when there are
// offsets.
cudaError_t launch_mx_no_k(const EpiParams& e, const int32_t* offsets, int32_t num_experts, cudaStream_t st);
// Stages of the ring for a tile of a_rows x bn; 0: its partial tiles do not fit.
int mx_gemm_stages(int bn, int format, int a_rows, int splits);


// The CTA-pair kernel: 256 x 256 tiles, persistent clusters of two.
cudaError_t launch_mx_pair(int format, const MxMaps& m, const MxGemmParams& p, int clusters, cudaStream_t st);
// Clusters that can be resident at once.
int mx_pair_max_clusters(int format);

}  // namespace qg
