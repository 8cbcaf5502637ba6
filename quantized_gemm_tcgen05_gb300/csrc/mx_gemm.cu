// Instantiations of the one-tile 4-bit microscaled product, and what is left of a
// product without K.
#include "mx_gemm.cuh"
#include "mx_quant.cuh"

namespace qg {

namespace {

// A block a row.
__global__ void __launch_bounds__(256)
    mx_no_k_kernel(const __grid_constant__ EpiParams e, const int32_t* offsets, int32_t num_experts) {
    const int lane = threadIdx.x % 32;
    EpiArith ar = epi_arith(e);
    ar.alpha = 0.0f;  // (of no products)
    for (int64_t m = blockIdx.x; m < e.M; m += gridDim.x) {
        if (offsets && !mx_expert_of(offsets, num_experts, e.M, m, lane).holds(m)) continue;
        for (int64_t n = threadIdx.x; n < e.N; n += 256) {
            if (!mx_block_in_bounds(e, m, 1, n, 1)) continue;
            const float c = e.beta != 0.0f ? ld_elem(e.C, e.d_type, m * e.ldc + n) : 0.0f;
            float x, unused;
            with_epi_act(e, [&](auto act) {
                mx_value2_any<decltype(act)::value>(ar, e.d_type, 0.0f, 0.0f, c, c, bias_at(ar, n), 0.0f, x, unused);
            });
            st_elem(e.D, e.d_type, m * e.ldd + n, x);
        }
    }
}

}  // namespace

cudaError_t launch_mx_no_k(const EpiParams& e, const int32_t* offsets, int32_t num_experts, cudaStream_t st) {
    mx_no_k_kernel<<<(unsigned)(e.M < 8192 ? e.M : 8192), 256, 0, st>>>(e, offsets, num_experts);
    return cudaGetLastError();
}

cudaError_t launch_mx_gemm(int bn, int format, const MxMaps& m, const MxGemmParams& p, int grid, cudaStream_t st) {
    const bool nv = format == MXF_NVFP4;
    switch (bn) {
        case 64: return nv ? launch_mx_bn<64, true>(m, p, grid, st) : launch_mx_bn<64, false>(m, p, grid, st);
        case 128: return nv ? launch_mx_bn<128, true>(m, p, grid, st) : launch_mx_bn<128, false>(m, p, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

int mx_gemm_stages(int bn, int format, int a_rows, int splits) {
    const bool nv = format == MXF_NVFP4;
    if (bn == 64) return nv ? MxCfg<64, true>::max_stages(a_rows, splits) : MxCfg<64, false>::max_stages(a_rows, splits);
    return nv ? MxCfg<128, true>::max_stages(a_rows, splits) : MxCfg<128, false>::max_stages(a_rows, splits);
}

}  // namespace qg
