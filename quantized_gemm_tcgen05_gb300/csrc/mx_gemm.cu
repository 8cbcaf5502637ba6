// Instantiations of the one-tile 4-bit microscaled product.
#include "mx_gemm.cuh"

namespace qg {

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
