// Instantiations of the CTA-pair 4-bit microscaled product.
#include "mx_pair.cuh"

namespace qg {

cudaError_t launch_mx_pair(int format, const MxMaps& m, const MxGemmParams& p, int clusters, cudaStream_t st) {
    return format == MXF_NVFP4 ? launch_mx_pair_t<true>(m, p, clusters, st) : launch_mx_pair_t<false>(m, p, clusters, st);
}

int mx_pair_max_clusters(int format) {
    return format == MXF_NVFP4 ? mx_pair_clusters_t<true>() : mx_pair_clusters_t<false>();
}

}  // namespace qg
