// What every int8 product does with a finished sum.
#pragma once
#include "mx_epilogue.cuh"
#include "s8_params.h"

namespace qg {

// An exact integer sum to the value that the fused steps start from: converted,
// times the token's factor alpha * sa, times the channel's.  Every kernel takes
// it from here, so results do not depend on which one served the call.
__device__ __forceinline__ float s8_scaled(int32_t sum, float token, float channel) {
    return __fmul_rn(__fmul_rn((float)sum, token), channel);
}

__device__ __forceinline__ float s8_token_factor(const S8GemmParams& p, int64_t m) {
    return p.sa ? __fmul_rn(p.epi.alpha, p.sa[m]) : p.epi.alpha;
}
__device__ __forceinline__ float s8_channel_factor(const S8GemmParams& p, int64_t expert, int64_t n) {
    return p.sb ? p.sb[expert * p.epi.N + n] : 1.0f;
}

}  // namespace qg
