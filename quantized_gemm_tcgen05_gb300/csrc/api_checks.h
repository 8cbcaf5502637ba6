// Checks of arguments that the operators' C entry points share.  Host code only.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "gemm.h"
#include "handle_internal.h"

namespace qg {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// How rows may be moved: 2 in 32-byte pieces, 1 in 16-byte ones, 0 by element.
inline int row_alignment(const void* p, int64_t ld, int64_t element) {
    if (!p) return 2;
    return aligned(p, 32) && ld * element % 32 == 0 ? 2 : aligned(p, 16) && ld * element % 16 == 0 ? 1 : 0;
}
inline const void* past(const void* p, int64_t n, int64_t element) {
    return p ? static_cast<const char*>(p) + n * element : nullptr;
}
inline int64_t float_size(int32_t t) { return t == GEMM_F32 ? 4 : (t == GEMM_F16 || t == GEMM_BF16) ? 2 : 0; }

inline int check_matrix(const gemm_layout_t* d, int32_t order, int64_t rows, int64_t cols) {
    if (d->order != order) return GEMM_ERR_UNSUPPORTED;
    if (d->rows != rows || d->cols != cols || d->num < 1) return GEMM_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX) return GEMM_ERR_INVALID_ARG;
    const int64_t inner = order == GEMM_ROW_MAJOR ? cols : rows;
    if (d->ld < (inner > 0 ? inner : 1) || d->ld > ((int64_t)1 << 40)) return GEMM_ERR_INVALID_ARG;
    if (d->num > 1 && (d->batch_stride < 0 || d->batch_stride > ((int64_t)1 << 50))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// Whether the offsets of `num` matrices of `lines` lines stay far from 2^63.
inline bool offsets_fit(const gemm_layout_t* d, int64_t lines) {
    const __int128 line = (__int128)lines * d->ld, all = d->num > 1 ? (__int128)d->num * d->batch_stride : 0;
    return line + all < (__int128)1 << 58;
}

inline int check_experts(gemm_handle_t h, const int32_t* offsets, int32_t experts) {
    if (!offsets && experts == 0) return GEMM_OK;
    if (!offsets || experts < 1 || experts > 4096) return GEMM_ERR_INVALID_ARG;
    if (!aligned(offsets, 4) || !handle_device_pointer(h, offsets)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

inline int status_of(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_CUDA;
}

// Nothing throws across the C ABI.
template <typename F>
inline int guarded(gemm_handle_t h, F&& f) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    try {
        const int rc = handle_bind(h);
        return rc ? rc : f();
    } catch (...) {
        return GEMM_ERR_CUDA;
    }
}

}  // namespace qg
