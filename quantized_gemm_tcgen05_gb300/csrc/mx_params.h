// Parameter blocks of the 4-bit microscaled kernels (include/gemm_mx.h) and
// the integer layout rules they share with the host.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kparams.h"

namespace qg {

enum MxFormat : int32_t { MXF_MXFP4 = 1, MXF_NVFP4 = 2 };

constexpr int MX_ATOM_ROWS = 128;   // rows of a scale atom
constexpr int MX_ATOM_BYTES = 512;  // 128 rows x 4 blocks
constexpr int MX_KSTEP = 256;       // codes of one 128-byte swizzle row

QG_HD int32_t mx_block(int32_t format) { return format == MXF_NVFP4 ? 16 : 32; }
// Atoms along K of one atom row.
QG_HD int64_t mx_atoms(int32_t format, int64_t cols) { return ceil_div(cols, 4 * (int64_t)mx_block(format)); }

// Constants of a launch: g, RN(6 g) and its reciprocal, rounded.
struct MxScaleConst {
    float g, six_g, inv_six_g;
};
inline MxScaleConst mx_scale_const(float g) { return MxScaleConst{g, 6.0f * g, 1.0f / (6.0f * g)}; }

// Quantisation and its inverse: one matrix of `rows` x `cols`, or `num` of them.
struct MxQuantParams {
    const void* X;  // values in (quantise); codes in (dequantise)
    const void* x_end;  // quantise: past the last value
    void* Y;        // codes out; values out
    uint8_t* S;     // scales
    int64_t rows, cols;
    int64_t ldx, x_bstride;  // of the values, elements
    int64_t ldq, q_bstride;  // of the codes, bytes
    int64_t s_bstride;       // bytes
    int32_t num;
    int32_t type;            // of the values (DType)
    int32_t format;
    int32_t vec;             // values: base and rows 32-byte (2) or 16-byte (1) aligned, or neither (0)
    int32_t atoms;           // scale atoms of a row
    MxScaleConst c;
    const int32_t* offsets;  // rows sorted by expert: device int32[num_experts + 1], or null
    int32_t num_experts;
};

struct MxNormParams {
    const void *F, *R;
    const void *f_end, *r_end, *post_end, *pre_end, *gate_end;  // past the last value of each
    void* O;
    uint8_t *Q, *S;
    int64_t rows, cols, ldf, ldr, ldo, ldq;  // ldq in bytes
    int32_t type, format;
    int32_t vec;    // F, R, O: as in MxQuantParams
    int32_t atoms;  // scale atoms of a row
    int32_t sm_count;
    float eps, residual_scale;
    MxScaleConst c;
    const void *post, *pre, *gate;
    int32_t weight_type, gate_type;
    int64_t gate_ld;
    int32_t wvec, gvec;  // weights, gate: likewise
    const int32_t* offsets;  // rows sorted by expert, or null
    int32_t num_experts;
};

cudaError_t launch_mx_quantize(const MxQuantParams& p, cudaStream_t st);
cudaError_t launch_mx_dequantize(const MxQuantParams& p, cudaStream_t st);
cudaError_t launch_mx_norm(const MxNormParams& p, cudaStream_t st);

}  // namespace qg
