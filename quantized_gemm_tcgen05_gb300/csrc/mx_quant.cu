// Quantisation to 4-bit microscaled formats and its inverse.
//
// Both are one pass over memory: values in once, codes and scales out once
// (2.56 bytes a value for 16-bit input), bounded by HBM.  A warp takes 512
// consecutive columns of a row: every lane 16 values, its loads, its 8 bytes
// of codes and (every fourth or eighth lane) its 4 bytes of scales contiguous
// with its neighbours'.  The block maximum needs no shared memory: a lane
// holds a whole NVFP4 block, two lanes an MXFP4 one.
#include "common.cuh"
#include "mx_quant.cuh"

namespace qg {

namespace {

constexpr int QWARPS = 8;  // rows per block

template <typename T, bool NVF4>
__global__ void __launch_bounds__(32 * QWARPS) mx_quantize_kernel(const __grid_constant__ MxQuantParams p) {
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * QWARPS + warp;
    if (r >= p.rows) return;
    const int64_t chunk = (int64_t)blockIdx.y * 32 + lane;
    const int64_t atoms = mx_atoms(NVF4 ? MXF_NVFP4 : MXF_MXFP4, p.cols);
    const int64_t chunk_end = atoms * (NVF4 ? 4 : 8);
    griddep_wait();
    const int64_t srow = p.offsets ? mx_expert_row(p.offsets, p.num_experts, r, lane) : r;
    if (srow < 0) return;
    const T* row = static_cast<const T*>(p.X) + blockIdx.z * p.x_bstride + r * p.ldx;
    float v[16];
    mx_load16(row, chunk * 16, p.cols, p.vec, v);
    uint2 codes;
    const uint32_t byte = mx_quantize16<NVF4>(v, p.tensor_scale, p.six_g, codes);
    mx_store_codes(static_cast<uint8_t*>(p.Y) + blockIdx.z * p.q_bstride + r * p.ldq, chunk * 16, p.cols, codes);
    // blocks past the row's end are padding: zero, whatever an empty block's scale would be
    const bool pad = (NVF4 ? chunk * 16 : chunk / 2 * 32) >= p.cols;
    mx_store_scales<NVF4>(p.S + blockIdx.z * p.s_bstride, srow, chunk, chunk_end, atoms, pad ? 0u : byte, lane);
}

// E2M1 codes as E4M3 bytes: the magnitude by a byte permute over the eight of
// them, the sign to bit 7.  w: four codes in its low 16 bits.
__device__ __forceinline__ uint32_t mx_codes_e4m3(uint32_t w) {
    const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, w & 0x7777u);
    const uint32_t sign = ((w & 0x8u) << 4) | ((w & 0x80u) << 8) | ((w & 0x800u) << 12) | ((w & 0x8000u) << 16);
    return mag | sign;
}

__device__ __forceinline__ float2 mx_code_pair(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 t, u;\n\tmov.b16 {t, u}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "h"((uint16_t)byte));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct E4M3Out {};  // the codes' own values

template <typename T, bool NVF4>
__global__ void __launch_bounds__(32 * QWARPS) mx_dequantize_kernel(const __grid_constant__ MxQuantParams p) {
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * QWARPS + warp;
    if (r >= p.rows) return;
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + lane) * 16;
    griddep_wait();
    const int64_t srow = p.offsets ? mx_expert_row(p.offsets, p.num_experts, r, lane) : r;
    if (srow < 0 || c0 >= p.cols) return;
    const uint8_t* q = static_cast<const uint8_t*>(p.X) + blockIdx.z * p.q_bstride + r * p.ldq + c0 / 2;
    uint2 codes = make_uint2(0, 0);
    if (c0 + 16 <= p.cols) {
        codes = __ldg(reinterpret_cast<const uint2*>(q));
    } else {
        const int64_t n = (p.cols - c0 + 1) / 2;
        for (int i = 0; i < 8; ++i)
            if (i < n) (i < 4 ? codes.x : codes.y) |= (uint32_t)q[i] << (8 * (i % 4));
    }
    if constexpr (std::is_same<T, E4M3Out>::value) {
        uint8_t* out = static_cast<uint8_t*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx + c0;
        const uint32_t w[4] = {mx_codes_e4m3(codes.x), mx_codes_e4m3(codes.x >> 16), mx_codes_e4m3(codes.y),
                               mx_codes_e4m3(codes.y >> 16)};
        if (p.vec && c0 + 16 <= p.cols) {
            *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c0 + i < p.cols) out[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    } else {
        const int64_t atoms = mx_atoms(NVF4 ? MXF_NVFP4 : MXF_MXFP4, p.cols);
        const float s = mx_scale_value<NVF4>(
            p.S[blockIdx.z * p.s_bstride + mx_scale_at(srow, c0 / (NVF4 ? 16 : 32), atoms)]);
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = mx_code_pair(((i < 4 ? codes.x : codes.y) >> (8 * (i % 4))) & 0xFFu);
            // code * scale is exact (2 + 4 significant bits); the product with g is rounded, then D
            v[2 * i] = f.x * s * p.tensor_scale;
            v[2 * i + 1] = f.y * s * p.tensor_scale;
        }
        mx_store16(static_cast<T*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx, c0, p.cols, p.vec, v);
    }
}

template <typename F>
cudaError_t mx_launch(F kernel, const MxQuantParams& p, int64_t chunks, cudaStream_t st) {
    const int64_t gx = ceil_div(p.rows, QWARPS), gy = ceil_div(chunks, 32);
    if (gx > INT32_MAX || gy > 65535 || p.num > 65535) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)gx, (unsigned)gy, (unsigned)p.num);
    cfg.blockDim = dim3(32 * QWARPS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantParams& p, cudaStream_t st) {
    const bool nv = p.format == MXF_NVFP4;
    const int64_t chunks = mx_atoms(p.format, p.cols) * (nv ? 4 : 8);
    switch (p.type) {
        case DT_F32: return nv ? mx_launch(mx_quantize_kernel<float, true>, p, chunks, st) : mx_launch(mx_quantize_kernel<float, false>, p, chunks, st);
        case DT_F16: return nv ? mx_launch(mx_quantize_kernel<__half, true>, p, chunks, st) : mx_launch(mx_quantize_kernel<__half, false>, p, chunks, st);
        case DT_BF16: return nv ? mx_launch(mx_quantize_kernel<__nv_bfloat16, true>, p, chunks, st) : mx_launch(mx_quantize_kernel<__nv_bfloat16, false>, p, chunks, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_mx_dequantize(const MxQuantParams& p, cudaStream_t st) {
    const bool nv = p.format == MXF_NVFP4;
    const int64_t chunks = ceil_div(p.cols, 16);
    switch (p.type) {
        case DT_F32: return nv ? mx_launch(mx_dequantize_kernel<float, true>, p, chunks, st) : mx_launch(mx_dequantize_kernel<float, false>, p, chunks, st);
        case DT_F16: return nv ? mx_launch(mx_dequantize_kernel<__half, true>, p, chunks, st) : mx_launch(mx_dequantize_kernel<__half, false>, p, chunks, st);
        case DT_BF16: return nv ? mx_launch(mx_dequantize_kernel<__nv_bfloat16, true>, p, chunks, st) : mx_launch(mx_dequantize_kernel<__nv_bfloat16, false>, p, chunks, st);
        case DT_E4M3: return mx_launch(mx_dequantize_kernel<E4M3Out, true>, p, chunks, st);  // no scales read
        default: return cudaErrorInvalidValue;
    }
}

// ---- residual norm -------------------------------------------------------------------

namespace {

// Sum over the block in a fixed order; every thread gets it.  red: one float
// per warp.
__device__ __forceinline__ float mx_block_sum(float x, float* red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    const int warps = blockDim.x / 32;
    if (warps == 1) return x;
    __syncthreads();  // the previous sum has been read
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < warps; ++i) s += red[i];
    return s;
}

__device__ __forceinline__ void mx_load16_any(const void* p, int32_t type, int64_t at, int64_t c0, int64_t cols,
                                              bool vec, float (&v)[16]) {
    if (type == DT_F32)
        mx_load16(static_cast<const float*>(p) + at, c0, cols, vec, v);
    else if (type == DT_F16)
        mx_load16(static_cast<const __half*>(p) + at, c0, cols, vec, v);
    else
        mx_load16(static_cast<const __nv_bfloat16*>(p) + at, c0, cols, vec, v);
}

// A block per row; the row stays in registers between the two norms, NC
// chunks of 16 values a thread, so F, R are read once and r', codes and scales
// written once.  Sums of squares in fp32 over 16 * NC values a thread, then
// over the block.  Bounded by HBM when there are many rows, by the two block
// sums' latency when there are few.
template <typename T, bool NVF4, int NC>
__global__ void __launch_bounds__(NC == 1 ? 256 : 512) mx_norm_kernel(const __grid_constant__ MxNormParams p) {
    __shared__ float red[32];
    griddep_launch_dependents();
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x % 32;
    const float inv = 1.0f / (float)p.cols;
    griddep_wait();
    float v[NC][16];
    if (p.F) {
        const T* frow = static_cast<const T*>(p.F) + r * p.ldf;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            mx_load16(frow, ((int64_t)i * blockDim.x + threadIdx.x) * 16, p.cols, p.vec, v[i]);
            if (p.post) {
#pragma unroll
                for (int j = 0; j < 16; ++j) ss = fmaf(v[i][j], v[i][j], ss);
            }
        }
        const float rs = p.post ? rsqrtf(fmaf(mx_block_sum(ss, red), inv, p.eps)) : 1.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c0 = ((int64_t)i * blockDim.x + threadIdx.x) * 16;
            if (p.post) {
                float w[16];
                mx_load16_any(p.post, p.weight_type, 0, c0, p.cols, p.wvec, w);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[i][j] = v[i][j] * rs * w[j];
            }
            if (p.gate) {
                float w[16];
                mx_load16_any(p.gate, p.gate_type, r * p.gate_ld, c0, p.cols, p.gvec, w);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[i][j] *= w[j];
            }
        }
    }
    const T* rrow = static_cast<const T*>(p.R) + r * p.ldr;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c0 = ((int64_t)i * blockDim.x + threadIdx.x) * 16;
        float x[16];
        mx_load16(rrow, c0, p.cols, p.vec, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            // the sum is rounded to the residual's type before it is normed, so
            // y is the norm of what O holds
            v[i][j] = p.F ? MxIn<T>::round(fmaf(p.residual_scale, v[i][j], x[j])) : x[j];
            ss = fmaf(v[i][j], v[i][j], ss);
        }
        if (p.O) mx_store16(static_cast<T*>(p.O) + r * p.ldo, c0, p.cols, p.vec, v[i]);
    }
    const float rs = rsqrtf(fmaf(mx_block_sum(ss, red), inv, p.eps));
    const int64_t atoms = mx_atoms(NVF4 ? MXF_NVFP4 : MXF_MXFP4, p.cols);
    const int64_t chunk_end = atoms * (NVF4 ? 4 : 8);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t chunk = (int64_t)i * blockDim.x + threadIdx.x, c0 = chunk * 16;
        if (p.pre) {
            float w[16];
            mx_load16_any(p.pre, p.weight_type, 0, c0, p.cols, p.wvec, w);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = v[i][j] * rs * w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] *= rs;
        }
        uint2 codes;
        const uint32_t byte = mx_quantize16<NVF4>(v[i], p.tensor_scale, p.six_g, codes);
        mx_store_codes(p.Q + r * p.ldq, c0, p.cols, codes);
        const bool pad = (NVF4 ? c0 : chunk / 2 * 32) >= p.cols;
        mx_store_scales<NVF4>(p.S, r, chunk, chunk_end, atoms, pad ? 0u : byte, lane);
    }
}

template <typename T, bool NVF4, int NC>
cudaError_t mx_norm_launch(const MxNormParams& p, int threads, cudaStream_t st) {
    return launch_pdl(mx_norm_kernel<T, NVF4, NC>, (int)p.rows, threads, 0, st, p);
}

template <typename T, bool NVF4>
cudaError_t mx_norm_pick(const MxNormParams& p, cudaStream_t st) {
    const int64_t chunks = mx_atoms(p.format, p.cols) * (NVF4 ? 4 : 8);
    // one chunk a thread up to 256 threads, then two, then four
    const int nc = chunks <= 256 ? 1 : (chunks <= 1024 ? 2 : 4);
    const int64_t threads = ceil_div(ceil_div(chunks, nc), 32) * 32;
    if (threads > (nc == 1 ? 256 : 512)) return cudaErrorInvalidValue;
    switch (nc) {
        case 1: return mx_norm_launch<T, NVF4, 1>(p, (int)threads, st);
        case 2: return mx_norm_launch<T, NVF4, 2>(p, (int)threads, st);
        default: return mx_norm_launch<T, NVF4, 4>(p, (int)threads, st);
    }
}

}  // namespace

cudaError_t launch_mx_norm(const MxNormParams& p, cudaStream_t st) {
    const bool nv = p.format == MXF_NVFP4;
    switch (p.type) {
        case DT_F32: return nv ? mx_norm_pick<float, true>(p, st) : mx_norm_pick<float, false>(p, st);
        case DT_F16: return nv ? mx_norm_pick<__half, true>(p, st) : mx_norm_pick<__half, false>(p, st);
        case DT_BF16: return nv ? mx_norm_pick<__nv_bfloat16, true>(p, st) : mx_norm_pick<__nv_bfloat16, false>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qg
