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

constexpr int QWARPS = 8;  // warps of a block, a row each

// 32 registers, so that 64 warps an SM keep the loads going: 30 us for 4096 x
// 14336 bf16 (150 MB: 5.0 TB/s); with two rows a warp and 50 registers 30.6.
// NVFP4 spills 16 bytes a thread for them (f32: 40).
template <typename T, bool NVF4>
__global__ void __launch_bounds__(32 * QWARPS, 8) mx_quantize_kernel(const __grid_constant__ MxQuantParams p) {
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = (int)blockIdx.x * QWARPS + warp;
    const int chunk = (int)blockIdx.y * 32 + lane, cols = (int)p.cols;
    const int chunk_end = p.atoms * (NVF4 ? 4 : 8);
    if (r >= p.rows) return;
    griddep_wait();
    const Raw16<T> raw = mx_load16<false>(static_cast<const T*>(p.X) + blockIdx.z * p.x_bstride + r * p.ldx, chunk * 16, cols, p.vec,
                                    p.X, p.x_end);
    int64_t srow = r;
    if (p.offsets) {
        const MxExpertSpan e = mx_expert_of(p.offsets, p.num_experts, p.rows, r, lane);
        if (!e.holds(r)) return;
        srow = e.row0 + (r - e.lo);
    }
    uint2 codes;
    const uint32_t byte = mx_quantize16<NVF4>(mx_values<T>(raw), p.c, codes);
    mx_store_codes(static_cast<uint8_t*>(p.Y) + blockIdx.z * p.q_bstride + r * p.ldq, chunk * 16, cols, codes);
    mx_store_scales<NVF4>(p.S + blockIdx.z * p.s_bstride + mx_scale_row_at(srow, p.atoms), chunk, chunk_end, cols, byte, lane);
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

// a * g for a result that is rounded once more, to 16 bits: towards zero, and odd
// when something was cut off, so that the second rounding sees on which side of a
// tie the product lies (rounded to nearest first, one tensor scale in some 1400 puts
// a code's value on the wrong side in f16, one in 8000 in bf16).  4096 x 14336 to
// bf16 takes 29.0 us with it, 26.8 without (with a branch around it for a g that makes
// the products exact 29.0 for such a g, 30.4 for others).
__device__ __forceinline__ float mul_odd(float a, float g) {
    const float t = __fmul_rz(a, g);
    return fmaf(a, g, -t) != 0.0f ? __uint_as_float(__float_as_uint(t) | 1u) : t;
}

struct E4M3Out {};  // the codes' own values

constexpr int DROWS = 2;  // rows a warp of the inverse takes: it has so little to do for one

// A lane takes 16 codes from either half of 1024: its neighbours' follow directly,
// so whatever the rows' alignment, a warp's accesses are contiguous.
template <typename T, bool NVF4, bool ALIGNED>
__global__ void __launch_bounds__(32 * QWARPS) mx_dequantize_kernel(const __grid_constant__ MxQuantParams p) {
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r0 = (int)blockIdx.x * (QWARPS * DROWS) + warp;
    const int first = ((int)blockIdx.y * 64 + lane) * 16, cols = (int)p.cols;
    if (r0 >= p.rows) return;
    griddep_wait();
    uint2 w[DROWS][2];
#pragma unroll
    for (int j = 0; j < DROWS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c0 = first + 512 * h;
            const uint8_t* q = static_cast<const uint8_t*>(p.X) + blockIdx.z * p.q_bstride + (r0 + j * QWARPS) * p.ldq + c0 / 2;
            w[j][h] = make_uint2(0, 0);
            if (r0 + j * QWARPS >= p.rows) continue;
            if (c0 + 16 <= cols) {
                w[j][h] = *reinterpret_cast<const uint2*>(q);
            } else if (c0 < cols) {
                const int n = (cols - c0 + 1) / 2;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < n) (i < 4 ? w[j][h].x : w[j][h].y) |= (uint32_t)q[i] << (8 * (i % 4));
            }
        }
    MxExpertSpan e{0, p.rows, 0};
    if (p.offsets) e = mx_expert_of(p.offsets, p.num_experts, p.rows, r0, lane);
#pragma unroll
    for (int j = 0; j < DROWS; ++j) {
        const int r = r0 + j * QWARPS;
        if (r >= p.rows) break;
        if (!e.holds(r)) e = mx_expert_of(p.offsets, p.num_experts, p.rows, r, lane);
        if (!e.holds(r)) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c0 = first + 512 * h;
            const uint2 u = w[j][h];
            if constexpr (std::is_same<T, E4M3Out>::value) {
                uint8_t* out = static_cast<uint8_t*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx + c0;
                const uint32_t v[4] = {mx_codes_e4m3(u.x), mx_codes_e4m3(u.x >> 16), mx_codes_e4m3(u.y), mx_codes_e4m3(u.y >> 16)};
                if (!ALIGNED) mx_store_words<uint8_t, 4>(out, v, c0 + 16 <= cols, lane);
                if (c0 + 16 <= cols) {
                    if (ALIGNED) *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < cols) out[i] = (uint8_t)(v[i / 4] >> (8 * (i % 4)));
                }
            } else {
                const uint8_t* sp = p.S + blockIdx.z * p.s_bstride + mx_scale_row_at(e.row0 + (r - e.lo), p.atoms);
                const float s = c0 < cols ? mx_scale_value<NVF4>(sp[mx_block_at(c0 / (NVF4 ? 16 : 32))]) : 0.0f;
                Row16 v;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = mx_code_pair(((i < 4 ? u.x : u.y) >> (8 * (i % 4))) & 0xFFu);
                    // code * scale is exact (2 + 4 significant bits)
                    if constexpr (NVF4 && sizeof(T) == 2)
                        v.p[i] = pack2(mul_odd(f.x * s, p.c.g), mul_odd(f.y * s, p.c.g));
                    else
                        v.p[i] = pack2(f.x * s * p.c.g, f.y * s * p.c.g);
                }
                mx_store16<ALIGNED>(static_cast<T*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx, c0, cols, p.vec, mx_round<T>(v), lane);
            }
        }
    }
}

template <typename F>
cudaError_t mx_launch(F kernel, const MxQuantParams& p, int rows, int64_t chunks, cudaStream_t st) {
    const int64_t gx = ceil_div(p.rows, rows), gy = ceil_div(chunks, 32);
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
    const int64_t chunks = (int64_t)p.atoms * (nv ? 4 : 8);
    switch (p.type) {
        case DT_F32: return nv ? mx_launch(mx_quantize_kernel<float, true>, p, QWARPS, chunks, st) : mx_launch(mx_quantize_kernel<float, false>, p, QWARPS, chunks, st);
        case DT_F16: return nv ? mx_launch(mx_quantize_kernel<__half, true>, p, QWARPS, chunks, st) : mx_launch(mx_quantize_kernel<__half, false>, p, QWARPS, chunks, st);
        case DT_BF16: return nv ? mx_launch(mx_quantize_kernel<__nv_bfloat16, true>, p, QWARPS, chunks, st) : mx_launch(mx_quantize_kernel<__nv_bfloat16, false>, p, QWARPS, chunks, st);
        default: return cudaErrorInvalidValue;
    }
}

template <typename T>
static cudaError_t mx_dequantize_pick(const MxQuantParams& p, cudaStream_t st) {
    const bool nv = p.format == MXF_NVFP4;
    const int64_t chunks = ceil_div(p.cols, 32);
    constexpr int rows = QWARPS * DROWS;
    if (p.vec)
        return nv ? mx_launch(mx_dequantize_kernel<T, true, true>, p, rows, chunks, st)
                  : mx_launch(mx_dequantize_kernel<T, false, true>, p, rows, chunks, st);
    return nv ? mx_launch(mx_dequantize_kernel<T, true, false>, p, rows, chunks, st)
              : mx_launch(mx_dequantize_kernel<T, false, false>, p, rows, chunks, st);
}

cudaError_t launch_mx_dequantize(const MxQuantParams& p, cudaStream_t st) {
    switch (p.type) {
        case DT_F32: return mx_dequantize_pick<float>(p, st);
        case DT_F16: return mx_dequantize_pick<__half>(p, st);
        case DT_BF16: return mx_dequantize_pick<__nv_bfloat16>(p, st);
        case DT_E4M3: return mx_dequantize_pick<E4M3Out>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qg
