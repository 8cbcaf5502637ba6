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

// 32 registers, so that 64 warps an SM keep the loads going: 28.4 us for 4096 x
// 14336 bf16 (150 MB: 5.3 TB/s); with two rows a warp and 50 registers 30.6.
template <typename T, bool NVF4>
__global__ void __launch_bounds__(32 * QWARPS, 8) mx_quantize_kernel(const __grid_constant__ MxQuantParams p) {
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = (int)blockIdx.x * QWARPS + warp;
    const int chunk = (int)blockIdx.y * 32 + lane, cols = (int)p.cols;
    const int chunk_end = p.atoms * (NVF4 ? 4 : 8);
    if (r >= p.rows) return;
    griddep_wait();
    const Raw16<T> raw = mx_load16(static_cast<const T*>(p.X) + blockIdx.z * p.x_bstride + r * p.ldx, chunk * 16, cols, p.vec);
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

struct E4M3Out {};  // the codes' own values

constexpr int DROWS = 2;  // rows a warp of the inverse takes: it has so little to do for one

// A lane takes 16 codes from either half of 1024: its neighbours' follow directly,
// so whatever the rows' alignment, a warp's accesses are contiguous.
template <typename T, bool NVF4>
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
            if (c0 >= cols) break;
            const uint2 u = w[j][h];
            if constexpr (std::is_same<T, E4M3Out>::value) {
                uint8_t* out = static_cast<uint8_t*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx + c0;
                const uint32_t v[4] = {mx_codes_e4m3(u.x), mx_codes_e4m3(u.x >> 16), mx_codes_e4m3(u.y), mx_codes_e4m3(u.y >> 16)};
                if (p.vec && c0 + 16 <= cols) {
                    *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < cols) out[i] = (uint8_t)(v[i / 4] >> (8 * (i % 4)));
                }
            } else {
                const uint8_t* sp = p.S + blockIdx.z * p.s_bstride + mx_scale_row_at(e.row0 + (r - e.lo), p.atoms);
                const float s = mx_scale_value<NVF4>(sp[mx_block_at(c0 / (NVF4 ? 16 : 32))]);
                Row16 v;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = mx_code_pair(((i < 4 ? u.x : u.y) >> (8 * (i % 4))) & 0xFFu);
                    // code * scale is exact (2 + 4 significant bits); the product with g is rounded, then D
                    v.p[i] = pack2(f.x * s * p.c.g, f.y * s * p.c.g);
                }
                mx_store16(static_cast<T*>(p.Y) + blockIdx.z * p.x_bstride + r * p.ldx, c0, cols, p.vec, mx_round<T>(v));
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

cudaError_t launch_mx_dequantize(const MxQuantParams& p, cudaStream_t st) {
    const bool nv = p.format == MXF_NVFP4;
    const int64_t chunks = ceil_div(p.cols, 32);
    switch (p.type) {
        case DT_F32: return nv ? mx_launch(mx_dequantize_kernel<float, true>, p, QWARPS * DROWS, chunks, st) : mx_launch(mx_dequantize_kernel<float, false>, p, QWARPS * DROWS, chunks, st);
        case DT_F16: return nv ? mx_launch(mx_dequantize_kernel<__half, true>, p, QWARPS * DROWS, chunks, st) : mx_launch(mx_dequantize_kernel<__half, false>, p, QWARPS * DROWS, chunks, st);
        case DT_BF16: return nv ? mx_launch(mx_dequantize_kernel<__nv_bfloat16, true>, p, QWARPS * DROWS, chunks, st) : mx_launch(mx_dequantize_kernel<__nv_bfloat16, false>, p, QWARPS * DROWS, chunks, st);
        case DT_E4M3: return mx_launch(mx_dequantize_kernel<E4M3Out, true>, p, QWARPS * DROWS, chunks, st);  // no scales read
        default: return cudaErrorInvalidValue;
    }
}

// ---- residual norm -------------------------------------------------------------------

namespace {

// Sum over the block in a fixed order; every thread gets it.  red: 16 floats of
// this sum's own.
__device__ __forceinline__ float mx_block_sum(float x, float4* red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    const int warps = blockDim.x / 32;
    if (warps == 1) return x;
    if (threadIdx.x % 32 == 0) reinterpret_cast<float*>(red)[threadIdx.x / 32] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < warps; i += 4) {
        const float4 f = red[i / 4];  // floats past the last warp's are zero
        s += (f.x + f.y) + (f.z + f.w);
    }
    return s;
}

__device__ __forceinline__ Row16 mx_load16_any(const void* p, int32_t type, int64_t at, int c0, int cols, int vec) {
    if (type == DT_BF16) return mx_values<__nv_bfloat16>(mx_load16(static_cast<const __nv_bfloat16*>(p) + at, c0, cols, vec));
    if (type == DT_F16) return mx_values<__half>(mx_load16(static_cast<const __half*>(p) + at, c0, cols, vec));
    return mx_values<float>(mx_load16(static_cast<const float*>(p) + at, c0, cols, vec));
}

__device__ __forceinline__ float mx_sum_squares(const Row16& v, float ss) {
    uint64_t a = pack2(ss, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fma2(v.p[j], v.p[j], a);
    float x, y;
    unpack2(a, x, y);
    return x + y;
}

// A block takes rows blockIdx.x, + gridDim.x, ...; a row stays in registers
// between the two norms, NC chunks of 16 values a thread, so F, R are read once
// and r', codes and scales written once.  Sums of squares in fp32 over 16 * NC
// values a thread, then over the block.
//
// A row is a chain of load, sum, sum, store of about 4 us, so with a block a row
// the chain's latency bounds it (29.4 us for 4096 x 4096 bf16, 3.7 TB/s, whatever
// is taken out of the arithmetic).  With one chunk a thread the next row's F and R
// are requested before the present row's sums, which hides the loads (16-bit
// types; two rows of fp32 do not fit the registers).
template <typename T, bool NVF4, int NC>
__global__ void __launch_bounds__(NC == 1 ? 256 : 512, NC == 1 ? 3 : 1) mx_norm_kernel(const __grid_constant__ MxNormParams p) {
    // partial sums of the first and the second norm; two sets, so that a row's are
    // not overwritten while a slower warp still reads the previous row's
    __shared__ float4 red_all[2][8];
    griddep_launch_dependents();
    if (threadIdx.x < 64) reinterpret_cast<float*>(red_all)[threadIdx.x] = 0.0f;
    __syncthreads();
    const int lane = threadIdx.x % 32, cols = (int)p.cols;
    const float inv = 1.0f / (float)cols;
    const uint64_t sc2 = pack2(p.residual_scale, p.residual_scale);
    const int chunk_end = p.atoms * (NVF4 ? 4 : 8);
    constexpr bool AHEAD = NC == 1 && sizeof(T) == 2;
    // where registers do not hold both inputs, R is loaded after the first sum
    constexpr bool EARLY = NC * MxIn<T>::LOADS <= 4;
    Raw16<T> f[NC], x[EARLY ? NC : 1];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c0 = (i * (int)blockDim.x + (int)threadIdx.x) * 16;
            if (p.F) f[i] = mx_load16(static_cast<const T*>(p.F) + r * p.ldf, c0, cols, p.vec);
            if constexpr (EARLY) x[i] = mx_load16(static_cast<const T*>(p.R) + r * p.ldr, c0, cols, p.vec);
        }
    };
    griddep_wait();
    if (AHEAD) load(blockIdx.x);
    int it = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, ++it) {
        float4* red = red_all[it & 1];
        if (!AHEAD) load(r);
        Row16 v[NC];
        if (p.F) {
#pragma unroll
            for (int i = 0; i < NC; ++i) v[i] = mx_values<T>(f[i]);
        }
        const Raw16<T> now = x[0];
        if (AHEAD && r + gridDim.x < p.rows) load(r + gridDim.x);
        if (p.F) {
            if (p.post) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i) ss = mx_sum_squares(v[i], ss);
                const float rs = rsqrtf(fmaf(mx_block_sum(ss, red), inv, p.eps));
                const uint64_t rs2 = pack2(rs, rs);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const Row16 w = mx_load16_any(p.post, p.weight_type, 0, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.wvec);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i].p[j] = mul2(mul2(v[i].p[j], rs2), w.p[j]);
                }
            }
            if (p.gate) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const Row16 w = mx_load16_any(p.gate, p.gate_type, r * p.gate_ld, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.gvec);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i].p[j] = mul2(v[i].p[j], w.p[j]);
                }
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c0 = (i * (int)blockDim.x + (int)threadIdx.x) * 16;
            Raw16<T> raw = AHEAD ? now : x[EARLY ? i : 0];
            if constexpr (!EARLY) raw = mx_load16(static_cast<const T*>(p.R) + r * p.ldr, c0, cols, p.vec);
            Row16 s = mx_values<T>(raw);
            if (p.F) {
                // the sum is rounded to the residual's type before it is normed, so
                // y is the norm of what O holds
#pragma unroll
                for (int j = 0; j < 8; ++j) s.p[j] = fma2(sc2, v[i].p[j], s.p[j]);
                raw = mx_round<T>(s);
                s = mx_values<T>(raw);
            }
            v[i] = s;
            ss = mx_sum_squares(s, ss);
            if (p.O) mx_store16(static_cast<T*>(p.O) + r * p.ldo, c0, cols, p.vec, raw);
        }
        const float rs = rsqrtf(fmaf(mx_block_sum(ss, red + 4), inv, p.eps));
        const uint64_t rs2 = pack2(rs, rs);
        int64_t scale_row = r;
        if (p.offsets) {
            const MxExpertSpan e = mx_expert_of(p.offsets, p.num_experts, p.rows, r, lane);
            if (!e.holds(r)) continue;  // (O is written, Q and S are not)
            scale_row = e.row0 + (r - e.lo);
        }
        uint8_t* srow = p.S + mx_scale_row_at(scale_row, p.atoms);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int chunk = i * (int)blockDim.x + (int)threadIdx.x;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].p[j] = mul2(v[i].p[j], rs2);
            if (p.pre) {
                const Row16 w = mx_load16_any(p.pre, p.weight_type, 0, chunk * 16, cols, p.wvec);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].p[j] = mul2(v[i].p[j], w.p[j]);
            }
            uint2 codes;
            const uint32_t byte = mx_quantize16<NVF4>(v[i], p.c, codes);
            mx_store_codes(p.Q + r * p.ldq, chunk * 16, cols, codes);
            mx_store_scales<NVF4>(srow, chunk, chunk_end, cols, byte, lane);
        }
    }
}

template <typename T, bool NVF4, int NC>
cudaError_t mx_norm_launch(const MxNormParams& p, int threads, cudaStream_t st) {
    const int64_t resident = (int64_t)p.sm_count * (NC == 1 ? 768 / threads : 1);
    return launch_pdl(mx_norm_kernel<T, NVF4, NC>, (int)(p.rows < resident ? p.rows : resident), threads, 0, st, p);
}

template <typename T, bool NVF4>
cudaError_t mx_norm_pick(const MxNormParams& p, cudaStream_t st) {
    const int64_t chunks = (int64_t)p.atoms * (NVF4 ? 4 : 8);
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
