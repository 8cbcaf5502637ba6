// Rows of tokens: quantised to int8 with a scale each, in place or by expert;
// copied by expert; and the experts' rows summed up per token.  One pass over
// memory each, bounded by HBM.
#include "common.cuh"
#include "moe_params.h"
#include "mx_quant.cuh"

namespace qg {

namespace {

// launch_pdl with a grid of several dimensions.
template <typename P>
cudaError_t launch_pdl3(void (*kernel)(const P), dim3 grid, int block, cudaStream_t st, const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Two packed fp32 sums, each rounded to nearest.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Sixteen codes RN(x * f), |x * f| <= 127 but for the product's own rounding: the product is
// rounded to fp32, then 1.5 * 2^23 added, whose sum has the nearest integer (ties to
// even) in its lowest bits.  (The sum is not packed: a packed product and a packed
// sum are contracted to one operation with one rounding, whatever they say.)
__device__ __forceinline__ uint4 s8_codes16(const Row16& v, float f) {
    const uint64_t f2 = pack2(f, f);
    constexpr float MAGIC = 12582912.0f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b, c, d;
        unpack2(mul2(v.p[2 * i], f2), a, b);
        unpack2(mul2(v.p[2 * i + 1], f2), c, d);
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, MAGIC)), __float_as_uint(__fadd_rn(b, MAGIC)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, MAGIC)), __float_as_uint(__fadd_rn(d, MAGIC)), 0x0040);
        w[i] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Warp-wide (lanes hold consecutive chunks): a chunk's codes to row `y`.
__device__ __forceinline__ void s8_store16(uint8_t* y, int c0, int cols, int yvec, const uint4& q, int lane) {
    const bool whole = c0 + 16 <= cols;
    if (yvec) {
        if (whole) *reinterpret_cast<uint4*>(y + c0) = q;
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        mx_store_words<uint8_t, 4>(y + c0, w, whole, lane);
    }
    if (!whole) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c0 + i < cols) y[c0 + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// A block a row: NC chunks of 16 values a thread stay in registers between the
// maximum and the codes.
template <typename T, int NC, bool ALIGNED, int THREADS>
__global__ void __launch_bounds__(THREADS, NC == 2 ? 2048 / THREADS * 3 / 4 : 1) row_quantize_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float red[32];
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int64_t r = blockIdx.x;
    const int cols = p.cols;
    griddep_wait();
    const T* x = static_cast<const T*>(p.X) + blockIdx.y * p.x_bstride + r * p.ldx;
    Raw16<T> raw[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) raw[i] = mx_load16<ALIGNED>(x, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.vec, p.X, p.x_end);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) amax = max_nan(amax, mx_amax16(mx_values<T>(raw[i])));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if (warps > 1) {
        if (lane == 0) red[warp] = amax;
        __syncthreads();
        amax = lane < warps ? red[lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    }
    const bool fine = amax < INFINITY;  // false for NaN
    const float s = __fdiv_rn(amax, 127.0f);
    const bool normal = s >= 0x1p-126f;
    const float f = !fine ? 0.0f : normal ? __fdiv_rn(127.0f, amax) : 0x1p126f;
    const float scale = !fine ? __uint_as_float(0x7FC00000u) : normal ? s : 0x1p-126f;
    uint4 q[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        q[i] = s8_codes16(mx_values<T>(raw[i]), f);
        if (!fine) q[i] = make_uint4(0, 0, 0, 0);
    }
    uint8_t* base = static_cast<uint8_t*>(p.Y) + blockIdx.y * p.y_bstride;
    for (int j = 0; j < p.topk; ++j) {
        const int64_t to = p.map ? (int64_t)p.map[r * p.topk + j] : r;
        if (to < 0 || to >= p.y_rows) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i) s8_store16(base + to * p.ldy, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.yvec, q[i], lane);
        if (threadIdx.x == 0) p.S[blockIdx.y * p.y_rows + to] = scale;
    }
}

// Rows longer than the registers of a block hold: read twice.
template <typename T>
__global__ void __launch_bounds__(1024) row_quantize_long_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float red[32];
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t r = blockIdx.x;
    const int cols = p.cols, end = (cols + 511) / 512 * 32;  // whole warps of chunks
    griddep_wait();
    const T* x = static_cast<const T*>(p.X) + blockIdx.y * p.x_bstride + r * p.ldx;
    float amax = 0.0f;
    for (int c = threadIdx.x; c < end; c += blockDim.x)
        amax = max_nan(amax, mx_amax16(mx_values<T>(mx_load16<false>(x, c * 16, cols, p.vec, p.X, p.x_end))));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if (lane == 0) red[warp] = amax;
    __syncthreads();
    amax = red[lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    const bool fine = amax < INFINITY;
    const float s = __fdiv_rn(amax, 127.0f);
    const bool normal = s >= 0x1p-126f;
    const float f = !fine ? 0.0f : normal ? __fdiv_rn(127.0f, amax) : 0x1p126f;
    const float scale = !fine ? __uint_as_float(0x7FC00000u) : normal ? s : 0x1p-126f;
    uint8_t* base = static_cast<uint8_t*>(p.Y) + blockIdx.y * p.y_bstride;
    for (int c = threadIdx.x; c < end; c += blockDim.x) {
        uint4 q = s8_codes16(mx_values<T>(mx_load16<false>(x, c * 16, cols, p.vec, p.X, p.x_end)), f);
        if (!fine) q = make_uint4(0, 0, 0, 0);
        for (int j = 0; j < p.topk; ++j) {
            const int64_t to = p.map ? (int64_t)p.map[r * p.topk + j] : r;
            if (to < 0 || to >= p.y_rows) continue;
            s8_store16(base + to * p.ldy, c * 16, cols, p.yvec, q, lane);
        }
    }
    if (threadIdx.x == 0)
        for (int j = 0; j < p.topk; ++j) {
            const int64_t to = p.map ? (int64_t)p.map[r * p.topk + j] : r;
            if (to >= 0 && to < p.y_rows) p.S[blockIdx.y * p.y_rows + to] = scale;
        }
}

// Many rows want many bytes in flight: two chunks a thread in half the threads, few
// registers (4096 rows of 16-bit values: 4096 columns 9.6 us, with one chunk 10.7; 8192
// 17.1, 20.0; 14336 35.6, 38.9 at 4.9 TB/s; f32 x 14336 45 us at 6.5 TB/s).
template <typename T>
cudaError_t quantize_t(const RowsParams& p, cudaStream_t st) {
    const int64_t chunks = ceil_div(p.cols, 16);
    dim3 grid((unsigned)p.rows, (unsigned)p.num);
    auto threads = [&](int nc) { return (int)(ceil_div(ceil_div(chunks, nc), 32) * 32); };
    if (chunks > 2048) return launch_pdl3(row_quantize_long_kernel<T>, grid, 1024, st, p);
    if (chunks > 512) {
        if (p.vec) return launch_pdl3(row_quantize_kernel<T, 2, true, 1024>, grid, threads(2), st, p);
        if (chunks <= 1024) return launch_pdl3(row_quantize_kernel<T, 1, false, 1024>, grid, threads(1), st, p);
        return launch_pdl3(row_quantize_kernel<T, 2, false, 1024>, grid, threads(2), st, p);
    }
    if (!p.vec) return launch_pdl3(row_quantize_kernel<T, 1, false, 512>, grid, threads(1), st, p);
    if constexpr (sizeof(T) == 2) {
        if (chunks >= 128 && p.rows >= 1024) return launch_pdl3(row_quantize_kernel<T, 2, true, 256>, grid, threads(2), st, p);
    }
    return launch_pdl3(row_quantize_kernel<T, 1, true, 512>, grid, threads(1), st, p);
}

// Bytes copied in units of U: a block a row, or several where rows are few. 1333 x 4104
// f16 to six rows each: 14.8 us, 77 MB at 5.2 TB/s.
template <typename U>
__global__ void __launch_bounds__(256) row_copy_kernel(const __grid_constant__ RowsParams p) {
    griddep_launch_dependents();
    const int64_t r = blockIdx.x, bytes = (int64_t)p.cols * p.element, units = bytes / (int64_t)sizeof(U);
    const char* x = static_cast<const char*>(p.X) + r * p.ldx * p.element;
    griddep_wait();
    for (int64_t c = blockIdx.y * (int64_t)blockDim.x + threadIdx.x; c < units; c += (int64_t)gridDim.y * blockDim.x) {
        const U u = reinterpret_cast<const U*>(x)[c];
        for (int j = 0; j < p.topk; ++j) {
            const int64_t to = p.map[r * p.topk + j];
            if (to >= 0 && to < p.y_rows) reinterpret_cast<U*>(static_cast<char*>(p.Y) + to * p.ldy * p.element)[c] = u;
        }
    }
    // what is left is less than a unit
    if (blockIdx.y == 0 && threadIdx.x < bytes - units * (int64_t)sizeof(U)) {
        const int64_t c = units * (int64_t)sizeof(U) + threadIdx.x;
        for (int j = 0; j < p.topk; ++j) {
            const int64_t to = p.map[r * p.topk + j];
            if (to >= 0 && to < p.y_rows) static_cast<char*>(p.Y)[to * p.ldy * p.element + c] = x[c];
        }
    }
}

// A thread has 16 columns of a token; four of its rows are in flight together. 4096 x 4096
// bf16, six rows a token and C: 45 us, 269 MB at 5.9 TB/s; rows that no vector access
// fits (3001 x 4097) 2.6 TB/s.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ CombineParams p) {
    griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x % 32, c0 = ((int)blockIdx.y * 128 + (int)threadIdx.x) * 16, cols = p.cols;
    griddep_wait();
    const bool use_c = p.beta != 0.0f;
    Raw16<T> c;
    if (use_c) c = mx_load16<ALIGNED>(static_cast<const T*>(p.C) + t * p.ldc, c0, cols, p.vec, p.C, p.c_end);
    Row16 sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum.p[i] = 0;
    for (int j0 = 0; j0 < p.topk; j0 += 4) {
        Raw16<T> y[4];
        float w[4];
        bool in[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool some = j0 + q < p.topk;
            const int64_t at = t * p.topk + j0 + q;
            const int64_t row = some ? (int64_t)p.map[at] : -1;
            w[q] = some ? p.weights[at] : 0.0f;
            in[q] = row >= 0 && row < p.y_rows;
            if (in[q]) y[q] = mx_load16<ALIGNED>(static_cast<const T*>(p.Y) + row * p.ldy, c0, cols, p.vec, p.Y, p.y_end);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (j0 + q >= p.topk) break;
            const uint64_t w2 = pack2(w[q], w[q]);
            if (in[q]) {
                const Row16 v = mx_values<T>(y[q]);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum.p[i] = fma2(w2, v.p[i], sum.p[i]);
            } else {
                const uint64_t z2 = pack2(w[q] * 0.0f, w[q] * 0.0f);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum.p[i] = add2(sum.p[i], z2);
            }
        }
    }
    if (use_c) {
        const Row16 v = mx_values<T>(c);
        const uint64_t b2 = pack2(p.beta, p.beta);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum.p[i] = fma2(b2, v.p[i], sum.p[i]);
    }
    mx_store16<ALIGNED>(static_cast<T*>(p.D) + t * p.ldd, c0, cols, p.vec, mx_round<T>(sum), lane);
}

}  // namespace

cudaError_t launch_row_quantize(const RowsParams& p, cudaStream_t st) {
    switch (p.type) {
        case DT_F32: return quantize_t<float>(p, st);
        case DT_F16: return quantize_t<__half>(p, st);
        case DT_BF16: return quantize_t<__nv_bfloat16>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_row_copy(const RowsParams& p, cudaStream_t st) {
    // few rows are spread over several blocks each
    const int64_t per = ceil_div((int64_t)p.cols * p.element, 256 * p.copy_unit);
    const int64_t parts = p.rows >= 1024 ? 1 : ceil_div(1024, p.rows);
    dim3 grid((unsigned)p.rows, (unsigned)(per < 1 ? 1 : per < parts ? per : parts));
    switch (p.copy_unit) {
        case 16: return launch_pdl3(row_copy_kernel<uint4>, grid, 256, st, p);
        case 8: return launch_pdl3(row_copy_kernel<uint2>, grid, 256, st, p);
        case 4: return launch_pdl3(row_copy_kernel<uint32_t>, grid, 256, st, p);
        case 2: return launch_pdl3(row_copy_kernel<uint16_t>, grid, 256, st, p);
        default: return launch_pdl3(row_copy_kernel<uint8_t>, grid, 256, st, p);
    }
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t st) {
    dim3 grid((unsigned)p.tokens, (unsigned)ceil_div(p.cols, 128 * 16));
    switch (p.type) {
        case DT_F32: return p.vec ? launch_pdl3(combine_kernel<float, true>, grid, 128, st, p) : launch_pdl3(combine_kernel<float, false>, grid, 128, st, p);
        case DT_F16: return p.vec ? launch_pdl3(combine_kernel<__half, true>, grid, 128, st, p) : launch_pdl3(combine_kernel<__half, false>, grid, 128, st, p);
        case DT_BF16: return p.vec ? launch_pdl3(combine_kernel<__nv_bfloat16, true>, grid, 128, st, p) : launch_pdl3(combine_kernel<__nv_bfloat16, false>, grid, 128, st, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qg
