// The residual norm that quantises its result: what lies between two blocks, in
// one pass over a row.
#include "common.cuh"
#include "mx_quant.cuh"

namespace qg {

namespace {

// Sum over the block in a fixed order; every thread gets it.  red: 32 floats of
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

template <bool ALIGNED>
__device__ __forceinline__ Row16 mx_load16_any(const void* p, int32_t type, int64_t at, int c0, int cols, int vec,
                                               const void* hi) {
    if (type == DT_BF16) return mx_values<__nv_bfloat16>(mx_load16<ALIGNED>(static_cast<const __nv_bfloat16*>(p) + at, c0, cols, vec, p, hi));
    if (type == DT_F16) return mx_values<__half>(mx_load16<ALIGNED>(static_cast<const __half*>(p) + at, c0, cols, vec, p, hi));
    return mx_values<float>(mx_load16<ALIGNED>(static_cast<const float*>(p) + at, c0, cols, vec, p, hi));
}

__device__ __forceinline__ float mx_sum_squares(const Row16& v, float ss) {
    uint64_t a = pack2(ss, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fma2(v.p[j], v.p[j], a);
    float x, y;
    unpack2(a, x, y);
    return x + y;
}

// Whether two rows' inputs fit a thread's registers.
template <typename T, int NC, bool WIDE>
constexpr bool MX_NORM_AHEAD = NC == 1 && !WIDE && sizeof(T) == 2;

// A block takes rows blockIdx.x, + gridDim.x, ...; a row stays in registers
// between the two norms, NC chunks of 16 values a thread, so F, R are read once
// and r', codes and scales written once.  Sums of squares in fp32 over 16 * NC
// values a thread, then over the block.
//
// A row is a chain of load, sum, sum, store of about 4 us; with a block a row
// that latency and some 580 instructions a warp and chunk bound it (30 us for
// 4096 x 4096 bf16, 110 MB at 3.7 TB/s).  With one chunk a thread of a 16-bit type
// the next row's F and R are requested before the present row's sums (1.5 us less).
//
// ALIGNED: every row starts on a 16-byte boundary (the code for rows that do not
// would cost the others registers).
//
// WIDE: more than 256 threads a row (rows beyond 4096 columns) with 64 registers
// each.  One or two rows an SM then, whose chain of sums nothing hides: 4096 rows
// of 8192 columns take 66 us (3.3 TB/s), of 14336 136 us (2.8 TB/s).  Two chunks a
// thread in half the threads were slower (3001 x 9001, not aligned, with a gate
// per element: 232 us, here 172).  The 64 registers spill: 32 to 144 bytes a thread
// with 16-bit types, 236 to 316 with f32, more where a thread has two chunks (beyond
// 16384 columns).  Of the other forms only f32 (4096 x 4096: 52 us) and unaligned rows do.
template <typename T, bool NVF4, int NC, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(WIDE ? 1024 : 256, WIDE ? 1 : 3) mx_norm_kernel(const __grid_constant__ MxNormParams p) {
    // partial sums of the first and the second norm; two sets, so that a row's are
    // not overwritten while a slower warp still reads the previous row's
    __shared__ float4 red_all[2][16];
    griddep_launch_dependents();
    for (int i = threadIdx.x; i < 128; i += blockDim.x) reinterpret_cast<float*>(red_all)[i] = 0.0f;
    __syncthreads();
    const int lane = threadIdx.x % 32, cols = (int)p.cols;
    const float inv = 1.0f / (float)cols;
    const uint64_t sc2 = pack2(p.residual_scale, p.residual_scale);
    const int chunk_end = p.atoms * (NVF4 ? 4 : 8);
    constexpr bool AHEAD = MX_NORM_AHEAD<T, NC, WIDE>;
    // where registers do not hold both inputs, R is loaded after the first sum
    constexpr bool EARLY = NC * MxIn<T>::LOADS <= 4;
    Raw16<T> f[NC], x[EARLY ? NC : 1];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c0 = (i * (int)blockDim.x + (int)threadIdx.x) * 16;
            if (p.F) f[i] = mx_load16<ALIGNED>(static_cast<const T*>(p.F) + r * p.ldf, c0, cols, p.vec, p.F, p.f_end);
            if constexpr (EARLY) x[i] = mx_load16<ALIGNED>(static_cast<const T*>(p.R) + r * p.ldr, c0, cols, p.vec, p.R, p.r_end);
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
                    const Row16 w = mx_load16_any<ALIGNED>(p.post, p.weight_type, 0, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.wvec, p.post_end);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i].p[j] = mul2(mul2(v[i].p[j], rs2), w.p[j]);
                }
            }
            if (p.gate) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const Row16 w = mx_load16_any<ALIGNED>(p.gate, p.gate_type, r * p.gate_ld, (i * (int)blockDim.x + (int)threadIdx.x) * 16, cols, p.gvec, p.gate_end);
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
            if constexpr (!EARLY) raw = mx_load16<ALIGNED>(static_cast<const T*>(p.R) + r * p.ldr, c0, cols, p.vec, p.R, p.r_end);
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
            if (p.O) mx_store16<ALIGNED>(static_cast<T*>(p.O) + r * p.ldo, c0, cols, p.vec, raw, lane);
        }
        const float rs = rsqrtf(fmaf(mx_block_sum(ss, red + 8), inv, p.eps));
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
                const Row16 w = mx_load16_any<ALIGNED>(p.pre, p.weight_type, 0, chunk * 16, cols, p.wvec, p.pre_end);
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

template <typename T, bool NVF4, int NC, bool WIDE>
cudaError_t mx_norm_launch(const MxNormParams& p, int threads, cudaStream_t st) {
    // blocks that walk the rows only where they request a row ahead
    const int64_t resident = (int64_t)p.sm_count * (768 / threads);
    const int grid = (int)(MX_NORM_AHEAD<T, NC, WIDE> && p.rows > resident ? resident : p.rows);
    if (p.vec && p.wvec && p.gvec) return launch_pdl(mx_norm_kernel<T, NVF4, NC, WIDE, true>, grid, threads, 0, st, p);
    return launch_pdl(mx_norm_kernel<T, NVF4, NC, WIDE, false>, grid, threads, 0, st, p);
}

template <typename T, bool NVF4>
cudaError_t mx_norm_pick(const MxNormParams& p, cudaStream_t st) {
    const int64_t chunks = (int64_t)p.atoms * (NVF4 ? 4 : 8);
    const int nc = chunks <= 1024 ? 1 : 2;  // one chunk a thread up to 16384 columns, then two
    const int64_t threads = ceil_div(ceil_div(chunks, nc), 32) * 32;
    if (threads > 1024) return cudaErrorInvalidValue;
    if (nc == 2) return mx_norm_launch<T, NVF4, 2, true>(p, (int)threads, st);
    if (threads > 256) return mx_norm_launch<T, NVF4, 1, true>(p, (int)threads, st);
    return mx_norm_launch<T, NVF4, 1, false>(p, (int)threads, st);
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
