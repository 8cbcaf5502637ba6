// Streaming int8 product on the CUDA cores, one token at a time: B's codes are the
// work, four products an instruction (dp4a) into exact 32-bit sums.
//
// A warp owns R = 4 rows of B and one of `kslices` contiguous slices of K; its lanes
// take U 16-byte chunks at a time.  A block of 8 warps covers 8 / kslices row groups for
// one token.  Lanes' and slices' sums are integers: any order gives the same.
//
// Measured: 1x4096x14336 13.3 us (59 MB: 4.4 TB/s), launch and the last warps' sums a
// third of it.  Two, four or eight tokens a warp were no quicker than the tensor cores
// (2x4096x14336 18.5 us, there 15.6) and, by experts, no quicker than a token each (32
// rows by 32 experts of 2048 x 4096: 40.7 us, with two 41.8, four 42.0, eight 48.9).
#include "s8_epilogue.cuh"

namespace qg {

namespace {

constexpr int R = 4, WARPS = 8, U = 2;

// Chunk c of a row of K codes; past K zeros, and nothing is read there.
__device__ __forceinline__ uint4 chunk_of(const int8_t* row, int64_t c, int64_t K) {
    if ((c + 1) * 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row) + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (c * 16 + i < K) w[i / 4] |= (uint32_t)(uint8_t)row[c * 16 + i] << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int s) {
    s = __dp4a((int)a.x, (int)b.x, s);
    s = __dp4a((int)a.y, (int)b.y, s);
    s = __dp4a((int)a.z, (int)b.z, s);
    return __dp4a((int)a.w, (int)b.w, s);
}

__global__ void __launch_bounds__(WARPS * 32, 4) s8_gemv_kernel(const __grid_constant__ S8GemmParams p) {
    __shared__ int32_t red[WARPS][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.kslices, per_block = WARPS / S;
    const int gi = warp / S, s = warp % S;
    const int64_t N = p.epi.N, K = p.K;
    const int64_t nchunk = (K + 15) / 16, cps = (nchunk + S - 1) / S;
    const int64_t cbeg = s * cps, cend = cbeg + cps < nchunk ? cbeg + cps : nchunk;
    const int64_t ngroups = (N + R - 1) / R;
    griddep_launch_dependents();
    if (!p.offsets) {
        // warm L2 with this warp's first codes while the previous kernel in the stream
        // finishes (a hint: L2 is where memory is coherent)
        const int64_t grp = (int64_t)blockIdx.x * per_block + gi;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = cbeg + lane + 32 * u;
                if (grp * R + r < N && c < cend) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.B + (grp * R + r) * p.ldb + c * 16));
            }
    }
    griddep_wait();
    int expert = 0, rows = 1;
    int64_t row = blockIdx.y, atom_row = 0;
    if (p.offsets && !mx_expert_block(p.offsets, p.num_experts, p.epi.M, 1, blockIdx.y, lane, &expert, &row, &rows, &atom_row)) return;
    if (rows <= 0) return;
    const int8_t* A = p.A + row * p.lda;
    const int8_t* B = p.B + expert * p.b_bs;
    const EpiArith ar0 = epi_arith(p.epi);
    for (int64_t gbase = (int64_t)blockIdx.x * per_block; gbase < ngroups; gbase += (int64_t)gridDim.x * per_block) {
        const int64_t grp = gbase + gi;
        int32_t acc[R] = {};
        if (grp < ngroups) {
            const int8_t* brow[R];
#pragma unroll
            for (int r = 0; r < R; ++r)  // (rows past N read the last one; their sums are not stored)
                brow[r] = B + (grp * R + r < N ? grp * R + r : N - 1) * p.ldb;
            for (int64_t c = cbeg + lane; c < cend; c += 32 * U) {
                uint4 b[U][R];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (c + 32 * u < cend) b[u][r] = chunk_of(brow[r], c + 32 * u, K);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c + 32 * u >= cend) break;
                    const uint4 a = chunk_of(A, c + 32 * u, K);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r] = dot16(a, b[u][r], acc[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int32_t v = __reduce_add_sync(0xFFFFFFFFu, acc[r]);
            if (lane == 0) red[warp][r] = v;
        }
        __syncthreads();
        // a thread takes a pair of neighbouring columns
        for (int t = threadIdx.x; t < per_block * (R / 2); t += WARPS * 32) {
            const int g2 = t / (R / 2), r = t % (R / 2) * 2;
            const int64_t n = (gbase + g2) * R + r;
            if (n >= N) continue;
            const int have = N - n < 2 ? 1 : 2;
            if (!mx_block_in_bounds(p.epi, row, 1, n, have)) continue;
            int32_t s0 = 0, s1 = 0;
            for (int k = 0; k < S; ++k) {
                s0 += red[g2 * S + k][r];
                s1 += red[g2 * S + k][r + 1];
            }
            EpiArith ar = ar0;
            ar.alpha = 1.0f;
            const float token = s8_token_factor(p, row);
            const float v0 = s8_scaled(s0, token, s8_channel_factor(p, expert, n));
            const float v1 = have > 1 ? s8_scaled(s1, token, s8_channel_factor(p, expert, n + 1)) : 0.0f;
            const bool use_c = ar.beta != 0.0f;
            const float c0 = use_c ? ld_elem(p.epi.C, p.epi.d_type, row * p.epi.ldc + n) : 0.0f;
            const float c1 = use_c && have > 1 ? ld_elem(p.epi.C, p.epi.d_type, row * p.epi.ldc + n + 1) : 0.0f;
            float x0, x1;
            with_epi_act(p.epi, [&](auto act) {
                constexpr int ACT = decltype(act)::value;
                const float b0 = ACT >= 0 ? bias_at(ar, n) : 0.0f, b1 = ACT >= 0 && have > 1 ? bias_at(ar, n + 1) : 0.0f;
                mx_value2_any<ACT>(ar, p.epi.d_type, v0, v1, c0, c1, b0, b1, x0, x1);
            });
            st_elem(p.epi.D, p.epi.d_type, row * p.epi.ldd + n, x0);
            if (have > 1) st_elem(p.epi.D, p.epi.d_type, row * p.epi.ldd + n + 1, x1);
        }
        __syncthreads();  // red[] is written again
    }
}

}  // namespace

int s8_gemv_slices(int64_t n, int64_t k, int64_t tokens, int sm_count) {
    // as many slices as leave all warps resident at once and every lane a chunk
    // (1x4096x14336: 13.3 us in four, 15.5 in eight, 17.8 in two; 1x14336x4096 14.2 us
    // unsliced, 16 in two or four)
    const int64_t groups = ceil_div(n, R), nchunk = ceil_div(k, 16), resident = (int64_t)sm_count * 32;
    int s = 1;
    while (s < WARPS && groups * tokens * 2 * s <= resident && nchunk / (2 * s) >= 32) s *= 2;
    return s;
}

cudaError_t launch_s8_gemv(const S8GemmParams& p, cudaStream_t st) {
    if (p.tiles_m < 1 || p.tiles_m > 65535 || p.tile_rows != 1) return cudaErrorInvalidValue;
    const int64_t groups = ceil_div(p.epi.N, R), blocks = ceil_div(groups, WARPS / p.kslices);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 1 << 30 ? blocks : 1 << 30), (unsigned)p.tiles_m);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, s8_gemv_kernel, p);
}

}  // namespace qg
