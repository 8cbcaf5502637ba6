// Epilogue pieces of the 4-bit microscaled products: 32 accumulator columns of
// one row, held by one thread, to D.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"
#include "mx_gemm.h"

namespace qg {

// Checked build: rows m0 .. + rows - 1, columns n0 .. + cols - 1 inside D (and C).
__device__ __forceinline__ bool mx_block_in_bounds(const EpiParams& e, int64_t m0, int rows, int64_t n0, int64_t cols) {
    if (!elem_in_bounds(e, m0 * e.ldd + n0, (rows - 1) * e.ldd + cols, e.d_extent)) return false;
    return e.beta == 0.0f || elem_in_bounds(e, m0 * e.ldc + n0, (rows - 1) * e.ldc + cols, e.c_extent);
}

// 32-byte global accesses: a whole sector per lane.
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Bring `count` columns of C's row m, from n on, into L2 before they are needed.
__device__ __forceinline__ void mx_prefetch_c(const EpiParams& e, int64_t m, int64_t n, int64_t count) {
    const int64_t es = e.d_type == DT_F32 ? 4 : 2;
    const char* p = static_cast<const char*>(e.C) + (m * e.ldc + n) * es;
    for (int64_t b = 0; b < count * es; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + b));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + count * es - es));
}

// x * Phi(x) of two values for a 16-bit D, as max(x, 0) - w Q(w) with w = |x| and
// Q the upper tail of the normal distribution, Q(w) = exp(-w^2 / 2) M(w).  M is a
// polynomial of degree 7 in 1 / (1 + 0.35 w), fitted for the least relative error on
// [0, 13.5] (2.9e-7); further out exp(-w^2 / 2) is below fp32's normal numbers and
// the tail is 0.  With the approximate exponential and reciprocal the result is
// within 4e-6 of x Phi(x), relative, for x >= -6, and within 2e-5 down to -13.
// 0.5 x (1 + erf), which cancels for negative x, leaves 1e-7 |x| instead, a few
// parts in a hundred at -5: of 8192 values from -13 to 13 it rounds 1391 to another
// bf16 than the nearest, this none.  22 operations for two values, four of them in
// the special function unit, against thirty apiece with erff: 4096x14336x4096 with
// GELU takes 112 us to bf16 (NVFP4) and 105 to f16 (MXFP4), with erff 144 and 146.
__device__ __forceinline__ uint64_t mx_gelu2(uint64_t x) {
    constexpr float c[8] = {-4.887409466e-02f, 2.018410696e-01f, -2.401753938e-01f, 1.661134462e-02f,
                            -1.557545603e-01f, -1.334135110e-01f, -1.402618247e-01f, 2.682103994e-05f};
    float x0, x1;
    unpack2(x, x0, x1);
    const uint64_t w = pack2(fminf(fabsf(x0), 16.0f), fminf(fabsf(x1), 16.0f));
    float d0, d1, e0, e1;
    unpack2(fma2(w, pack2(0.35f, 0.35f), pack2(1.0f, 1.0f)), d0, d1);
    const uint64_t t = pack2(rcp_approx(d0), rcp_approx(d1));
    unpack2(mul2(mul2(w, w), pack2(-0.72134752044f, -0.72134752044f)), e0, e1);  // -log2(e) / 2
    const uint64_t e = pack2(ex2_approx(e0), ex2_approx(e1));
    uint64_t m = pack2(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fma2(m, t, pack2(c[i], c[i]));
    const uint64_t h = mul2(x, pack2(0.5f, 0.5f));
    unpack2(h, x0, x1);
    // (x + |x|) / 2: a NaN stays one, and -inf gives one, as -inf * 0 does with erff
    const uint64_t top = pack2(x0 + fabsf(x0), x1 + fabsf(x1));
    return fma2(mul2(w, e), m, top);  // m is -M
}

// Two neighbouring columns' values: alpha * acc + beta * c, then the fused steps
// of ACT with the columns' biases.  Every form of the epilogue takes them from
// here, each step rounded by itself, so that a value does not depend on where in
// D its column lies, on D's alignment or on which kernel wrote it.
template <int ACT, int DT>
__device__ __forceinline__ void mx_value2(const EpiArith& e, float a0, float a1, float c0, float c1, float b0, float b1,
                                          float& x0, float& x1) {
    x0 = e.beta != 0.0f ? fmaf(e.alpha, a0, e.beta * c0) : __fmul_rn(e.alpha, a0);
    x1 = e.beta != 0.0f ? fmaf(e.alpha, a1, e.beta * c1) : __fmul_rn(e.alpha, a1);
    if constexpr (ACT >= 0) {
        x0 = __fadd_rn(x0, b0);
        x1 = __fadd_rn(x1, b1);
        if constexpr (ACT == 0) {
            x0 = e.relu && x0 < 0.0f ? 0.0f : x0;
            x1 = e.relu && x1 < 0.0f ? 0.0f : x1;
        } else if constexpr (DT == DT_F32) {
            x0 = 0.5f * x0 * (1.0f + erff(x0 * 0.70710678118654752f));
            x1 = 0.5f * x1 * (1.0f + erff(x1 * 0.70710678118654752f));
        } else {
            unpack2(mx_gelu2(pack2(x0, x1)), x0, x1);
        }
    }
}

// The same where D's type is known at run time only (the 16-bit types' values differ
// in the rounding to come).
template <int ACT>
__device__ __forceinline__ void mx_value2_any(const EpiArith& e, int32_t d_type, float a0, float a1, float c0, float c1,
                                              float b0, float b1, float& x0, float& x1) {
    if (ACT == 2 && d_type != DT_F32)
        mx_value2<ACT, DT_F16>(e, a0, a1, c0, c1, b0, b1, x0, x1);
    else
        mx_value2<ACT, DT_F32>(e, a0, a1, c0, c1, b0, b1, x0, x1);
}

// 64 accumulator columns (TMEM address ta, this warp's 32 rows, a row per lane).
__device__ __forceinline__ void mx_load64(uint32_t ta, float (&v)[2][32]) {
    tmem_load_chunk<32>(ta, v[0]);
    tmem_load_chunk<32>(ta + 32, v[1]);
}

// The same as finished 16-bit values: w[j] holds columns n0 + 2 j and 2 j + 1.
template <int ACT, int DT>
__device__ __forceinline__ void mx_pack64(const EpiParams& e, float alpha, const float (&v)[2][32], int64_t n0,
                                          uint32_t (&w)[32], int lane) {
    EpiArith ar = epi_arith(e);
    ar.alpha = alpha;
    ar.beta = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float bl = ACT >= 0 ? bias_at(ar, n0 + 32 * c + lane) : 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float b0 = 0.0f, b1 = 0.0f;
            if constexpr (ACT >= 0) {
                b0 = __shfl_sync(0xFFFFFFFFu, bl, 2 * j);
                b1 = __shfl_sync(0xFFFFFFFFu, bl, 2 * j + 1);
            }
            float x0, x1;
            mx_value2<ACT, DT>(ar, v[c][2 * j], v[c][2 * j + 1], 0.0f, 0.0f, b0, b1, x0, x1);
            if constexpr (DT == DT_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
                w[16 * c + j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(x0, x1);
                w[16 * c + j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
}
__device__ __forceinline__ void mx_pack64_any(const EpiParams& e, float alpha, const float (&v)[2][32], int64_t n0,
                                              uint32_t (&w)[32], int lane) {
    with_epi_act(e, [&](auto act) {
        if (e.d_type == DT_BF16)
            mx_pack64<decltype(act)::value, DT_BF16>(e, alpha, v, n0, w, lane);
        else
            mx_pack64<decltype(act)::value, DT_F16>(e, alpha, v, n0, w, lane);
    });
}

// The 64 packed columns through `stage` (32 rows of 128 bytes, 16-byte chunks
// XOR-permuted by the row): in, a row per lane; out, four lanes to a row, so
// every global request is a whole 128-byte line.  Storing the rows a lane each
// instead sends four times the requests, which cost 4096x14336x4096 19 us of
// 110.  d: row 0's first column; ld in elements; rows: rows that exist.
__device__ __forceinline__ void mx_stage64(uint8_t* stage, const uint32_t (&w)[32], int lane) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}
__device__ __forceinline__ void mx_store64(const uint8_t* stage, uint16_t* d, int64_t ld, int rows, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + lane / 4, part = lane % 4;
        const uint4 a = *reinterpret_cast<const uint4*>(stage + r * 128 + (((2 * part) ^ (r & 7)) << 4));
        const uint4 b = *reinterpret_cast<const uint4*>(stage + r * 128 + (((2 * part + 1) ^ (r & 7)) << 4));
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (r < rows) st32(d + r * ld + 16 * part, w);
    }
}

// Columns n0 .. n0+31 of row m (valid for this lane when `row_ok`), values v
// before alpha.  Every lane of the warp takes part.  Vector form: every lane
// moves its own row's 64 or 128 bytes in 32-byte pieces, whole sectors each, so
// no transposition is needed.  Otherwise (rows not 32-byte aligned, or the
// tile's last columns) the warp turns the block through `stage` (32 x 33
// floats) and each lane takes one column, row after row.
template <int ACT, int DT>
__device__ __forceinline__ void mx_store_block_t(const EpiParams& ep, bool vec32, float alpha, int64_t m0,
                                                 int rows, int64_t n0, float (&v)[32], float* stage, int lane) {
    const EpiParams e = ep;
    if (!mx_block_in_bounds(e, m0, rows, n0, e.N - n0 < 32 ? e.N - n0 : 32)) return;
    EpiArith ar = epi_arith(e);
    ar.alpha = alpha;
    const int64_t m = m0 + lane;
    const bool use_c = e.beta != 0.0f;
    if (vec32 && n0 + 32 <= e.N) {
        const float bl = ACT >= 0 ? bias_at(ar, n0 + lane) : 0.0f;
        constexpr int ES = DT == DT_F32 ? 4 : 2, PER = 32 / ES;  // elements per piece
        char* d = static_cast<char*>(e.D) + (m * e.ldd + n0) * ES;
        const char* c = static_cast<const char*>(e.C) + (m * e.ldc + n0) * ES;
        const bool ok = lane < rows;
#pragma unroll
        for (int q = 0; q < 32 / PER; ++q) {
            float cv[PER];
#pragma unroll
            for (int t = 0; t < PER; ++t) cv[t] = 0.0f;
            if (use_c && ok) {
                uint32_t w[8];
                ld32(c + 32 * q, w);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if constexpr (DT == DT_F32) {
                        cv[t] = __uint_as_float(w[t]);
                    } else {
                        const float2 f = DT == DT_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[t]))
                                                       : __half22float2(*reinterpret_cast<const __half2*>(&w[t]));
                        cv[2 * t] = f.x;
                        cv[2 * t + 1] = f.y;
                    }
                }
            }
            float x[PER];
#pragma unroll
            for (int t = 0; t < PER; t += 2) {
                float b0 = 0.0f, b1 = 0.0f;
                if constexpr (ACT >= 0) {
                    b0 = __shfl_sync(0xFFFFFFFFu, bl, PER * q + t);
                    b1 = __shfl_sync(0xFFFFFFFFu, bl, PER * q + t + 1);
                }
                mx_value2<ACT, DT>(ar, v[PER * q + t], v[PER * q + t + 1], cv[t], cv[t + 1], b0, b1, x[t], x[t + 1]);
            }
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if constexpr (DT == DT_F32) {
                    w[t] = __float_as_uint(x[t]);
                } else if constexpr (DT == DT_BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * t], x[2 * t + 1]);
                    w[t] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __half2 h = __floats2half2_rn(x[2 * t], x[2 * t + 1]);
                    w[t] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            if (ok) st32(d + 32 * q, w);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = v[j];
    __syncwarp();
    const int64_t n = n0 + lane;
    if (n < e.N) {
        const float b = ACT >= 0 ? bias_at(ar, n) : 0.0f;
        float c[32];  // every row's C in flight together
#pragma unroll
        for (int r = 0; r < 32; ++r) c[r] = use_c && r < rows ? ld_elem(e.C, DT, (m0 + r) * e.ldc + n) : 0.0f;
#pragma unroll
        for (int r = 0; r < 32; r += 2) {
            float x0, x1;
            mx_value2<ACT, DT>(ar, stage[r * 33 + lane], stage[r * 33 + 33 + lane], c[r], c[r + 1], b, b, x0, x1);
            if (r < rows) st_elem(e.D, DT, (m0 + r) * e.ldd + n, x0);
            if (r + 1 < rows) st_elem(e.D, DT, (m0 + r + 1) * e.ldd + n, x1);
        }
    }
    __syncwarp();
}

template <int DT>
__device__ __forceinline__ void mx_store_block_dt(const EpiParams& e, bool vec32, float alpha, int64_t m0, int rows,
                                                  int64_t n0, float (&v)[32], float* stage, int lane) {
    with_epi_act(e, [&](auto act) {
        mx_store_block_t<decltype(act)::value, DT>(e, vec32, alpha, m0, rows, n0, v, stage, lane);
    });
}

// rows: rows of this warp's 32 that exist (m0 .. m0 + rows - 1).
__device__ __forceinline__ void mx_store_block(const EpiParams& e, bool vec32, float alpha, int64_t m0, int rows,
                                               int64_t n0, float (&v)[32], float* stage, int lane) {
    if (e.d_type == DT_BF16)
        mx_store_block_dt<DT_BF16>(e, vec32, alpha, m0, rows, n0, v, stage, lane);
    else if (e.d_type == DT_F16)
        mx_store_block_dt<DT_F16>(e, vec32, alpha, m0, rows, n0, v, stage, lane);
    else
        mx_store_block_dt<DT_F32>(e, vec32, alpha, m0, rows, n0, v, stage, lane);
}

// Warp-wide: block b (of `bm` rows) of rows sorted by expert -> expert, its first
// row, its rows (those below M, the rows there are; 0 or fewer: none), and, for a bm
// that is a multiple of 128, the scale atom row it starts on.  Returns false past the
// last block.  Offsets that are no partition of the rows may give any expert and row
// (the sums of their blocks may wrap), but none outside 0 .. M - 1.
__device__ __forceinline__ bool mx_expert_block(const int32_t* off, int32_t E, int64_t M, int bm, int64_t b, int lane,
                                                int* expert, int64_t* row0, int* rows, int64_t* atom_row) {
    int64_t blocks = 0, tiles = 0;
    for (int32_t e0 = 0; e0 < E; e0 += 32) {
        const int32_t e = e0 + lane;
        const int64_t lo = e < E ? off[e] : 0, hi = e < E ? off[e + 1] : 0;
        const int64_t m = hi > lo ? hi - lo : 0;
        const int nb = (int)((m + bm - 1) / bm), nt = (int)((m + MX_ATOM_ROWS - 1) / MX_ATOM_ROWS);
        int pb = nb, pt = nt;  // inclusive prefix sums
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int ub = __shfl_up_sync(0xFFFFFFFFu, pb, d), ut = __shfl_up_sync(0xFFFFFFFFu, pt, d);
            if (lane >= d) {
                pb += ub;
                pt += ut;
            }
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, b < blocks + pb);
        if (hit) {
            const int l = __ffs((int)hit) - 1;
            const int64_t q = b - blocks - __shfl_sync(0xFFFFFFFFu, pb - nb, l);  // block within the expert
            const int64_t left = __shfl_sync(0xFFFFFFFFu, m, l) - q * bm;
            *expert = e0 + l;
            *row0 = __shfl_sync(0xFFFFFFFFu, lo, l) + q * bm;
            const int64_t room = M - *row0;
            *rows = *row0 < 0 || room < 0 ? 0 : (int)(left < bm ? (left < room ? left : room) : (bm < room ? bm : room));
            *atom_row = tiles + __shfl_sync(0xFFFFFFFFu, pt - nt, l) + q * (bm / MX_ATOM_ROWS);
            return true;
        }
        blocks += __shfl_sync(0xFFFFFFFFu, pb, 31);
        tiles += __shfl_sync(0xFFFFFFFFu, pt, 31);
    }
    return false;
}

}  // namespace qg
