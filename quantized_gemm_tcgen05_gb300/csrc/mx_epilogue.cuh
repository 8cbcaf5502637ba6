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

// x * Phi(x) of two values for a 16-bit D.  erf(z) = z P(y), y = z^2, with P the
// Chebyshev interpolant of degree 15 of erf(sqrt y) / sqrt y on [0, 3.9^2] in
// u = 2 y / 3.9^2 - 1 (beyond, erf is 1 to 4e-8), all in fp32: |error| <= 1.5e-7 |x|,
// where erff's 1 + erf leaves 6e-8 |x|.  Twenty packed operations for two values
// against some thirty apiece: with erff the epilogue held the next tile's main
// loop up for two thirds of its own length.
__device__ __forceinline__ uint64_t mx_gelu2(uint64_t x) {
    constexpr float c[16] = {-8.173368988e-04f, 1.944994321e-03f, -1.153882593e-03f, 1.828000415e-03f,
                             -7.548484486e-03f, 1.368475612e-02f, -1.924535446e-02f, 2.906646766e-02f,
                             -4.289200157e-02f, 5.792884529e-02f, -7.378227264e-02f, 9.066636860e-02f,
                             -1.095340773e-01f, 1.346912831e-01f, -1.810110509e-01f, 3.625839651e-01f};
    constexpr float top = 3.9f;
    float a, b;
    unpack2(mul2(x, pack2(0.70710678118654752f, 0.70710678118654752f)), a, b);
    const uint64_t z = pack2(fminf(fmaxf(a, -top), top), fminf(fmaxf(b, -top), top));
    const uint64_t u = fma2(mul2(z, z), pack2(2.0f / (top * top), 2.0f / (top * top)), pack2(-1.0f, -1.0f));
    uint64_t r = pack2(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) r = fma2(r, u, pack2(c[i], c[i]));
    const uint64_t h = mul2(x, pack2(0.5f, 0.5f));
    return fma2(h, mul2(r, z), h);  // NaN stays NaN through h
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
            if constexpr (ACT == 2) {
                const uint64_t a2 = pack2(ar.alpha, ar.alpha);
                unpack2(mx_gelu2(fma2(a2, pack2(v[c][2 * j], v[c][2 * j + 1]), pack2(b0, b1))), x0, x1);
            } else {
                x0 = epi_value<ACT>(ar, v[c][2 * j], 0.0f, b0);
                x1 = epi_value<ACT>(ar, v[c][2 * j + 1], 0.0f, b1);
            }
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
            for (int t = 0; t < PER; ++t) {
                const float b = ACT >= 0 ? __shfl_sync(0xFFFFFFFFu, bl, PER * q + t) : 0.0f;
                // (GELU of a 16-bit D: below, two values at a time)
                x[t] = epi_value<ACT == 2 && DT != DT_F32 ? 0 : ACT>(ar, v[PER * q + t], cv[t], b);
            }
            if constexpr (ACT == 2 && DT != DT_F32) {
#pragma unroll
                for (int t = 0; t < PER; t += 2) unpack2(mx_gelu2(pack2(x[t], x[t + 1])), x[t], x[t + 1]);
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
        for (int r = 0; r < 32; ++r)
            if (r < rows) st_elem(e.D, DT, (m0 + r) * e.ldd + n, epi_value<ACT>(ar, stage[r * 33 + lane], c[r], b));
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

// Warp-wide: block b (of `bm` rows, a multiple of 128) of rows sorted by
// expert -> expert, its first row, its rows (those below M, the rows there are),
// and the scale atom row it starts on.  Returns false past the last block.
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
