// Device pieces of 4-bit microscaled quantisation: a thread holds 16
// consecutive values of a row (one NVFP4 block, half an MXFP4 block).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx_params.h"

namespace qg {

// 16 bytes of T per load.
template <typename T>
struct MxIn;
template <>
struct MxIn<float> {
    static constexpr int LOADS = 4;
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
        v[0] = __uint_as_float(w.x);
        v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z);
        v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float round(float x) { return x; }
    static __device__ __forceinline__ void st(float* p, float x) { *p = x; }
    static __device__ __forceinline__ uint4 pack(const float* v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct MxIn<__half> {
    static constexpr int LOADS = 2;
    static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float round(float x) { return __half2float(__float2half_rn(x)); }
    static __device__ __forceinline__ void st(__half* p, float x) { *p = __float2half_rn(x); }
    static __device__ __forceinline__ uint4 pack(const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct MxIn<__nv_bfloat16> {
    static constexpr int LOADS = 2;
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
    static __device__ __forceinline__ uint4 pack(const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// Sixteen values of a row from column c0 on; zero past `cols`.  Plain loads:
// the residual norm may write where it read.
template <typename T>
__device__ __forceinline__ void mx_load16(const T* row, int64_t c0, int64_t cols, bool vec, float (&v)[16]) {
    if (vec && c0 + 16 <= cols) {
        uint4 w[MxIn<T>::LOADS];
#pragma unroll
        for (int i = 0; i < MxIn<T>::LOADS; ++i) w[i] = *(reinterpret_cast<const uint4*>(row + c0) + i);
#pragma unroll
        for (int i = 0; i < MxIn<T>::LOADS; ++i) MxIn<T>::unpack(w[i], v + i * (16 / MxIn<T>::LOADS));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = c0 + i < cols ? MxIn<T>::one(row + c0 + i) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void mx_store16(T* row, int64_t c0, int64_t cols, bool vec, const float (&v)[16]) {
    if (vec && c0 + 16 <= cols) {
#pragma unroll
        for (int i = 0; i < MxIn<T>::LOADS; ++i)
            *(reinterpret_cast<uint4*>(row + c0) + i) = MxIn<T>::pack(v + i * (16 / MxIn<T>::LOADS));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c0 + i < cols) MxIn<T>::st(row + c0 + i, v[i]);
    }
}

// Eight values to eight codes, value 0 in bits 3:0: nearest, ties to even, magnitudes
// above 6 to 6.
__device__ __forceinline__ uint32_t mx_codes8(const float* w) {
    uint32_t r;
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
        "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
        : "=r"(r)
        : "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "f"(w[4]), "f"(w[5]), "f"(w[6]), "f"(w[7]));
    return r;
}

__device__ __forceinline__ uint32_t mx_e4m3_byte(float t) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(t));
    return r & 0xFFu;
}

__device__ __forceinline__ float mx_e4m3_value(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
    return __half2float(__ushort_as_half((uint16_t)(h & 0xFFFFu)));
}

// Value of a scale byte (NaN for the formats' NaN patterns).
template <bool NVF4>
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
    if constexpr (NVF4) return mx_e4m3_value(byte);
    return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// One thread's 16 values to codes; returns the block's scale byte.  Every lane
// of the warp takes part (MXFP4 blocks span an even lane and the next one).
// NVFP4's quotient x / u, u = s g: with r = RN(1/u), q0 = RN(x r) and the exact
// remainder q0 u - x, RN(q0 - remainder * r) is the correctly rounded quotient
// (Markstein's theorem), so a quotient that lies on a tie of the 4-bit grid is
// found there (and -0 stays -0 with these signs).  MXFP4's is a product with a power of two, exact.
template <bool NVF4>
__device__ __forceinline__ uint32_t mx_quantize16(const float (&v)[16], float g, float six_g, uint2& codes) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // magnitudes order as integers, NaN above infinity
        const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        amax = a > amax ? a : amax;
    }
    if constexpr (!NVF4) {
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, amax, 1);
        amax = o > amax ? o : amax;
    }
    const bool fine = amax < 0x7F800000u;
    float w[16];
    uint32_t byte;
    if constexpr (NVF4) {
        byte = mx_e4m3_byte(fminf(__fdiv_rn(__uint_as_float(amax), six_g), 448.0f));
        const float u = mx_e4m3_value(byte) * g;
        const bool live = fine && u > 0.0f;
        const float r = live ? __frcp_rn(u) : 0.0f;
        const float m = live ? u : 0.0f;
        if (byte == 0x7Eu) {  // the scale stands at its largest: the quotient may be anything, up to infinity
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = live ? __fdiv_rn(v[i], u) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = live ? v[i] : 0.0f;
                const float q0 = x * r;
                w[i] = fmaf(fmaf(q0, m, -x), -r, q0);
            }
        }
        if (!fine) byte = 0x7Fu;
    } else {
        const int e = (int)(amax >> 23) - 2;
        byte = e > 0 ? (uint32_t)e : 0u;
        const float r = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = fine ? v[i] * r : 0.0f;
        if (!fine) byte = 0xFFu;
    }
    codes = make_uint2(mx_codes8(w), mx_codes8(w + 8));
    return byte;
}

// Store a thread's codes: 8 bytes, or what of them lies before the row's end.
__device__ __forceinline__ void mx_store_codes(uint8_t* row, int64_t c0, int64_t cols, const uint2& codes) {
    if (c0 + 16 <= cols) {
        *reinterpret_cast<uint2*>(row + c0 / 2) = codes;
    } else if (c0 < cols) {
        const int64_t n = (cols - c0 + 1) / 2;  // codes past the row's end are zero
        for (int i = 0; i < 8; ++i)
            if (i < n) row[c0 / 2 + i] = (uint8_t)((i < 4 ? codes.x >> (8 * i) : codes.y >> (8 * i - 32)) & 0xFFu);
    }
}

// Store the scales of the warp's blocks, four blocks (one row's share of an
// atom) per store.  chunk: this lane's 16-value chunk; lanes hold consecutive
// chunks of one row, the warp's first a multiple of 8; chunks at or past
// chunk_end are not stored.  srow: the scale row.
template <bool NVF4>
__device__ __forceinline__ void mx_store_scales(uint8_t* S, int64_t srow, int64_t chunk, int64_t chunk_end,
                                                int64_t atoms, uint32_t byte, int lane) {
    constexpr int PER = NVF4 ? 1 : 2;  // lanes per block
    uint32_t w = byte;
    w |= __shfl_down_sync(0xFFFFFFFFu, byte, PER) << 8;
    const uint32_t hi = __shfl_down_sync(0xFFFFFFFFu, w, 2 * PER);
    w = (w & 0xFFFFu) | (hi << 16);
    if (lane % (4 * PER) == 0 && chunk < chunk_end)
        *reinterpret_cast<uint32_t*>(S + mx_scale_at(srow, chunk / PER, atoms)) = w;
}

// Warp-wide: the scale row of token row r when rows are sorted by expert (each
// expert starts on an atom row), or -1 when no expert holds it.
__device__ __forceinline__ int64_t mx_expert_row(const int32_t* off, int32_t E, int64_t r, int lane) {
    int64_t tiles = 0;
    for (int32_t e0 = 0; e0 < E; e0 += 32) {
        const int32_t e = e0 + lane;
        const int64_t lo = e < E ? off[e] : 0, hi = e < E ? off[e + 1] : 0;
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, e < E && r >= lo && r < hi);
        int32_t n = hi > lo ? (int32_t)((hi - lo + 127) / 128) : 0;
        const int first = hit ? __ffs((int)hit) - 1 : 32;
        if (lane >= first) n = 0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
        tiles += n;
        if (hit) return tiles * MX_ATOM_ROWS + (r - __shfl_sync(0xFFFFFFFFu, lo, first));
    }
    return -1;
}

}  // namespace qg
