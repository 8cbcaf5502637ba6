// Device pieces of 4-bit microscaled quantisation: a thread holds 16
// consecutive values of a row (one NVFP4 block, half an MXFP4 block).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "mx_params.h"
#include "mx_rows.h"

namespace qg {

// ---- rows that start anywhere -----------------------------------------------
//
// A lane's 16 values are W words (W = 4, 8 or 16) of a row that need not start on
// a 16-byte boundary; the boundary's distance is the same for every lane of the
// warp.  Loads take the 16-byte granules that hold the words and shift; stores
// shift the warp's words onto the granules, every lane completing its last one
// from its neighbour.  Element by element instead, a warp's accesses touch each
// sector sixteen times.

// out = the W words that start `bytes` (0 .. 15, the same in every lane) into c.
template <int W>
__device__ __forceinline__ void mx_shift_words(uint32_t (&c)[W + 4], int bytes, uint32_t (&out)[W]) {
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < W + 3; ++i) c[i] = c[i + 1];
    }
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < W + 2; ++i) c[i] = c[i + 2];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = __funnelshift_r(c[i], c[i + 1], (bytes & 3) * 8);
}

// Whether the granules that hold [p, p + bytes) lie inside [lo, hi).
__device__ __forceinline__ bool mx_granules_inside(const void* p, int bytes, const void* lo, const void* hi) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), first = a & ~uintptr_t(15), last = (a + bytes + 15) & ~uintptr_t(15);
    return first >= reinterpret_cast<uintptr_t>(lo) && last <= reinterpret_cast<uintptr_t>(hi);
}

// W words from p (granules inside the tensor).
template <int W>
__device__ __forceinline__ void mx_load_words(const void* p, uint32_t (&out)[W]) {
    const int o = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - o);
    uint32_t c[W + 4];
#pragma unroll
    for (int i = 0; i < W / 4 + 1; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i < W / 4 || o) u = g[i];
        c[4 * i] = u.x;
        c[4 * i + 1] = u.y;
        c[4 * i + 2] = u.z;
        c[4 * i + 3] = u.w;
    }
    mx_shift_words<W>(c, o, out);
}

// Warp-wide: every lane with `mine` stores its W words at p, lanes' words one after
// another; the lanes with `mine` are the first ones of the warp.  T: the element
// (p is aligned to it), by which the ends of the warp's run are stored.
template <typename T, int W>
__device__ __forceinline__ void mx_store_words(void* p, const uint32_t (&w)[W], bool mine, int lane) {
    const int o = (int)(reinterpret_cast<uintptr_t>(p) & 15), a = (16 - o) & 15;  // bytes up to the first boundary
    uint32_t c[W + 4], out[W];
#pragma unroll
    for (int i = 0; i < W; ++i) c[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[W + i] = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
    const bool next = __shfl_down_sync(0xFFFFFFFFu, mine ? 1 : 0, 1) && lane < 31;
    if (!mine) return;
    mx_shift_words<W>(c, a, out);
    uint4* g = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) + a);
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
        if (i < W / 4 - 1 || next || a == 0) g[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    if (a == 0) return;
    constexpr int ES = (int)sizeof(T), PER = 4 / ES;  // elements of a word
    auto element = [&](int i) {
        uint32_t v = 0;
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (k == i / PER) v = w[k];
        return (T)(v >> (8 * ES * (i % PER)));
    };
    T* e = static_cast<T*>(p);
    if (lane == 0)  // up to the first boundary of the run
        for (int i = 0; i < a / ES; ++i) e[i] = element(i);
    if (!next)  // past its last one
        for (int i = (4 * W - o) / ES; i < 4 * W / ES; ++i) e[i] = element(i);
}

// Sixteen values as eight packed pairs.
struct Row16 {
    uint64_t p[8];
};

// 16 bytes of T: 16 / sizeof(T) values, as pairs.
template <typename T>
struct MxIn;
template <>
struct MxIn<float> {
    using Bits = uint32_t;
    static constexpr int LOADS = 4;
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ void st(float* p, float x) { *p = x; }
    static __device__ __forceinline__ void unpack(const uint4& w, uint64_t* v) {
        v[0] = pack2(__uint_as_float(w.x), __uint_as_float(w.y));
        v[1] = pack2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t* v) {
        float f[4];
        unpack2(v[0], f[0], f[1]);
        unpack2(v[1], f[2], f[3]);
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct MxIn<__half> {
    using Bits = uint16_t;
    static constexpr int LOADS = 2;
    static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ void st(__half* p, float x) { *p = __float2half_rn(x); }
    static __device__ __forceinline__ void unpack(const uint4& w, uint64_t* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[i] = pack2(f.x, f.y);
        }
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(v[i], a, b);
            const __half2 h = __floats2half2_rn(a, b);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct MxIn<__nv_bfloat16> {
    using Bits = uint16_t;
    static constexpr int LOADS = 2;
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void unpack(const uint4& w, uint64_t* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(v[i], a, b);
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// The bits of sixteen values of a row, as 16-byte words.
template <typename T>
struct Raw16 {
    uint4 w[MxIn<T>::LOADS];
};

// Sixteen values of a row from column c0 on; zero past `cols`.  Plain loads:
// the residual norm may write where it read.  vec: 2 rows 32-byte aligned, one
// 32-byte load a half of two (every request then covers whole sectors), 1 rows
// 16-byte aligned, 0 neither.
// lo, hi: the tensor's bytes.  ALIGNED: vec is known not to be 0.
template <bool ALIGNED, typename T>
__device__ __forceinline__ Raw16<T> mx_load16(const T* row, int c0, int cols, int vec, const void* lo, const void* hi) {
    Raw16<T> r;
    if (!ALIGNED && !vec && c0 + 16 <= cols && mx_granules_inside(row + c0, 16 * (int)sizeof(T), lo, hi)) {
        mx_load_words<4 * MxIn<T>::LOADS>(row + c0, reinterpret_cast<uint32_t(&)[4 * MxIn<T>::LOADS]>(r.w));
    } else if ((ALIGNED || vec) && c0 + 16 <= cols) {
        if (vec == 2) {
#pragma unroll
            for (int i = 0; i < MxIn<T>::LOADS; i += 2) {
                uint4 &a = r.w[i], &b = r.w[i + 1];
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                             : "l"(reinterpret_cast<const uint4*>(row + c0) + i)
                             : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < MxIn<T>::LOADS; ++i) r.w[i] = *(reinterpret_cast<const uint4*>(row + c0) + i);
        }
    } else {
        uint64_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = pack2(c0 + 2 * i < cols ? MxIn<T>::one(row + c0 + 2 * i) : 0.0f,
                         c0 + 2 * i + 1 < cols ? MxIn<T>::one(row + c0 + 2 * i + 1) : 0.0f);
#pragma unroll
        for (int i = 0; i < MxIn<T>::LOADS; ++i) r.w[i] = MxIn<T>::pack(v + i * (8 / MxIn<T>::LOADS));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ Row16 mx_values(const Raw16<T>& r) {
    Row16 v;
#pragma unroll
    for (int i = 0; i < MxIn<T>::LOADS; ++i) MxIn<T>::unpack(r.w[i], v.p + i * (8 / MxIn<T>::LOADS));
    return v;
}

// Rounded to T.
template <typename T>
__device__ __forceinline__ Raw16<T> mx_round(const Row16& v) {
    Raw16<T> r;
#pragma unroll
    for (int i = 0; i < MxIn<T>::LOADS; ++i) r.w[i] = MxIn<T>::pack(v.p + i * (8 / MxIn<T>::LOADS));
    return r;
}

// Warp-wide (lanes hold consecutive chunks of a row).
template <bool ALIGNED, typename T>
__device__ __forceinline__ void mx_store16(T* row, int c0, int cols, int vec, const Raw16<T>& r, int lane) {
    if (!ALIGNED && !vec) {
        using E = typename MxIn<T>::Bits;
        mx_store_words<E, 4 * MxIn<T>::LOADS>(row + c0, reinterpret_cast<const uint32_t(&)[4 * MxIn<T>::LOADS]>(r.w),
                                              c0 + 16 <= cols, lane);
    }
    if (c0 + 16 <= cols) {
        if (!ALIGNED && !vec) return;
        if (vec == 2) {
#pragma unroll
            for (int i = 0; i < MxIn<T>::LOADS; i += 2) {
                const uint4 &a = r.w[i], &b = r.w[i + 1];
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                 reinterpret_cast<uint4*>(row + c0) + i),
                             "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                             : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < MxIn<T>::LOADS; ++i) *(reinterpret_cast<uint4*>(row + c0) + i) = r.w[i];
        }
    } else {
        const Row16 v = mx_values<T>(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, b;
            unpack2(v.p[i], a, b);
            if (c0 + 2 * i < cols) MxIn<T>::st(row + c0 + 2 * i, a);
            if (c0 + 2 * i + 1 < cols) MxIn<T>::st(row + c0 + 2 * i + 1, b);
        }
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

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN when either is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Largest magnitude of 16 values; NaN when one of them is.
__device__ __forceinline__ float mx_amax16(const Row16& v) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        unpack2(v.p[i], a, b);
        m[i] = max_nan(fabsf(a), fabsf(b));
    }
    return max_nan(max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3])), max_nan(max_nan(m[4], m[5]), max_nan(m[6], m[7])));
}

// One thread's 16 values to codes; returns the block's scale byte.  Every lane
// of the warp takes part (MXFP4 blocks span an even lane and the next one).
//
// NVFP4's quotients x / u, u = s g, and amax / (6 g): with r = RN(1/u), q0 = RN(x r)
// and the exact remainder e = u q0 - x, RN(q0 - e r) is the correctly rounded
// quotient (Markstein's theorem), so a quotient that lies on a tie of the 4-bit
// grid is found there.  Here x is -v and the codes' signs are turned at the end:
// no operand has to be negated, three packed operations do two values, and a
// zero keeps its sign.  MXFP4's quotient is a product with a power of two.
template <bool NVF4>
__device__ __forceinline__ uint32_t mx_quantize16(const Row16& v, const MxScaleConst& c, uint2& codes) {
    float amax = mx_amax16(v);
    if constexpr (!NVF4) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    const bool fine = amax < __uint_as_float(0x7F800000u);  // false for NaN
    float w[16];
    if constexpr (NVF4) {
        const float t0 = amax * c.inv_six_g;
        // far above the largest scale the quotient's last bit does not matter
        // (and its remainder may overflow)
        const float t = t0 < 1024.0f ? fmaf(fmaf(t0, c.six_g, -amax), -c.inv_six_g, t0) : 448.0f;
        const uint32_t byte = mx_e4m3_byte(fminf(t, 448.0f));
        const float u = mx_e4m3_value(byte) * c.g;
        const float nr = -__frcp_rn(u);
        if (byte == 0x7Eu) {  // the scale stands at its largest: the quotient may be anything, up to infinity
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a, b;
                unpack2(v.p[i], a, b);
                w[2 * i] = __fdiv_rn(-a, u);
                w[2 * i + 1] = __fdiv_rn(-b, u);
            }
        } else {
            const uint64_t nr2 = pack2(nr, nr), u2 = pack2(u, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t q0 = mul2(v.p[i], nr2);
                unpack2(fma2(fma2(q0, u2, v.p[i]), nr2, q0), w[2 * i], w[2 * i + 1]);
            }
        }
        const bool live = fine && byte != 0;  // u = 0: no reciprocal, no codes
        codes = make_uint2(live ? mx_codes8(w) ^ 0x88888888u : 0u, live ? mx_codes8(w + 8) ^ 0x88888888u : 0u);
        return fine ? byte : 0x7Fu;
    } else {
        const int e = (int)(__float_as_uint(amax) >> 23) - 2;
        const uint32_t byte = e > 0 ? (uint32_t)e : 0u;
        const float r = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
        const uint64_t r2 = pack2(r, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) unpack2(mul2(v.p[i], r2), w[2 * i], w[2 * i + 1]);
        codes = make_uint2(fine ? mx_codes8(w) : 0u, fine ? mx_codes8(w + 8) : 0u);
        return fine ? byte : 0xFFu;
    }
}

// Store a thread's codes: 8 bytes, or what of them lies before the row's end.
__device__ __forceinline__ void mx_store_codes(uint8_t* row, int c0, int cols, const uint2& codes) {
    if (c0 + 16 <= cols) {
        *reinterpret_cast<uint2*>(row + c0 / 2) = codes;
    } else if (c0 < cols) {
        const int n = (cols - c0 + 1) / 2;  // codes past the row's end are zero
        for (int i = 0; i < 8; ++i)
            if (i < n) row[c0 / 2 + i] = (uint8_t)((i < 4 ? codes.x >> (8 * i) : codes.y >> (8 * i - 32)) & 0xFFu);
    }
}

// Byte of row srow's first scale; block b's lies mx_block_at(b) further.
__device__ __forceinline__ int64_t mx_scale_row_at(int64_t srow, int atoms) {
    const uint32_t in = (uint32_t)srow % MX_ATOM_ROWS;
    return (int64_t)((uint32_t)srow / MX_ATOM_ROWS) * atoms * MX_ATOM_BYTES + in % 32 * 16 + in / 32 * 4;
}
__device__ __forceinline__ int64_t mx_block_at(int b) { return (int64_t)(b / 4) * MX_ATOM_BYTES + b % 4; }

// Store the scales of the warp's blocks, four blocks (one row's share of an
// atom) per store.  S: the row's first scale.  chunk: this lane's 16-value chunk;
// lanes hold consecutive chunks of one row, the warp's first a multiple of 8;
// chunks at or past chunk_end are not stored, blocks past the row's end are
// padding: zero, whatever an empty block's scale would be.
template <bool NVF4>
__device__ __forceinline__ void mx_store_scales(uint8_t* S, int chunk, int chunk_end, int cols, uint32_t byte, int lane) {
    constexpr int PER = NVF4 ? 1 : 2;  // lanes per block
    if (chunk / PER * (16 * PER) >= cols) byte = 0;
    uint32_t w = byte;
    w |= __shfl_down_sync(0xFFFFFFFFu, byte, PER) << 8;
    const uint32_t hi = __shfl_down_sync(0xFFFFFFFFu, w, 2 * PER);
    w = (w & 0xFFFFu) | (hi << 16);
    if (lane % (4 * PER) == 0 && chunk < chunk_end) *reinterpret_cast<uint32_t*>(S + mx_block_at(chunk / PER)) = w;
}

// Rows lo .. hi - 1 of one expert, and the scale row of the first (an expert
// starts on an atom row).  Offsets that are no partition of the rows cannot lead
// past the scales: a span ends with the `rows` / 128 + E atom rows (mx_span_end).
struct MxExpertSpan {
    int64_t lo, hi, row0;
    __device__ __forceinline__ bool holds(int64_t r) const { return r >= lo && r < hi; }
};

// Warp-wide: the expert that holds row r of rows sorted by expert; a span without
// it when none does, or when it has no scales.
__device__ __forceinline__ MxExpertSpan mx_expert_of(const int32_t* off, int32_t E, int64_t rows, int64_t r, int lane) {
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
        if (hit) {
            const int64_t at = __shfl_sync(0xFFFFFFFFu, lo, first), end = __shfl_sync(0xFFFFFFFFu, hi, first);
            return MxExpertSpan{at, mx_span_end(at, end, tiles, rows, E), tiles * MX_ATOM_ROWS};
        }
    }
    return MxExpertSpan{0, 0, 0};
}

}  // namespace qg
