// Device pieces of the int8 products on the tensor cores.
//
// This GPU's tensor cores have no integer products to speak of, but every int8
// value is an f16 value, every product of two is exact in fp32, and so are sums of
// up to 1024 products (2^10 * 2^14 = 2^24).  The codes become f16 on their way:
// B's (the weights: the MMA's 128 rows) from shared memory into TMEM, which feeds the
// MMA's first operand and spares shared memory a write and a read of twice the bytes, A's
// (the tokens: the MMA's columns) back into shared memory.  After every 1024 of K
// the accumulator is converted and added to 32-bit integers, so sums are exact.
#pragma once
#include "s8_epilogue.cuh"

namespace qg {

// Sixteen codes to f16, in order: a byte b + 128 under the exponent of 1024 is the
// f16 value 1152 + b, and the difference to 1152 is exact.
__device__ __forceinline__ uint32_t s8_pair_f16(uint32_t biased, uint32_t select) {
    const uint32_t h = __byte_perm(biased, 0x64646464u, select);
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void s8_to_f16(const uint4& codes, uint32_t* out) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = w[i] ^ 0x80808080u;
        out[2 * i] = s8_pair_f16(b, 0x4140);
        out[2 * i + 1] = s8_pair_f16(b, 0x4342);
    }
}

// 128 rows of 128 codes (swizzled) to 64 TMEM columns of f16 pairs; a warp has the
// rows of its 32-lane quarter.  `taddr` includes the quarter's lane.
__device__ __forceinline__ void s8_weights_to_tmem(const uint8_t* raw, uint32_t taddr, int row) {
    const uint8_t* base = raw + row * 128;
    const int x = row & 7;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) s8_to_f16(*reinterpret_cast<const uint4*>(base + (((4 * half + c) ^ x) << 4)), r + 8 * c);
        tmem_st_32x32b(taddr + 32 * half, r);
    }
}

// `rows` rows (a multiple of 8) of 128 codes (swizzled) to two f16 operand tiles of
// 64 columns (swizzled), rows * 128 bytes each.  128 threads, eight rows of a
// 16-code chunk to eight threads: neither side has bank conflicts.
__device__ __forceinline__ void s8_tokens_to_f16(const uint8_t* raw, uint8_t* out, int rows, int thread) {
    const int r8 = thread & 7;
    for (int i = thread >> 3; i < rows; i += 16) {  // (eight chunks of rows / 8 octets)
        const int c = i & 7, row = (i >> 3) * 8 + r8;
        uint32_t h[8];
        s8_to_f16(*reinterpret_cast<const uint4*>(raw + row * 128 + ((c ^ r8) << 4)), h);
        uint8_t* tile = out + (c >> 2) * rows * 128 + row * 128;
        const int d = 2 * (c & 3);
        *reinterpret_cast<uint4*>(tile + ((d ^ r8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(tile + (((d + 1) ^ r8) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
}

// Four channels n .. n + 3 of one token: the values, and their store.
struct S8Channels {
    float scale[4], bias[4];
};
__device__ __forceinline__ S8Channels s8_channels(const S8GemmParams& P, const EpiArith& ar, int64_t expert, int64_t n) {
    S8Channels c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c.scale[j] = n + j < P.epi.N ? s8_channel_factor(P, expert, n + j) : 0.0f;
        c.bias[j] = bias_at(ar, n + j);
    }
    return c;
}
__device__ __forceinline__ void s8_finish4(const S8GemmParams& P, const EpiArith& ar, const S8Channels& ch, int64_t m, int64_t n, const int4& sum) {
    const EpiParams& e = P.epi;
    const int have = e.N - n < 4 ? (int)(e.N - n) : 4;
    if (have <= 0 || !mx_block_in_bounds(e, m, 1, n, have)) return;
    const float token = s8_token_factor(P, m);
    const int32_t s[4] = {sum.x, sum.y, sum.z, sum.w};
    float v[4], c[4] = {0.0f, 0.0f, 0.0f, 0.0f}, x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = s8_scaled(s[j], token, ch.scale[j]);
    if (ar.beta != 0.0f) {
        if (P.vec4 && have == 4) {
            const float4 f = ld4(e.C, e.d_type, m * e.ldc + n);
            c[0] = f.x, c[1] = f.y, c[2] = f.z, c[3] = f.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < have) c[j] = ld_elem(e.C, e.d_type, m * e.ldc + n + j);
        }
    }
    with_epi_act(e, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        mx_value2_any<ACT>(ar, e.d_type, v[0], v[1], c[0], c[1], ch.bias[0], ch.bias[1], x[0], x[1]);
        mx_value2_any<ACT>(ar, e.d_type, v[2], v[3], c[2], c[3], ch.bias[2], ch.bias[3], x[2], x[3]);
    });
    if (P.vec4 && have == 4) {
        st4(e.D, e.d_type, m * e.ldd + n, make_float4(x[0], x[1], x[2], x[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < have) st_elem(e.D, e.d_type, m * e.ldd + n + j, x[j]);
    }
}

}  // namespace qg
