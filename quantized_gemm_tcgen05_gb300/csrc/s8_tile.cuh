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

// Registers of a thread from here on, for whole groups of four warps.
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t* v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Half of a stage (64 codes of 128 channels and of `rows` tokens, a multiple of 16, at
// most 8 * OCTETS; 128-byte rows of 128 codes, swizzled) to f16: the channels' into 32
// TMEM columns, the tokens' into a swizzled operand tile.  A group of 128 threads: a
// thread has a channel, and with seven others eight tokens' chunks of 16 codes, so that
// neither side has bank conflicts.
// Codes are loaded just before their conversion, or all of them early (load), which takes
// registers: the CTA-pair kernel gains 4 us of 114 by it (4096^3), the one-tile kernel
// loses 10% where they spill.
template <int OCTETS>
struct HalfStage {
    static constexpr int N = (OCTETS + 3) / 4;
    uint4 w[4], x[N];
    uint32_t w_at, x_at, out_at;  // offsets in the stage and in the tile
    int octet;
    __device__ __forceinline__ HalfStage(int half, int row, int thread) {
        const int r8 = thread & 7, c = thread >> 3 & 3;
        octet = thread >> 5;  // ... and every fourth one after it
        w_at = (uint32_t)(row * 128 + (((4 * half) ^ (row & 7)) << 4));
        x_at = (uint32_t)((octet * 8 + r8) * 128 + (((4 * half + c) ^ r8) << 4));
        out_at = (uint32_t)((octet * 8 + r8) * 128 + (((2 * c) ^ r8) << 4));
    }
    // Shared-memory addresses of a stage's two tiles, and of the tokens' tile.
    __device__ __forceinline__ void load(uint32_t wraw, uint32_t xraw, int rows) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = lds128((wraw + w_at) ^ (c << 4));
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (octet + 4 * k < rows / 8) x[k] = lds128(xraw + x_at + 4096 * k);
    }
    __device__ __forceinline__ void store(uint32_t taddr, uint32_t out, int rows) const {
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            uint32_t r[16];
            s8_to_f16(w[c], r);
            s8_to_f16(w[c + 1], r + 8);
            tmem_st_32x32b(taddr + 8 * c, r);
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (octet + 4 * k < rows / 8) put(x[k], out + out_at + 4096 * k);
    }
    // Both, piece by piece; flip: 64 for the stage's other half.
    __device__ __forceinline__ void convert(uint32_t wraw, uint32_t xraw, uint32_t taddr, uint32_t out, int rows, uint32_t flip) const {
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = lds128((wraw + w_at) ^ (flip | c << 4));
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            uint32_t r[16];
            s8_to_f16(v[c], r);
            s8_to_f16(v[c + 1], r + 8);
            tmem_st_32x32b(taddr + 8 * c, r);
        }
#pragma unroll
        for (int k = 0; k < N; k += 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (k + q < N && octet + 4 * (k + q) < rows / 8) v[q] = lds128((xraw + x_at + 4096 * (k + q)) ^ flip);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (k + q < N && octet + 4 * (k + q) < rows / 8) put(v[q], out + out_at + 4096 * (k + q));
        }
    }
    static __device__ __forceinline__ void put(const uint4& codes, uint32_t to) {
        uint32_t h[8];
        s8_to_f16(codes, h);
        sts128(to, h);
        sts128(to ^ 16u, h + 4);
    }
};

// Four channels n .. n + 3: their factors and biases.
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
// Their values of token m, whose factor is `token`, and their store.
__device__ __forceinline__ void s8_finish4(const S8GemmParams& P, const EpiArith& ar, const S8Channels& ch, float token, int64_t m, int64_t n,
                                           const int4& sum) {
    const EpiParams& e = P.epi;
    const int have = e.N - n < 4 ? (int)(e.N - n) : 4;
    if (have <= 0 || !mx_block_in_bounds(e, m, 1, n, have)) return;
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
