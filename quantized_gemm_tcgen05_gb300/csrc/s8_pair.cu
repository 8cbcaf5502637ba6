// Int8 product on CTA pairs: persistent clusters of two, one tile of 256 channels x
// up to 192 tokens at a time (tcgen05.mma.cta_group::2).
//
// Each CTA takes in its 128 channels and its half of the tile's tokens, and turns
// both into f16: the channels' codes into its TMEM, the tokens' into its shared
// memory, in slots of 64 of K.  Two groups of four warps take a stage's two halves.
// The accumulator has two buffers; every 16 slots (1024 products) eight warps add the
// full one to 32-bit sums in registers, 96 of them a thread, and after the tile's
// last finish and store them, while the MMAs go on in the other buffer.
//
//   warps 0-3    TMA producer, (leader) MMAs, two without work
//   warps 4-11   sums and epilogue: a 32-lane quarter and half of the columns each
//   warps 12-27  f16 operands
// Measured (back-to-back launches, cold operands): 4096^3 116 us (1.18 PFLOP/s; the MMAs
// alone would take 68), with C 134, with GELU 130; 4096 x 14336 x 4096 370 us, 1.30
// PFLOP/s; 4096 rows by 8 experts 419. A slot takes 0.33 us of which its MMAs are 0.20; the
// rest is the chain from the slot's release to its next MMAs.
#include <atomic>

#include "mx_rows.h"
#include "s8_tile.cuh"

namespace qg {

namespace {

constexpr int THREADS = 896;
constexpr int TN = S8_PAIR_TOKENS, HALF = TN / 2;
constexpr int S = 4;   // raw stages: 128 of K
constexpr int NS = 4;  // f16 slots: 64 of K
constexpr uint32_t W_BYTES = 128 * 128, X_BYTES = HALF * 128, STAGE_BYTES = W_BYTES + X_BYTES;
constexpr uint32_t SLOT_BYTES = HALF * 128;
constexpr uint32_t RING_BYTES = S * STAGE_BYTES + NS * SLOT_BYTES;
constexpr int STAGE_PITCH = 36;  // words of a token's row in an epilogue warp's buffer
constexpr uint32_t EPI_BYTES = 8 * 32 * STAGE_PITCH * 4;
constexpr uint32_t AUX_BYTES = (2 * S + 2 * NS + 5) * 8 + 16;
constexpr uint32_t SMEM_BYTES = 1024 + RING_BYTES + EPI_BYTES + AUX_BYTES;
constexpr int SLOT_CHUNK = 2 * S8_CHUNK;  // slots whose sums fp32 holds exactly
static_assert(S % 2 == 0 && 2 * TN + 32 * NS <= 512 && SMEM_BYTES <= 232448 && STAGE_BYTES % 1024 == 0 && SLOT_BYTES % 1024 == 0, "");

// Registers of a thread: at launch, and by role.
constexpr int REGS_LAUNCH = 72, REGS_SUMS = 128, REGS_OPERANDS = 56, REGS_REST = 24;
static_assert(NS == 4 && 256 * REGS_SUMS + 128 * NS * REGS_OPERANDS + 128 * REGS_REST <= THREADS * REGS_LAUNCH, "what was launched is shared out");
struct Tile {
    int64_t n0, row0;
    int expert, rows, tn;  // rows that exist; the MMA's columns: a multiple of 32
};

// Tile t of the launch (warp-wide): token blocks vary fastest.  False past the end.
__device__ __forceinline__ bool pair_tile(const S8GemmParams& P, int64_t blocks, int64_t t, int lane, Tile& o) {
    if (t >= blocks * P.tiles_n) return false;
    const int64_t b = t % blocks;
    o.n0 = t / blocks * 256;
    o.expert = 0;
    if (P.offsets) {
        int64_t atom_row;
        if (!mx_expert_block(P.offsets, P.num_experts, P.epi.M, P.tile_rows, b, lane, &o.expert, &o.row0, &o.rows, &atom_row)) return false;
    } else {
        o.row0 = b * P.tile_rows;
        o.rows = (int)(P.epi.M - o.row0 < P.tile_rows ? P.epi.M - o.row0 : P.tile_rows);
    }
    o.tn = o.rows > 32 ? (o.rows + 31) / 32 * 32 : 32;
    return true;
}

__device__ __forceinline__ int64_t expert_blocks(const S8GemmParams& P, int lane) {
    int32_t n = 0;
    for (int32_t e = lane; e < P.num_experts; e += 32) n = mx_add_blocks(n, P.offsets[e], P.offsets[e + 1], P.tile_rows, P.tiles_m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    return n < P.tiles_m ? n : P.tiles_m;
}

// A block of 32 tokens (m0 ..) x 32 channels (n0 ..) of finished sums, in `stage` with
// a token a row: a lane has the same four channels of eight tokens, so that a token's
// 32 channels are stored together.  tokens: the factor of token `lane`.
template <int ACT, int DT, bool USE_C>
__device__ __forceinline__ void store_block(const S8GemmParams& P, const int32_t* stage, int64_t m0, int rows, int64_t n0, float tokens,
                                            const S8Channels& ch, int lane) {
    const EpiParams& e = P.epi;
    EpiArith ar = epi_arith(e);
    ar.alpha = 1.0f;
    const int64_t n = n0 + 4 * (lane & 7);
    const int have = e.N - n < 4 ? (int)(e.N - n) : 4;
    const bool vec = P.vec4 && have == 4;
    if constexpr (!USE_C) ar.beta = 0.0f;
    const bool whole = P.vec4 && n0 + 32 <= e.N && rows > 0;  // every lane's four channels exist
    const int64_t r0 = m0 + lane / 8;
    // four rows' C in flight together (one by one, each after the last one's store, they
    // took 4096^3 from 114 us to 181)
#pragma unroll 1
    for (int q0 = 0; q0 < 8; q0 += 4) {
        float c[4][4] = {};
        if (USE_C && whole) {
            // (no branch between the loads, and no conversion: the first one would wait)
            using Raw = std::conditional_t<DT == DT_F32, uint4, uint2>;
            Raw raw[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 4 * (q0 + q) + lane / 8, in = r < rows ? r : rows - 1;
                const int64_t at = (m0 + in) * e.ldc + n;
                raw[q] = *reinterpret_cast<const Raw*>(static_cast<const char*>(e.C) + at * (DT == DT_F32 ? 4 : 2));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (DT == DT_F32) {
                    c[q][0] = __uint_as_float(raw[q].x), c[q][1] = __uint_as_float(raw[q].y);
                    c[q][2] = __uint_as_float(raw[q].z), c[q][3] = __uint_as_float(raw[q].w);
                } else {
                    const uint32_t w[2] = {raw[q].x, raw[q].y};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 f = DT == DT_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]))
                                                       : __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                        c[q][2 * k] = f.x;
                        c[q][2 * k + 1] = f.y;
                    }
                }
            }
        } else if (USE_C) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 4 * (q0 + q) + lane / 8;
                const int64_t at = (r0 + 4 * (q0 + q)) * e.ldc + n;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r < rows && k < have) c[q][k] = ld_elem(e.C, DT, at + k);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 4 * (q0 + q) + lane / 8;
            const float token = __shfl_sync(0xFFFFFFFFu, tokens, r);
            if (r >= rows || have <= 0) continue;
            const int4 s = *reinterpret_cast<const int4*>(stage + r * STAGE_PITCH + 4 * (lane & 7));
            float x[4];
            mx_value2<ACT, DT>(ar, s8_scaled(s.x, token, ch.scale[0]), s8_scaled(s.y, token, ch.scale[1]), c[q][0], c[q][1], ch.bias[0], ch.bias[1],
                               x[0], x[1]);
            mx_value2<ACT, DT>(ar, s8_scaled(s.z, token, ch.scale[2]), s8_scaled(s.w, token, ch.scale[3]), c[q][2], c[q][3], ch.bias[2], ch.bias[3],
                               x[2], x[3]);
            const int64_t at = (r0 + 4 * (q0 + q)) * e.ldd + n;
            if (vec) {
                st4(e.D, DT, at, make_float4(x[0], x[1], x[2], x[3]));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < have) st_elem(e.D, DT, at + k, x[k]);
            }
        }
    }
}
__device__ __forceinline__ void store_block_any(const S8GemmParams& P, const int32_t* stage, int64_t m0, int rows, int64_t n0, float tokens,
                                                const S8Channels& ch, int lane) {
    with_epi_act(P.epi, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        auto typed = [&](auto use_c) {
            constexpr bool USE_C = decltype(use_c)::value;
            if (P.epi.d_type == DT_BF16)
                store_block<ACT, DT_BF16, USE_C>(P, stage, m0, rows, n0, tokens, ch, lane);
            else if (P.epi.d_type == DT_F16)
                store_block<ACT, DT_F16, USE_C>(P, stage, m0, rows, n0, tokens, ch, lane);
            else
                store_block<ACT, DT_F32, USE_C>(P, stage, m0, rows, n0, tokens, ch, lane);
        };
        if (P.epi.beta != 0.0f)
            typed(std::true_type{});
        else
            typed(std::false_type{});
    });
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    s8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ S8GemmParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* slots = smem + S * STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + RING_BYTES + EPI_BYTES);
    uint64_t* empty = full + S;        // a stage's codes have been read (8 warps)
    uint64_t* ready = empty + S;       // leader: both CTAs' operands of a K-step are in its two slots (16 warps)
    uint64_t* slot_free = ready + NS / 2;
    uint64_t* tfull = slot_free + NS;
    uint64_t* tempty = tfull + 2;      // leader: a buffer is in both CTAs' sums (16 warps)
    uint64_t* done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 8);
        }
        for (int s = 0; s < NS / 2; ++s) mbar_init(&ready[s], 16);
        for (int s = 0; s < NS; ++s) mbar_init(&slot_free[s], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 16);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot, tmem_w = tmem + 2 * TN;
    griddep_launch_dependents();
    griddep_wait();
    const Guard g{P.status, P.timeout_ns, abort_flag};
    const int64_t pid = blockIdx.x >> 1;
    const int64_t blocks = P.offsets ? expert_blocks(P, lane) : P.tiles_m;
    const int nslots = 2 * P.k_steps;  // of a tile

    if (warp < 4) {
        regs_down<REGS_REST>();
        if (warp == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            bool ok = true;
            Tile t;
            for (int64_t i = pid; ok && pair_tile(P, blocks, i, lane, t); i += P.programs) {
                const int32_t w0 = (int32_t)(t.n0 + 128 * rank), x0 = (int32_t)(t.row0 + rank * (t.tn / 2));
                for (int k = 0; k < P.k_steps; ++k) {
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(&empty[s], ph ^ 1, g, SITE_PRODUCER_EMPTY));
                    if (!ok) break;
                    uint8_t* w = smem + (uint32_t)s * STAGE_BYTES;
                    armed |= 1u << s;
                    armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[s], STAGE_BYTES);
                        if (P.b3d)
                            tma_load_3d(w, &tmB, &full[s], k * S8_KSTEP, w0, t.expert);
                        else
                            tma_load_2d(w, &tmB, &full[s], k * S8_KSTEP, w0);
                        tma_load_2d(w + W_BYTES, &tmA, &full[s], k * S8_KSTEP, x0);
                    }
                    __syncwarp();
                    if (++s == S) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (lane == 0) {
                // never leave with copies in flight into this CTA's shared memory
                for (int i = 0; i < S; ++i)
                    if (armed & (1u << i)) wait_bar_drain(&full[i], (armed_par >> i) & 1u, g);
            }
            __syncwarp();
        } else if (warp == 1 && leader) {
            // ---------------- MMAs (even CTA) ----------------
            const uint64_t xd0 = make_sw128_kmajor_desc(smem_u32(slots));
            int slot = 0;
            uint32_t ph = 0, chunk = 0;
            bool ok = true, issued = false;
            Tile t;
            for (int64_t i = pid; ok && pair_tile(P, blocks, i, lane, t); i += P.programs) {
                const uint32_t idesc = make_idesc_f16(0, 256, t.tn);
                for (int j0 = 0; ok && j0 < nslots; j0 += SLOT_CHUNK, ++chunk) {
                    const uint32_t b = chunk & 1, d = tmem + TN * b;
                    const int n = nslots - j0 < SLOT_CHUNK ? nslots - j0 : SLOT_CHUNK;
                    ok = __all_sync(0xFFFFFFFFu, wait_bar_cluster(&tempty[b], ((chunk >> 1) & 1) ^ 1, g, SITE_MMA_TMEM_EMPTY));
                    // Two slots at a time: waiting and issuing take this warp some 500 cycles
                    // a turn, eight MMAs 768.
                    for (int j = 0; ok && j < n; j += 2) {
                        ok = __all_sync(0xFFFFFFFFu, wait_bar_cluster(&ready[slot / 2], ph, g, SITE_MMA_OPERAND));
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint64_t xd = xd0 + (uint64_t)((uint32_t)slot * (SLOT_BYTES / 16));
                        const uint32_t wa = tmem_w + 32 * slot;
                        if (elect_one()) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) umma_f16_ts_pair(d, wa + 8 * q, xd + 2 * q, idesc, q ? 1u : (uint32_t)j);
                            umma_commit_pair_mc(&slot_free[slot], 0x3);
#pragma unroll
                            for (int q = 0; q < 4; ++q) umma_f16_ts_pair(d, wa + 32 + 8 * q, xd + SLOT_BYTES / 16 + 2 * q, idesc, 1u);
                            umma_commit_pair_mc(&slot_free[slot + 1], 0x3);
                            if (j == n - 2) umma_commit_pair_mc(&tfull[b], 0x3);
                        }
                        __syncwarp();
                        issued = true;
                        if ((slot += 2) == NS) {
                            slot = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
            if (issued) {  // every issued MMA has finished before TMEM is freed
                if (elect_one()) umma_commit_pair_mc(done, 0x1);
                __syncwarp();
                wait_bar_drain(done, 0, g);
            }
            __syncwarp();
        }
    } else if (warp < 12) {
        // ---------------- sums and epilogue ----------------
        regs_up<REGS_SUMS>();
        const int quarter = warp % 4, half = (warp - 4) / 4;
        int32_t* stage = reinterpret_cast<int32_t*>(smem + RING_BYTES) + (warp - 4) * 32 * STAGE_PITCH;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t l_tempty = mapa_shared(smem_u32(tempty), 0);
        uint32_t chunk = 0;
        Tile t;
        EpiArith ar = epi_arith(P.epi);
        ar.alpha = 1.0f;
        bool ok = true;
        for (int64_t i = pid; ok && pair_tile(P, blocks, i, lane, t); i += P.programs) {
            const int cols = t.tn / 2, c0 = half * cols;  // this warp's columns: a multiple of 16
            const int64_t n0 = t.n0 + 128 * rank + 32 * quarter, m0 = t.row0 + c0;
            const int rows = t.rows - c0 < cols ? t.rows - c0 : cols;
            if (P.epi.beta != 0.0f && n0 < P.epi.N)
                for (int r = lane; r < rows; r += 32) mx_prefetch_c(P.epi, m0 + r, n0, P.epi.N - n0 < 32 ? P.epi.N - n0 : 32);
            int32_t sum[HALF];
#pragma unroll
            for (int q = 0; q < HALF; ++q) sum[q] = 0;
            for (int j = 0; j < nslots; j += SLOT_CHUNK, ++chunk) {
                const uint32_t b = chunk & 1;
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&tfull[b], (chunk >> 1) & 1, g, SITE_EPI_TMEM_FULL));
                if (!ok) break;
                tc_fence_after_sync();
                __syncwarp();
#pragma unroll
                for (int q = 0; q < HALF; q += 16)
                    if (q < cols) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(tmem + TN * b + c0 + q + lanes, v);
#pragma unroll
                        for (int r = 0; r < 16; ++r) sum[q + r] += __float2int_rn(__uint_as_float(v[r]));
                    }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(l_tempty + 8u * b);
            }
            if (!ok) break;
            if (rows <= 0 || n0 >= P.epi.N) continue;
            if (!mx_block_in_bounds(P.epi, m0, rows, n0, P.epi.N - n0 < 32 ? P.epi.N - n0 : 32)) continue;
            const S8Channels ch = s8_channels(P, ar, t.expert, n0 + 4 * (lane & 7));
#pragma unroll
            for (int q = 0; q < HALF; q += 32)
                if (q < rows) {
                    const float tokens = q + lane < rows ? s8_token_factor(P, m0 + q + lane) : 0.0f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) stage[k * STAGE_PITCH + lane] = sum[q + k];
                    __syncwarp();
                    store_block_any(P, stage, m0 + q, rows - q, n0, tokens, ch, lane);
                    __syncwarp();
                }
        }
    } else {
        // ---------------- f16 operands ----------------
        regs_down<REGS_OPERANDS>();
        const int slot = (warp - 12) / 4, half = slot & 1, thread = threadIdx.x & 127, row = warp % 4 * 32 + lane;
        const uint32_t taddr = tmem_w + 32 * slot + ((uint32_t)(warp % 4 * 32) << 16);
        const uint32_t l_ready = mapa_shared(smem_u32(&ready[slot / 2]), 0);
        const uint32_t out = smem_u32(slots) + slot * SLOT_BYTES;
        // slots and K-steps are counted through all tiles; a stage is always read by the
        // same two groups, so that none meets a phase of full[] out of turn
        uint32_t n = slot, end = 0;
        HalfStage<HALF / 8> codes(half, row, thread);
        bool ok = true;
        Tile t;
        for (int64_t i = pid; ok && pair_tile(P, blocks, i, lane, t); i += P.programs) {
            end += nslots;
            for (; n < end; n += NS) {
                const uint32_t step = n / 2, s = step % S;
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[s], (step / S) & 1, g, SITE_DQ_RAW));
                if (!ok) break;
                const uint32_t w = smem_u32(smem) + s * STAGE_BYTES;
                codes.load(w, w + W_BYTES, t.tn / 2);
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&slot_free[slot], ((n / NS) & 1) ^ 1, g, SITE_DQ_EMPTY));
                if (!ok) break;
                tc_fence_after_sync();
                __syncwarp();
                codes.store(taddr, out, t.tn / 2);
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&empty[s]);
                    if (leader)
                        mbar_arrive(&ready[slot / 2]);
                    else
                        mbar_arrive_remote_smem(l_ready);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the leader's MMAs and all cross-CTA arrivals are done
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, 512);
    }
}

cudaError_t configure() {
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        // the split of registers above holds for this many at launch; with fewer, the
        // warps that ask for more would wait for ever
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, s8_pair_kernel);
        if (e != cudaSuccess) return e;
        if (a.numRegs != REGS_LAUNCH) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(s8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_s8_pair(const S8Maps& m, const S8GemmParams& p, int clusters, cudaStream_t st) {
    if (p.tile_rows < 32 || p.tile_rows > TN || p.tile_rows % 32) return cudaErrorInvalidValue;
    const cudaError_t e = configure();
    if (e != cudaSuccess) return e;
    return launch_pdl(s8_pair_kernel, 2 * clusters, THREADS, SMEM_BYTES, st, m.a, m.b, p);
}

int s8_pair_max_clusters() {
    if (configure() != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, s8_pair_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace qg
