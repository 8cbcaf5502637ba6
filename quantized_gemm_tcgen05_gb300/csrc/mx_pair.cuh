// Product of two 4-bit microscaled operands on CTA pairs: persistent clusters
// of two, one 256 x 256 tile at a time (tcgen05.mma.cta_group::2).
//
// Per 256-wide K-step an SM takes in its 128 rows of A, its half of the 256 rows
// of B, the scale atom of its A rows and both atoms of B (a pair's MMA wants all
// of B's scales in both CTAs' TMEM): 38 KB for 128 x 256 x 256 products, the
// least per product that the accumulator's size allows.
//
// Measured (back-to-back launches): 4096^3 31 us, 4.4 PFLOP/s; 4096 x 14336 x 4096
// 80 us in MXFP4, 86 in NVFP4, 6.0 and 5.6 PFLOP/s.  A K-step takes 0.41 us where
// its copies alone take 0.34 with every SM at it (0.29 with a few) and its MMAs
// alone 0.25, so the copies come first; the tensor pipe is active 41% of the time,
// and neither L2 (28% of its throughput) nor the crossbar (24%) is near its limit.
// What did not help: sharing A between two neighbouring pairs by multicast (a
// fifth less asked of L2), fetching operands into L2 ahead, another order of
// tiles, copies of two K-steps at once in a ring of four (104 us), and giving the
// accumulator back earlier still (all of it parked in shared memory and a stage
// less: 98 us; a quarter parked and more registers: 91).  The epilogue shares the
// schedulers with the warps that issue copies and MMAs, so its instructions cost
// main loop time wherever they stand: GELU takes 86 us to 112.
//
// TMEM: 256 accumulator columns and as many scale buffers as the ring has
// stages.  Scales go from shared memory to TMEM through the registers of four
// warps, one per 32-lane quarter (every quarter holds all scales).  Copies by the
// tensor core's own queue (tcgen05.cp) are simpler but stand in line with the
// MMAs: twelve a K-step took 4096^3 from 38 to 58 us.
//
//   warp 0      TMA producer (both CTAs; the operands' bytes complete on the
//               leader's full[s], each CTA's scales on its own sfull[s])
//   warp 1      leader: MMAs
//   warps 2-9   epilogue: a warp takes 32 rows x 128 columns into registers, gives
//               the accumulator back, then stores; so the next tile's main loop
//               waits for eight warps' TMEM loads only, not for their stores
//   warps 10-13 scales: shared memory -> TMEM, then arrive on the leader's sready[s]
//
// Grouped problems: 256-row blocks of one expert's rows; the blocks that exist
// are counted on the device and shared out, so none is assigned in vain (no more
// of them than any partition of the rows has, whatever the offsets say).
#pragma once
#include <atomic>

#include "mx_epilogue.cuh"
#include "mx_rows.h"

namespace qg {

constexpr int MX_PAIR_THREADS = 448;

template <bool NVF4>
struct MxPairCfg {
    static constexpr int BN = 256;
    static constexpr uint32_t A_BYTES = 128 * 128, B_BYTES = 128 * 128;
    static constexpr uint32_t SA_BYTES = NVF4 ? 2048 : 1024, SB_BYTES = 2 * SA_BYTES;
    static constexpr int S_ATOMS = NVF4 ? 4 : 2;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
    static constexpr int STAGES = 5;
    static constexpr uint32_t SCALE_COLS = 12 * S_ATOMS;  // A 4, B 8 a K-atom
    static_assert(STAGE_BYTES % 1024 == 0 && BN + STAGES * SCALE_COLS <= 512, "");
    static constexpr uint32_t EPI_BYTES = 8 * (32 * 33 + 12) * 4;
    static constexpr uint32_t AUX_BYTES = (4 * STAGES + 3) * 8 + 16;
    static constexpr uint32_t SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + AUX_BYTES;
    static_assert(SMEM_BYTES <= 232448, "");
};

struct MxTile {
    int64_t n0, row0, atom_row;
    int expert, rows;  // rows of the 256 that exist
};

// Blocks of bm rows that rows sorted by expert make, at most `most` (every lane
// gets it).  `most` is below 2^24, so 32 lanes' sums fit.
__device__ __forceinline__ int64_t mx_expert_blocks(const int32_t* off, int32_t E, int bm, int32_t most, int lane) {
    int32_t n = 0;
    for (int32_t e = lane; e < E; e += 32) n = mx_add_blocks(n, off[e], off[e + 1], bm, most);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    return n < most ? n : most;
}

// Tile t of the launch (warp-wide): M blocks vary fastest.  False past the end.
__device__ __forceinline__ bool mx_pair_tile(const MxGemmParams& P, int64_t blocks, int64_t t, int lane, MxTile& o) {
    if (t >= blocks * P.tiles_n) return false;
    const int64_t b = t % blocks;
    o.n0 = t / blocks * 256;
    o.expert = 0;
    if (P.offsets) return mx_expert_block(P.offsets, P.num_experts, P.epi.M, 256, b, lane, &o.expert, &o.row0, &o.rows, &o.atom_row);
    o.row0 = b * 256;
    o.rows = (int)(P.epi.M - o.row0 < 256 ? P.epi.M - o.row0 : 256);
    o.atom_row = 2 * b;
    return true;
}

template <bool NVF4>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MX_PAIR_THREADS, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ MxGemmParams P) {
    using Cfg = MxPairCfg<NVF4>;
    constexpr int S = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* stage_all = reinterpret_cast<float*>(smem + S * Cfg::STAGE_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * Cfg::STAGE_BYTES + Cfg::EPI_BYTES);
    uint64_t* empty = full + S;
    uint64_t* sfull = empty + S;    // this CTA's scales are in shared memory
    uint64_t* sready = sfull + S;   // leader: both CTAs' scales are in TMEM (8 warps)
    uint64_t* tfull = sready + S;
    uint64_t* tempty = tfull + 1;  // leader: 16 epilogue warps of the pair
    uint64_t* done = tempty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sfull[s], 1);
            mbar_init(&sready[s], 8);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 16);
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();
    const Guard g{P.status, P.timeout_ns, abort_flag};
    const int64_t pid = blockIdx.x >> 1;
    const int64_t blocks = P.offsets ? mx_expert_blocks(P.offsets, P.num_experts, 256, P.tiles_m, lane) : P.tiles_m;
    const int64_t tiles = blocks * P.tiles_n;

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        int s = 0;
        uint32_t ph = 0, armed = 0, armed_par = 0;
        bool ok = true;
        MxTile t, next;
        const uint32_t l_full = mapa_shared(smem_u32(full), 0);
        // the next tile is looked up while the ring is full, not between tiles
        const int look = (P.k_steps < S ? P.k_steps : S) - 1;
        bool have = mx_pair_tile(P, blocks, pid, lane, t);
        for (int64_t i = pid; ok && have; i += P.programs, t = next) {
            const int32_t a0 = (int32_t)(t.row0 + 128 * rank), b0 = (int32_t)(t.n0 + 128 * rank);
            const int32_t sa0 = (int32_t)(t.atom_row + rank), sb0 = (int32_t)(t.n0 / 128);
            int32_t kx = 0, sx = 0;
            for (int k = 0; k < P.k_steps; ++k) {
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&empty[s], ph ^ 1, g, SITE_PRODUCER_EMPTY));
                if (!ok) break;
                uint8_t* a = smem + (uint32_t)s * Cfg::STAGE_BYTES;
                uint8_t* b = a + Cfg::A_BYTES;
                uint8_t* sa = b + Cfg::B_BYTES;
                uint8_t* sb = sa + Cfg::SA_BYTES;
                const uint32_t bar = l_full + 8u * s;
                armed |= 1u << s;
                armed_par = (armed_par & ~(1u << s)) | (ph << s);
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(&full[s], 2 * (Cfg::A_BYTES + Cfg::B_BYTES));
                    mbar_arrive_expect_tx(&sfull[s], Cfg::SA_BYTES + Cfg::SB_BYTES);
                    tma_load_2d(sa, &tmSA, &sfull[s], sx, sa0);
                    if (P.b3d) {
                        tma_load_3d(sb, &tmSB, &sfull[s], sx, sb0, t.expert);
                        tma_load_3d_pair(b, &tmB, bar, kx, b0, t.expert);
                    } else {
                        tma_load_2d(sb, &tmSB, &sfull[s], sx, sb0);
                        tma_load_2d_pair(b, &tmB, bar, kx, b0);
                    }
                    tma_load_2d_pair(a, &tmA, bar, kx, a0);
                }
                __syncwarp();
                if (k == look) have = mx_pair_tile(P, blocks, i + P.programs, lane, next);
                kx += 128;
                sx += (int32_t)(Cfg::SA_BYTES / 8);
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            // never leave with copies in flight into this CTA's shared memory
            for (int i = 0; i < S; ++i)
                if (armed & (1u << i)) {
                    wait_bar_drain(&sfull[i], (armed_par >> i) & 1u, g);
                    if (leader) wait_bar_drain(&full[i], (armed_par >> i) & 1u, g);
                }
            if (!leader && !ok) {
                // the odd CTA cannot see its operand copies complete (they land on
                // the leader's barriers); after an abort give them time to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1 && leader) {
        // ---------------- MMAs (even CTA) ----------------
        const uint64_t ad0 = make_sw128_kmajor_desc(smem_u32(smem));
        const uint64_t bd0 = make_sw128_kmajor_desc(smem_u32(smem) + Cfg::A_BYTES);
        int s = 0;
        uint32_t ph = 0, it = 0;
        bool ok = true, issued = false;
        for (int64_t i = pid; ok && i < tiles; i += P.programs, ++it) {
            // the accumulator's previous tile is in the epilogue's registers
            ok = __all_sync(0xFFFFFFFFu, wait_bar_cluster(tempty, (it & 1) ^ 1, g, SITE_MMA_TMEM_EMPTY));
            tc_fence_after_sync();
            for (int k = 0; ok && k < P.k_steps; ++k) {
                // the leader's scale warps have seen both CTAs' operands land before they arrive
                ok = __all_sync(0xFFFFFFFFu, wait_bar_cluster(&sready[s], ph, g, SITE_MMA_OPERAND));
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t ad = ad0 + (uint64_t)((uint32_t)s * (Cfg::STAGE_BYTES / 16));
                const uint64_t bd = bd0 + (uint64_t)((uint32_t)s * (Cfg::STAGE_BYTES / 16));
                const uint32_t ta = tmem + Cfg::BN + (uint32_t)s * Cfg::SCALE_COLS, tb = ta + 4 * Cfg::S_ATOMS;
                const uint32_t acc = k > 0 ? 1u : 0u;
                if (elect_one()) {
                    // always four: past K's end codes and scales are zeros
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (NVF4) {
                            umma_mx_ss_pair<true>(tmem, ad + 2 * q, bd + 2 * q, P.idesc, ta + 4 * q, tb + 8 * q, q ? 1u : acc);
                        } else {
                            const uint32_t id = (q & 1) * 2u;
                            umma_mx_ss_pair<false>(tmem, ad + 2 * q, bd + 2 * q, P.idesc | (id << 29) | (id << 4),
                                                   ta + 4 * (q / 2), tb + 8 * (q / 2), q ? 1u : acc);
                        }
                    }
                    umma_commit_pair_mc(&empty[s], 0x3);
                    if (k == P.k_steps - 1) umma_commit_pair_mc(tfull, 0x3);
                }
                __syncwarp();
                issued = true;
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (issued) {  // every issued MMA has finished before TMEM is freed
            if (elect_one()) umma_commit_pair_mc(done, 0x1);
            __syncwarp();
            wait_bar_drain(done, 0, g);
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ---------------- scales: shared memory -> TMEM ----------------
        const uint32_t quarter = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t l_sready = mapa_shared(smem_u32(sready), 0);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t i = pid; ok && i < tiles; i += P.programs) {
            for (int k = 0; k < P.k_steps; ++k) {
                // the scales are there; the buffer's previous readers are done (the
                // producer has waited for the same phase of empty[s])
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&sfull[s], ph, g, SITE_DQ_RAW));
                if (!ok) break;
                tc_fence_after_sync();
                const uint8_t* sa = smem + s * Cfg::STAGE_BYTES + Cfg::A_BYTES + Cfg::B_BYTES + lane * 16;
                const uint32_t ta = tmem + Cfg::BN + s * Cfg::SCALE_COLS + quarter;
                uint32_t ra[4 * Cfg::S_ATOMS], rb[8 * Cfg::S_ATOMS];
#pragma unroll
                for (int q = 0; q < 3 * Cfg::S_ATOMS; ++q) {
                    // A's atoms, then B's first 128 rows', then its second
                    const uint4 w = *reinterpret_cast<const uint4*>(sa + MX_ATOM_BYTES * q);
                    uint32_t* r = q < Cfg::S_ATOMS ? ra + 4 * q
                                                   : rb + 8 * (q % Cfg::S_ATOMS) + (q < 2 * Cfg::S_ATOMS ? 0 : 4);
                    r[0] = w.x;
                    r[1] = w.y;
                    r[2] = w.z;
                    r[3] = w.w;
                }
                tmem_st_32x32b(ta, ra);
                tmem_st_32x32b(ta + 4 * Cfg::S_ATOMS, rb);
                tmem_st_wait();
                if (leader) {
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[s], ph, g, SITE_MMA_FULL));
                    if (!ok) break;
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&sready[s]);  // (a release: what full[s] showed this warp, the MMA thread sees)
                    else
                        mbar_arrive_remote_relaxed(l_sready + 8u * s);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp >= 2) {
        // ---------------- epilogue ----------------
        const int ew = warp % 4, half = (warp - 2) / 4;
        float* stage = stage_all + (warp - 2) * (32 * 33 + 12);  // 16-byte aligned for the packed form
        const uint32_t l_tempty = mapa_shared(smem_u32(tempty), 0);
        uint32_t it = 0;
        MxTile t;
        for (int64_t i = pid; mx_pair_tile(P, blocks, i, lane, t); i += P.programs, ++it) {
            float alpha = P.epi.alpha;
            if (P.expert_alpha) alpha *= P.expert_alpha[t.expert];
            int rows = t.rows - 128 * (int)rank - 32 * ew;
            rows = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
            const int64_t m0 = t.row0 + 128 * rank + 32 * ew, n0 = t.n0 + 128 * half;
            if (P.epi.beta != 0.0f && lane < rows && n0 < P.epi.N)
                mx_prefetch_c(P.epi, m0 + lane, n0, P.epi.N - n0 < 128 ? P.epi.N - n0 : 128);
            if (!__all_sync(0xFFFFFFFFu, wait_bar(tfull, it & 1, g, SITE_EPI_TMEM_FULL))) break;
            tc_fence_after_sync();
            const uint32_t ta = tmem + 128 * half + ((uint32_t)(ew * 32) << 16);
            const bool packed = P.vec32 && P.epi.d_type != DT_F32 && P.epi.beta == 0.0f && n0 + 128 <= P.epi.N;
            if (packed && rows > 0 && mx_block_in_bounds(P.epi, m0, rows, n0, 128)) {
                // a 16-bit D without C: half of the values wait finished in shared
                // memory, half as they are in registers, so the accumulator is given
                // back before the second half is worked on and before the first store
                float v[2][32];
                uint32_t w[32];
                uint8_t* buf = reinterpret_cast<uint8_t*>(stage);
                mx_load64(ta, v);
                mx_pack64_any(P.epi, alpha, v, n0, w, lane);
                mx_stage64(buf, w, lane);
                mx_load64(ta + 64, v);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(l_tempty);
                uint16_t* d = static_cast<uint16_t*>(P.epi.D) + m0 * P.epi.ldd + n0;
                mx_store64(buf, d, P.epi.ldd, rows, lane);
                mx_pack64_any(P.epi, alpha, v, n0 + 64, w, lane);
                __syncwarp();
                mx_stage64(buf, w, lane);
                __syncwarp();
                mx_store64(buf, d + 64, P.epi.ldd, rows, lane);
                __syncwarp();
                continue;
            }
            if (rows > 0) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    if (n0 + 32 * c >= P.epi.N) break;
                    float v[32];
                    tmem_load_chunk<32>(ta + 32 * c, v);
                    mx_store_block(P.epi, P.vec32, alpha, m0, rows, n0 + 32 * c, v, stage, lane);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(l_tempty);
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

template <bool NVF4>
cudaError_t mx_pair_configure() {
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(mx_pair_kernel<NVF4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)MxPairCfg<NVF4>::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return cudaSuccess;
}

template <bool NVF4>
cudaError_t launch_mx_pair_t(const MxMaps& m, const MxGemmParams& p, int clusters, cudaStream_t st) {
    const cudaError_t e = mx_pair_configure<NVF4>();
    if (e != cudaSuccess) return e;
    return launch_pdl(mx_pair_kernel<NVF4>, 2 * clusters, MX_PAIR_THREADS, MxPairCfg<NVF4>::SMEM_BYTES, st, m.a, m.b, m.sa, m.sb, p);
}

template <bool NVF4>
int mx_pair_clusters_t() {
    if (mx_pair_configure<NVF4>() != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(MX_PAIR_THREADS, 1, 1);
    cfg.dynamicSmemBytes = MxPairCfg<NVF4>::SMEM_BYTES;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<NVF4>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace qg
