// Product of two 4-bit microscaled operands, one output tile per cluster.
//
// D = sum over blocks of sa * sb * (sum of code products): the tensor core
// multiplies the scales in (tcgen05.mma with block scales), fp32 accumulator in
// TMEM.  A stage holds one K-step of 256 codes: the 128-byte swizzled rows of A
// (up to 128) and of B (BN), and the scale atoms of both (128 rows x 256 codes
// each).  Four warps move the scales from shared memory to TMEM, one per
// 32-lane quarter (every quarter holds all of them); there are as many scale
// buffers as stages, so a buffer is free whenever its stage is.
//
// The tile's K-steps are shared out over the `splits` CTAs of a cluster.  When
// all of them are through, each sends every other its share of the columns of
// its fp32 partial tile (bulk copies into the idle ring, counted by the
// receiver's barrier), adds what it received in rank order and finishes its
// columns; how the CTAs announce themselves and leave, also when one of them gave
// up, stands in mx_exchange.h.  Nothing goes through global memory but operands
// and D, and no workspace is needed.  Bulk copies carry their own completion:
// cluster barriers and remote loads in their place took 4 us of a 9 us launch.
//
//   warp 0     TMA producer          warps 4-7  scales
//   warp 1     MMAs                  all        epilogue
//
// Two CTAs fit an SM (shared memory and TMEM both), so one's set-up and
// epilogue overlap the other's main loop.
//
// Only the rows of A that exist are copied (a_rows): with few rows the MMAs read
// whatever shared memory holds below them, which reaches only accumulator rows
// that are not stored.
#pragma once
#include <atomic>

#include "mx_epilogue.cuh"
#include "mx_exchange.h"

namespace qg {

constexpr int MX_THREADS = 256;

template <int BN, bool NVF4>
struct MxCfg {
    static constexpr uint32_t B_BYTES = BN * 128;
    static constexpr uint32_t S_BYTES = NVF4 ? 2048 : 1024;  // one operand's scale atoms of a K-step
    static constexpr int S_ATOMS = NVF4 ? 4 : 2;
    static constexpr uint32_t TMEM_COLS = 256;
    static constexpr uint32_t SCALE_COLS = 8 * S_ATOMS;  // A 4, B 4 a K-atom
    static constexpr int MAX_STAGES = (TMEM_COLS - BN) / SCALE_COLS < 8 ? (TMEM_COLS - BN) / SCALE_COLS : 8;
    static constexpr uint32_t AUX_BYTES = (3 * MAX_STAGES + 3) * 8 + 16;
    static constexpr uint32_t WARP_STAGE = (32 * 33 + 12) * 4;  // an epilogue warp's buffer
    // two CTAs an SM: at most half of its 228 KB, a kilobyte each reserved
    static constexpr uint32_t BUDGET = 113 * 1024;
    QG_HD static uint32_t stage_bytes(int a_rows) { return a_rows * 128u + B_BYTES + 2 * S_BYTES; }
    // the ring, with room below the last stage for the rows of A an MMA reads
    // beyond a_rows, and for what the epilogue keeps there: its warps' buffers,
    // or the partial tile sent and the shares received (rows of an odd pitch)
    QG_HD static uint32_t ring_bytes(int a_rows, int stages, int splits) {
        const uint32_t sb = stage_bytes(a_rows);
        uint32_t n = sb * (stages - 1) + (sb > 16384u ? sb : 16384u);
        const uint32_t epi = splits > 1 ? 2 * (BN / 4) * (a_rows + 1) * 16 : 8 * WARP_STAGE;
        return ((n > epi ? n : epi) + 1023) / 1024 * 1024;
    }
    static uint32_t smem_bytes(int a_rows, int stages, int splits) {
        const uint32_t n = 1024 + ring_bytes(a_rows, stages, splits) + AUX_BYTES;
        return n < 80 * 1024 ? 80 * 1024 : n;  // never three an SM: TMEM holds two
    }
    // 0: the partial tiles do not fit
    static int max_stages(int a_rows, int splits) {
        int s = MAX_STAGES;
        while (s > 0 && smem_bytes(a_rows, s, splits) > BUDGET) --s;
        return s < 2 ? 0 : s;
    }
};

// The steps of mx_exchange.h: announcements on `idle`, shares (`bytes` each) out of
// `parts` into the others' `recv`, counted by their `part`.
struct MxClusterLink {
    uint64_t *idle, *part;
    volatile uint32_t* warning;
    uint32_t parts, recv, bytes;
    int splits, rank;
    const Guard& g;
    __device__ __forceinline__ void expect() { mbar_arrive_expect_tx(part, (uint32_t)splits * bytes); }
    // (nothing is published: the arrivals are relaxed)
    __device__ __forceinline__ void announce(int z) { mbar_arrive_remote_relaxed(mapa_shared(smem_u32(idle), z)); }
    __device__ __forceinline__ bool await_announced() { return wait_bar_cluster_drain(idle, 0, g); }
    __device__ __forceinline__ void send(int z) {
        bulk_s2cluster(mapa_shared(recv + (uint32_t)rank * bytes, z), parts + (uint32_t)z * bytes, bytes,
                       mapa_shared(smem_u32(part), z));
    }
    __device__ __forceinline__ bool await_shares() { return wait_bar_cluster_drain(part, 0, g); }
    __device__ __forceinline__ void warn(int z) { st_cluster_fence(mapa_shared(smem_u32((const void*)warning), z), 1u); }
    __device__ __forceinline__ void arrive() { cluster_arrive_relaxed(); }
    __device__ __forceinline__ void wait() { cluster_wait(); }
    __device__ __forceinline__ bool warned() { return *warning != 0; }
    __device__ __forceinline__ void settle() { mx_settle(); }
};

template <int BN, bool NVF4>
__global__ void __launch_bounds__(MX_THREADS, 2)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ MxGemmParams P) {
    using Cfg = MxCfg<BN, NVF4>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = P.stages;
    const uint32_t a_bytes = (uint32_t)P.a_rows * 128u;
    const uint32_t stage_bytes = Cfg::stage_bytes(P.a_rows);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::ring_bytes(P.a_rows, S, P.splits));
    uint64_t* empty = full + Cfg::MAX_STAGES;
    uint64_t* sready = empty + Cfg::MAX_STAGES;  // the stage has landed and its scales are in TMEM (4 warps)
    uint64_t* tfull = sready + Cfg::MAX_STAGES;  // the accumulator is complete
    uint64_t* idle = tfull + 1;                  // every CTA of the cluster is through with its ring
    uint64_t* part = idle + 1;                   // the partial tiles' shares have arrived
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* warning = tmem_slot + 2;  // a CTA of the cluster has given up

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int splits = P.splits;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sready[s], 4);
        }
        mbar_init(tfull, 1);
        mbar_init(idle, (uint32_t)splits);
        mbar_init(part, 1);
        *abort_flag = 0;
        *warning = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (splits > 1) cluster_sync();  // every CTA's barriers exist before another's copies complete on them
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();

    const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
    const int64_t tile = blockIdx.x / splits;
    const int64_t tm = tile % P.tiles_m, tn = tile / P.tiles_m;
    const int k0 = (int)((int64_t)P.k_steps * rank / splits), k1 = (int)((int64_t)P.k_steps * (rank + 1) / splits);
    const int64_t n0 = tn * BN;
    const Guard g{P.status, P.timeout_ns, abort_flag};
    if (!P.offsets && warp == 0 && lane == 0) {
        // warm L2 with the first stages of the weights while the previous kernel
        // in the stream finishes (a hint: L2 is where memory is coherent)
        for (int k = k0; k < k1 && k < k0 + S; ++k) {
            tma_prefetch_l2_2d(&tmB, k * 128, (int32_t)n0);
            tma_prefetch_l2_2d(&tmSB, k * (int)(Cfg::S_BYTES / 8), (int32_t)(n0 / 128));
        }
    }

    griddep_wait();
    int expert = 0, rows = 0;
    int64_t row0 = 0, atom_row = 0;
    bool live = true;
    float alpha = P.epi.alpha;
    if (P.offsets) {
        live = mx_expert_block(P.offsets, P.num_experts, P.epi.M, 128, tm, lane, &expert, &row0, &rows, &atom_row);
        if (live && P.expert_alpha) alpha *= P.expert_alpha[expert];
    } else {
        row0 = tm * 128;
        rows = (int)(P.epi.M - row0 < 128 ? P.epi.M - row0 : 128);
        atom_row = tm;
    }

    bool ok = live;
    if (live && warp == 0) {
        int s = 0;
        uint32_t ph = 1;
        const uint32_t stage_tx = stage_bytes;
        int kx = k0 * 128, sx = k0 * (int)(Cfg::S_BYTES / 8);
        for (int k = k0; k < k1; ++k) {
            if (!__all_sync(0xFFFFFFFFu, wait_bar(&empty[s], ph, g, SITE_PRODUCER_EMPTY))) break;
            uint8_t* a = smem + (uint32_t)s * stage_bytes;
            uint8_t* b = a + a_bytes;
            uint8_t* sa = b + Cfg::B_BYTES;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], stage_tx);
                tma_load_2d(sa, &tmSA, &full[s], sx, (int32_t)atom_row);
                if (P.b3d) {
                    tma_load_3d(sa + Cfg::S_BYTES, &tmSB, &full[s], sx, (int32_t)(n0 / 128), expert);
                    tma_load_3d(b, &tmB, &full[s], kx, (int32_t)n0, expert);
                } else {
                    tma_load_2d(sa + Cfg::S_BYTES, &tmSB, &full[s], sx, (int32_t)(n0 / 128));
                    tma_load_2d(b, &tmB, &full[s], kx, (int32_t)n0);
                }
                tma_load_2d(a, &tmA, &full[s], kx, (int32_t)row0);
            }
            __syncwarp();
            kx += 128;
            sx += (int)(Cfg::S_BYTES / 8);
            if (++s == S) {
                s = 0;
                ph ^= 1;
            }
        }
    } else if (live && warp == 1) {
        const uint32_t sfb_off = 4 * Cfg::S_ATOMS + (uint32_t)(n0 % 128) / 32;
        const uint64_t ad0 = make_sw128_kmajor_desc(smem_u32(smem)), bd0 = make_sw128_kmajor_desc(smem_u32(smem) + a_bytes);
        uint64_t ad = ad0, bd = bd0;
        uint32_t ta = tmem + BN, acc = 0, ph = 0;
        int s = 0;
        for (int k = k0; k < k1; ++k) {
            // the scale warps have seen the whole stage land before they arrive here
            if (!__all_sync(0xFFFFFFFFu, wait_bar(&sready[s], ph, g, SITE_MMA_OPERAND))) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t tb = ta + sfb_off;
            if (elect_one()) {
                // always four: past K's end codes and scales are zeros
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (NVF4) {
                        umma_mx_ss<true>(tmem, ad + 2 * q, bd + 2 * q, P.idesc, ta + 4 * q, tb + 4 * q, q ? 1u : acc);
                    } else {
                        // an atom's four scales cover two instructions: bytes 0-1, then 2-3
                        const uint32_t id = (q & 1) * 2u;
                        umma_mx_ss<false>(tmem, ad + 2 * q, bd + 2 * q, P.idesc | (id << 29) | (id << 4),
                                          ta + 4 * (q / 2), tb + 4 * (q / 2), q ? 1u : acc);
                    }
                }
                umma_commit(&empty[s]);
                if (k == k1 - 1) umma_commit(tfull);
            }
            __syncwarp();
            acc = 1;
            ad += stage_bytes / 16;
            bd += stage_bytes / 16;
            ta += Cfg::SCALE_COLS;
            if (++s == S) {
                s = 0;
                ph ^= 1;
                ad = ad0;
                bd = bd0;
                ta = tmem + BN;
            }
        }
    } else if (live && warp < 4) {
        // two warps without a part in the main loop fetch the tile's C
        if (P.epi.beta != 0.0f && n0 < P.epi.N)
            for (int r = threadIdx.x - 64; r < rows; r += 64)
                mx_prefetch_c(P.epi, row0 + r, n0, P.epi.N - n0 < BN ? P.epi.N - n0 : BN);
    } else if (live) {
        const uint32_t quarter = (uint32_t)(warp % 4 * 32) << 16;
        int s = 0;
        uint32_t ph = 0;
        for (int k = k0; k < k1; ++k) {
            // the stage is there; the scale buffer's previous readers are done: the
            // producer has waited for that phase of empty[s]
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[s], ph, g, SITE_DQ_RAW));
            if (!ok) break;
            tc_fence_after_sync();
            const uint8_t* sa = smem + (uint32_t)s * stage_bytes + a_bytes + Cfg::B_BYTES + lane * 16;
            uint32_t r[8 * Cfg::S_ATOMS];
#pragma unroll
            for (int q = 0; q < 2 * Cfg::S_ATOMS; ++q) {
                const uint4 w = *reinterpret_cast<const uint4*>(sa + MX_ATOM_BYTES * q);
                r[4 * q] = w.x;
                r[4 * q + 1] = w.y;
                r[4 * q + 2] = w.z;
                r[4 * q + 3] = w.w;
            }
            tmem_st_32x32b(tmem + BN + (uint32_t)s * Cfg::SCALE_COLS + quarter, r);
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sready[s]);
            if (++s == S) {
                s = 0;
                ph ^= 1;
            }
        }
    }
    // every thread learns whether the accumulator is complete
    if (live) {
        ok = ok && wait_bar(tfull, 0, g, SITE_EPI_TMEM_FULL);
        tc_fence_after_sync();
    }
    bool all_ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (live && !all_ok) {
        // gave up: let copies in flight land and issued MMAs finish before shared memory and TMEM go
        mx_settle();
    }
    const int ew = warp % 4, half = warp / 4;
    const uint32_t tb = tmem + half * (BN / 2) + ((uint32_t)(ew * 32) << 16);
    const int wrows = rows - ew * 32 < 0 ? 0 : (rows - ew * 32 < 32 ? rows - ew * 32 : 32);
    if (splits == 1) {
        if (all_ok && wrows > 0) {
            uint8_t* buf = smem + warp * Cfg::WARP_STAGE;
            float* stage = reinterpret_cast<float*>(buf);
            const int64_t m0 = row0 + ew * 32, nh = n0 + half * (BN / 2);
            bool done = false;
            if constexpr (BN == 128) {
                if (P.vec32 && P.epi.d_type != DT_F32 && P.epi.beta == 0.0f && nh + 64 <= P.epi.N &&
                    mx_block_in_bounds(P.epi, m0, wrows, nh, 64)) {
                    float v[2][32];
                    uint32_t w[32];
                    mx_load64(tb, v);
                    mx_pack64_any(P.epi, alpha, v, nh, w, lane);
                    mx_stage64(buf, w, lane);
                    __syncwarp();
                    mx_store64(buf, static_cast<uint16_t*>(P.epi.D) + m0 * P.epi.ldd + nh, P.epi.ldd, wrows, lane);
                    done = true;
                }
            }
            if (!done) {
#pragma unroll 1
                for (int c = 0; c < BN / 64; ++c) {
                    if (nh + 32 * c >= P.epi.N) break;
                    float v[32];
                    tmem_load_chunk<32>(tb + 32 * c, v);
                    mx_store_block(P.epi, P.vec32, alpha, m0, wrows, nh + 32 * c, v, stage, lane);
                }
            }
        }
    } else {
        // partial tile -> shared memory, [quad of columns][row], rows at an odd pitch
        constexpr int QUADS = BN / 4;
        const uint32_t pitch = (uint32_t)(rows | 1) * 16u;
        const int nq = QUADS / splits;  // quads of this CTA's columns
        uint8_t* recv = smem + (size_t)QUADS * pitch;
        if (all_ok && wrows > 0) {
#pragma unroll 1
            for (int c = 0; c < BN / 64; ++c) {
                float v[32];
                tmem_load_chunk<32>(tb + 32 * c, v);
                if (lane < wrows) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4*>(smem + (half * (BN / 8) + 8 * c + j) * pitch + (ew * 32 + lane) * 16) =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
            }
        }
        fence_proxy_async_smem();  // ... visible to the bulk copies
        __syncthreads();
        if (live) {
            // (whether this CTA's part is right or not: the others wait for it)
            MxClusterLink link{idle, part, warning, smem_u32(smem), smem_u32(recv), (uint32_t)nq * pitch, splits, rank, g};
            ok = mx_exchange(link, splits, threadIdx.x == 0);
            all_ok = __syncthreads_and(all_ok && ok ? 1 : 0) != 0;
        }
        if (all_ok) {
            const EpiParams& e = P.epi;
            EpiArith ar = epi_arith(e);
            ar.alpha = alpha;
            for (int t = threadIdx.x; t < rows * nq; t += MX_THREADS) {
                const int q = t % nq, r = t / nq;
                const int64_t n = n0 + 4 * (rank * nq + q), m = row0 + r;
                if (n >= e.N) continue;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int z = 0; z < splits; ++z) {  // in K order
                    const float4 p = *reinterpret_cast<const float4*>(recv + (uint32_t)(z * nq + q) * pitch + r * 16);
                    sum.x += p.x;
                    sum.y += p.y;
                    sum.z += p.z;
                    sum.w += p.w;
                }
                float x[4];
                const int have = e.N - n < 4 ? (int)(e.N - n) : 4;
                if (!mx_block_in_bounds(e, m, 1, n, have)) continue;
                with_epi_act(e, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
                    float c[4], b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        c[j] = (e.beta != 0.0f && j < have) ? ld_elem(e.C, e.d_type, m * e.ldc + n + j) : 0.0f;
                        b[j] = ACT >= 0 ? bias_at(ar, n + j) : 0.0f;
                    }
                    mx_value2_any<ACT>(ar, e.d_type, sum.x, sum.y, c[0], c[1], b[0], b[1], x[0], x[1]);
                    mx_value2_any<ACT>(ar, e.d_type, sum.z, sum.w, c[2], c[3], b[2], b[3], x[2], x[3]);
                });
                if (P.vec32 && have == 4) {
                    st4(e.D, e.d_type, m * e.ldd + n, make_float4(x[0], x[1], x[2], x[3]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < have) st_elem(e.D, e.d_type, m * e.ldd + n + j, x[j]);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
    // shared memory goes only when nobody will read or write it any more
    if (live && splits > 1) {
        MxClusterLink link{idle, part, warning, 0, 0, 0, splits, rank, g};
        mx_exchange_leave(link);
    }
}

template <int BN, bool NVF4>
cudaError_t launch_mx_bn(const MxMaps& m, const MxGemmParams& p, int grid, cudaStream_t st) {
    using Cfg = MxCfg<BN, NVF4>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(mx_gemm_kernel<BN, NVF4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Cfg::BUDGET);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(MX_THREADS);
    cfg.dynamicSmemBytes = Cfg::smem_bytes(p.a_rows, p.stages, p.splits);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)p.splits;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<BN, NVF4>, m.a, m.b, m.sa, m.sb, p);
}

}  // namespace qg
