// Product of two 4-bit microscaled operands, one output tile per cluster.
//
// D = sum over blocks of sa * sb * (sum of code products): the tensor core
// multiplies the scales in (tcgen05.mma with block scales), fp32 accumulator in
// TMEM.  A stage holds one K-step of 256 codes: the 128-byte swizzled rows of A
// (up to 128) and of B (BN), and the scale atoms of both (128 rows x 256 codes
// each).  The MMA thread copies the atoms from shared memory to TMEM columns
// (tcgen05.cp, executed in order before the MMAs issued after it) and issues
// four MMAs of K = 64.  The scale columns are double-buffered: before step i
// overwrites a buffer, the MMAs of step i - 2 that read it have been waited for.
//
// The tile's K-steps are shared out over the `splits` CTAs of a cluster; their
// fp32 partial tiles are added in rank order through distributed shared
// memory, each CTA finishing its share of the columns.  Nothing goes through
// global memory but operands and D, and no workspace is needed.
//
// 128 threads: warp 0's first lane issues the copies, warp 1's the MMAs, then
// all four warps run the epilogue.  Two CTAs fit an SM (shared memory and TMEM
// both), so one's set-up and epilogue overlap the other's main loop.
//
// Only the rows of A that exist are copied (a_rows): with few rows the MMAs read
// whatever shared memory holds below them, which reaches only accumulator rows
// that are not stored.
#pragma once
#include <atomic>

#include "mx_epilogue.cuh"

namespace qg {

template <int BN, bool NVF4>
struct MxCfg {
    static constexpr uint32_t B_BYTES = BN * 128;
    static constexpr uint32_t S_BYTES = NVF4 ? 2048 : 1024;  // one operand's scale atoms of a K-step
    static constexpr int S_ATOMS = NVF4 ? 4 : 2;
    static constexpr int MAX_STAGES = 8;
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(BN + 64);
    static constexpr uint32_t AUX_BYTES = (2 * MAX_STAGES + 2) * 8 + 16;
    static constexpr uint32_t PART_PITCH = 129 * 16;  // a quad of columns x 128 rows, padded
    static constexpr uint32_t EPI_BYTES = BN / 4 * PART_PITCH;  // partial tile; also the 4 warps' 32 x 33 floats
    static uint32_t stage_bytes(int a_rows) { return a_rows * 128u + B_BYTES + 2 * S_BYTES; }
    // the ring, with room below the last stage for the rows of A an MMA reads beyond a_rows
    static uint32_t ring_bytes(int a_rows, int stages) {
        const uint32_t sb = stage_bytes(a_rows);
        uint32_t n = sb * stages;
        const uint32_t reach = sb * (stages - 1) + 128 * 128;
        if (n < reach) n = reach;
        return n < EPI_BYTES ? EPI_BYTES : n;
    }
    // two CTAs an SM: at most half of its 228 KB, a kilobyte each reserved
    static constexpr uint32_t BUDGET = 113 * 1024;
    static uint32_t smem_bytes(int a_rows, int stages) {
        const uint32_t n = 1024 + ring_bytes(a_rows, stages) + AUX_BYTES;
        return n < 80 * 1024 ? 80 * 1024 : n;  // never three an SM: TMEM holds two
    }
    static int max_stages(int a_rows) {
        int s = MAX_STAGES;
        while (s > 2 && smem_bytes(a_rows, s) > BUDGET) --s;
        return s;
    }
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int BN, bool NVF4>
__global__ void __launch_bounds__(128, 2)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ MxGemmParams P) {
    using Cfg = MxCfg<BN, NVF4>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = P.stages;
    const uint32_t a_bytes = (uint32_t)P.a_rows * 128u;
    const uint32_t stage_bytes = a_bytes + Cfg::B_BYTES + 2 * Cfg::S_BYTES;
    uint32_t ring_bytes = stage_bytes * (S - 1) + (stage_bytes > 16384u ? stage_bytes : 16384u);
    if (ring_bytes < Cfg::EPI_BYTES) ring_bytes = Cfg::EPI_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring_bytes);
    uint64_t* empty = full + Cfg::MAX_STAGES;
    uint64_t* tfull = empty + Cfg::MAX_STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tfull, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();

    const int rank = P.splits > 1 ? (int)cluster_ctarank() : 0;
    const int64_t tile = blockIdx.x / P.splits;
    const int64_t tm = tile % P.tiles_m, tn = tile / P.tiles_m;
    const int k0 = (int)((int64_t)P.k_steps * rank / P.splits), k1 = (int)((int64_t)P.k_steps * (rank + 1) / P.splits);
    const Guard g{P.status, P.timeout_ns, abort_flag};

    griddep_wait();
    int expert = 0, rows = 0;
    int64_t row0 = 0, atom_row = 0;
    bool live = true;
    float alpha = P.epi.alpha;
    if (P.offsets) {
        live = mx_expert_block(P.offsets, P.num_experts, 128, tm, lane, &expert, &row0, &rows, &atom_row);
        if (live && P.expert_alpha) alpha *= P.expert_alpha[expert];
    } else {
        row0 = tm * 128;
        rows = (int)(P.epi.M - row0 < 128 ? P.epi.M - row0 : 128);
        atom_row = tm;
    }
    const int64_t n0 = tn * BN;

    bool ok = live;
    if (live && warp == 0) {
        if (lane == 0) {
            for (int k = k0; k < k1; ++k) {
                const int i = k - k0, s = i % S;
                if (!wait_bar(&empty[s], ((i / S) & 1) ^ 1, g, SITE_PRODUCER_EMPTY)) break;
                uint8_t* a = smem + (size_t)s * stage_bytes;
                uint8_t* b = a + a_bytes;
                uint8_t* sa = b + Cfg::B_BYTES;
                mbar_arrive_expect_tx(&full[s], stage_bytes);
                tma_load_2d(a, &tmA, &full[s], k * 128, (int32_t)row0);
                tma_load_2d(sa, &tmSA, &full[s], k * (int)(Cfg::S_BYTES / 8), (int32_t)atom_row);
                if (P.b3d) {
                    tma_load_3d(b, &tmB, &full[s], k * 128, (int32_t)n0, expert);
                    tma_load_3d(sa + Cfg::S_BYTES, &tmSB, &full[s], k * (int)(Cfg::S_BYTES / 8), (int32_t)(n0 / 128), expert);
                } else {
                    tma_load_2d(b, &tmB, &full[s], k * 128, (int32_t)n0);
                    tma_load_2d(sa + Cfg::S_BYTES, &tmSB, &full[s], k * (int)(Cfg::S_BYTES / 8), (int32_t)(n0 / 128));
                }
            }
        }
        __syncwarp();
    } else if (live && warp == 1) {
        if (lane == 0) {
            const uint32_t sfa = tmem + BN, sfb = tmem + BN + 32;  // two buffers of 16 columns each
            const uint32_t sfb_off = (uint32_t)(n0 % 128) / 32;
            for (int k = k0; k < k1; ++k) {
                const int i = k - k0, s = i % S;
                if (!wait_bar(&full[s], (i / S) & 1, g, SITE_MMA_FULL)) {
                    ok = false;
                    break;
                }
                // the scale buffer's previous readers, the MMAs of step i - 2
                if (i >= 2 && !wait_bar(&empty[(i - 2) % S], ((i - 2) / S) & 1, g, SITE_MMA_OPERAND)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t a = smem_u32(smem + (size_t)s * stage_bytes);
                const uint32_t b = a + a_bytes, sa = b + Cfg::B_BYTES, sb = sa + Cfg::S_BYTES;
                const uint32_t ta = sfa + (i & 1) * 16, tb = sfb + (i & 1) * 16;
                const int na = P.k_atoms - 4 * k < 4 ? P.k_atoms - 4 * k : 4;  // 64-wide steps that exist
#pragma unroll
                for (int q = 0; q < Cfg::S_ATOMS; ++q) {
                    tmem_cp_scales(ta + 4 * q, make_scale_desc(sa + MX_ATOM_BYTES * q));
                    tmem_cp_scales(tb + 4 * q, make_scale_desc(sb + MX_ATOM_BYTES * q));
                }
                const uint64_t ad = make_sw128_kmajor_desc(a), bd = make_sw128_kmajor_desc(b);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= na) break;
                    const uint32_t acc = (i > 0 || q > 0) ? 1u : 0u;
                    if constexpr (NVF4)
                        umma_mx_ss<true>(tmem, ad + 2 * q, bd + 2 * q, P.idesc, ta + 4 * q, tb + 4 * q + sfb_off, acc);
                    else {
                        // an atom's four scales cover two instructions: bytes 0-1, then 2-3
                        const uint32_t id = (q & 1) * 2u;
                        umma_mx_ss<false>(tmem, ad + 2 * q, bd + 2 * q, P.idesc | (id << 29) | (id << 4),
                                          ta + 4 * (q / 2), tb + 4 * (q / 2) + sfb_off, acc);
                    }
                }
                umma_commit(&empty[s]);
            }
            if (ok) umma_commit(tfull);
        }
        __syncwarp();
    }
    // every thread learns whether the accumulator is complete
    if (live) {
        ok = wait_bar(tfull, 0, g, SITE_EPI_TMEM_FULL);
        tc_fence_after_sync();
    }
    const bool all_ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (live && !all_ok) {
        // gave up: let copies in flight land and issued MMAs finish before shared memory and TMEM go
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    const uint32_t tb = tmem + ((uint32_t)(warp * 32) << 16);
    const int wrows = rows - warp * 32 < 0 ? 0 : (rows - warp * 32 < 32 ? rows - warp * 32 : 32);
    if (P.splits == 1) {
        if (all_ok && wrows > 0) {
            float* stage = reinterpret_cast<float*>(smem) + warp * (32 * 33);
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                if (n0 + 32 * c >= P.epi.N) break;
                float v[32];
                tmem_load_chunk<32>(tb + 32 * c, v);
                mx_store_block(P.epi, P.vec32, alpha, row0 + warp * 32, wrows, n0 + 32 * c, v, stage, lane);
            }
        }
    } else {
        // partial tile -> shared memory, [quad of columns][row]
        if (all_ok && wrows > 0) {
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                float v[32];
                tmem_load_chunk<32>(tb + 32 * c, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4*>(smem + (8 * c + j) * Cfg::PART_PITCH + (warp * 32 + lane) * 16) =
                        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
        cluster_sync();
        if (all_ok) {
            constexpr int QUADS = BN / 4;
            const int q0 = QUADS * rank / P.splits, nq = QUADS * (rank + 1) / P.splits - q0;
            const EpiParams& e = P.epi;
            EpiArith ar = epi_arith(e);
            ar.alpha = alpha;
            const uint32_t base = smem_u32(smem);
            for (int t = threadIdx.x; t < rows * nq; t += 128) {
                const int q = q0 + t % nq, r = t / nq;
                const int64_t n = n0 + 4 * q, m = row0 + r;
                if (n >= e.N) continue;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int z = 0; z < P.splits; ++z) {  // in K order
                    const float4 p = ld_cluster_f4(mapa_shared(base + q * Cfg::PART_PITCH + r * 16, z));
                    sum.x += p.x;
                    sum.y += p.y;
                    sum.z += p.z;
                    sum.w += p.w;
                }
                const float a4[4] = {sum.x, sum.y, sum.z, sum.w};
                float x[4];
                const int have = e.N - n < 4 ? (int)(e.N - n) : 4;
                with_epi_act(e, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float c = (e.beta != 0.0f && j < have) ? ld_elem(e.C, e.d_type, m * e.ldc + n + j) : 0.0f;
                        x[j] = epi_value<ACT>(ar, a4[j], c, ACT >= 0 ? bias_at(ar, n + j) : 0.0f);
                    }
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
        cluster_sync();  // no CTA leaves while another reads its partial tile
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
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
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = Cfg::smem_bytes(p.a_rows, p.stages);
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
