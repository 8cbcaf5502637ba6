// Int8 product on the tensor cores, one tile of 128 channels x up to TN tokens per
// cluster.
//
// A stage holds one K-step: 128 codes (one 128-byte swizzle row) of 128 channels
// and of the tile's tokens.  Groups of four warps take the stages in turn, or their
// halves, and turn their codes into f16 operands: the channels' into a slot of TMEM, the
// tokens' into one of shared memory.  The accumulator has two buffers of TN columns; after 16
// slots (1024 products) other warps add the full one to 32-bit sums in their registers
// while the MMAs go on in the other.
//
// The tile's K-steps are shared out over the `splits` CTAs of a cluster, whose sums
// meet as in mx_exchange.h: every CTA finishes its share of the tokens.  Integer
// sums, so the order does not matter.
//
//   warp 0     TMA producer     warp 1   MMAs     warps 2-3  fetch the tile's C
//   then 4 or 8 warps of sums, 8 or 16 of operands (up to 32 tokens two CTAs share an
//   SM, each with half as many); the epilogue is all warps'
// Measured (back-to-back launches, cold operands): up to 32 tokens 16x4096x14336 16 us,
// 32 rows by 8 experts of 14336 x 4096 83 us (5.7 TB/s); up to 128 tokens 256x4096x4096
// 22.0 us in two K slices, 128x14336x4096 28.7 and 512x4096x4096 28.4 (the CTA pair, which is
// chosen for these two, 27.5 and 26.3). A K-step is a chain of waits of half a microsecond
// (without conversion and MMAs 77x11002x4104 took 23 us of 29), set-up, first data and
// end of a CTA 5 to 7.5 us.
#include <atomic>

#include "mx_exchange.h"
#include "s8_tile.cuh"

namespace qg {

namespace {

template <int TN>
struct Cfg {
    static constexpr bool WIDE = TN > 32;
    static constexpr int CTAS = WIDE ? 1 : 2;       // per SM
    static constexpr int SUM_WARPS = WIDE ? 8 : 4;
    static constexpr int GROUPS = WIDE ? 4 : 2;     // of operand warps: two take a stage's halves, or one both
    static constexpr int HALVES = WIDE ? 1 : 2;
    static constexpr int THREADS = 128 + 32 * SUM_WARPS + 128 * GROUPS;
    static constexpr int COLS = TN / (SUM_WARPS / 4);  // of a warp's sums
    static constexpr int MAX_SLOTS = WIDE ? 8 : 6;
    QG_HD static int slots(int tn) { return WIDE ? (tn <= 96 ? 8 : 4) : 6; }
    static constexpr int MAX_STAGES = 12;
    static constexpr uint32_t W_BYTES = 128 * 128;
    static constexpr uint32_t AUX_BYTES = (2 * MAX_STAGES + MAX_SLOTS + 6) * 8 + 16 + (256 + TN) * 4;
    static constexpr uint32_t BUDGET = 233472 / CTAS - 1024;  // of a CTA's shared memory
    static constexpr uint32_t TMEM_COLS = WIDE ? 512 : 256;
    static_assert(2 * TN + 32 * MAX_SLOTS <= TMEM_COLS && MAX_SLOTS % GROUPS == 0, "");
    // The ring holds as many stages as there is room for, by the tile's tokens: what
    // is in flight bounds the kernel (with 4 stages of 26 KB a K-step took 0.55 us,
    // whatever the other warps did).  Their number is even: then a stage is always read by
    // the same groups, and none meets a phase of full[] out of turn.
    QG_HD static uint32_t stage_bytes(int tn) { return W_BYTES + (uint32_t)tn * 128u; }
    QG_HD static uint32_t slot_bytes(int tn) { return (uint32_t)tn * 128u; }
    QG_HD static int stages(int tn) {
        const int n = (int)((BUDGET - 1024 - AUX_BYTES - slots(tn) * slot_bytes(tn)) / stage_bytes(tn));
        return (n < MAX_STAGES ? n : MAX_STAGES) / 2 * 2;
    }
    QG_HD static uint32_t ring_bytes(int tn) { return (uint32_t)stages(tn) * stage_bytes(tn) + slots(tn) * slot_bytes(tn); }
    QG_HD static uint32_t sum_bytes(int tn) { return (uint32_t)tn * 512u; }  // [token][channel], in the ring when it is idle
    static uint32_t smem_bytes(int tn) { return 1024 + ring_bytes(tn) + AUX_BYTES; }
    // registers of a thread: at launch, and by role where they differ
    static constexpr int REGS_LAUNCH = WIDE ? 72 : 64, REGS_SUMS = 104, REGS_OPERANDS = 56, REGS_REST = 56;
    static_assert(!WIDE || 32 * SUM_WARPS * REGS_SUMS + 128 * GROUPS * REGS_OPERANDS + 128 * REGS_REST <= THREADS * REGS_LAUNCH,
                  "what was launched is shared out");
};
constexpr int SLOT_CHUNK = 2 * S8_CHUNK;  // slots whose sums fp32 holds exactly

// The steps of mx_exchange.h for sums: shares are runs of tokens, `each` but for the
// last ones.
struct SumsLink {
    uint64_t *idle, *part;
    volatile uint32_t* warning;
    uint32_t parts, recv;
    int splits, rank, rows, each;
    const Guard& g;
    __device__ __forceinline__ int first(int z) const { return z * each < rows ? z * each : rows; }
    __device__ __forceinline__ int count(int z) const { return first(z + 1) - first(z); }
    __device__ __forceinline__ void expect() { mbar_arrive_expect_tx(part, (uint32_t)(splits * count(rank)) * 512u); }
    // (nothing is published: the arrivals are relaxed)
    __device__ __forceinline__ void announce(int z) { mbar_arrive_remote_relaxed(mapa_shared(smem_u32(idle), z)); }
    __device__ __forceinline__ bool await_announced() { return wait_bar_cluster_drain(idle, 0, g); }
    __device__ __forceinline__ void send(int z) {
        const int n = count(z);
        if (n)
            bulk_s2cluster(mapa_shared(recv + (uint32_t)(rank * n) * 512u, z), parts + (uint32_t)first(z) * 512u, (uint32_t)n * 512u,
                           mapa_shared(smem_u32(part), z));
    }
    __device__ __forceinline__ bool await_shares() { return wait_bar_cluster_drain(part, 0, g); }
    __device__ __forceinline__ void warn(int z) { st_cluster_fence(mapa_shared(smem_u32((const void*)warning), z), 1u); }
    __device__ __forceinline__ void arrive() { cluster_arrive_relaxed(); }
    __device__ __forceinline__ void wait() { cluster_wait(); }
    __device__ __forceinline__ bool warned() { return *warning != 0; }
    __device__ __forceinline__ void settle() { mx_settle(); }
};

template <int TN>
__global__ void __launch_bounds__(Cfg<TN>::THREADS, Cfg<TN>::CTAS)
    s8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ S8GemmParams P) {
    using C = Cfg<TN>;
    constexpr int G = C::GROUPS;
    const int splits = P.splits, tn = P.tile_rows;
    const int S = C::stages(tn), NS = C::slots(tn);
    const uint32_t stage_bytes = C::stage_bytes(tn), slot_bytes = C::slot_bytes(tn), ring_bytes = C::ring_bytes(tn);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* slots = smem + S * stage_bytes;
    int32_t* sums = reinterpret_cast<int32_t*>(smem);  // once the ring is idle
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring_bytes);
    uint64_t* empty = full + C::MAX_STAGES;  // a stage's codes have been read
    uint64_t* ready = empty + C::MAX_STAGES;  // a K-step's operands are in its two slots
    uint64_t* slot_free = ready + C::MAX_SLOTS / 2;
    uint64_t* tfull = slot_free + C::MAX_SLOTS / 2;  // an accumulator buffer is complete
    uint64_t* tempty = tfull + 2;      // ... and in the sums
    uint64_t* idle = tempty + 2;       // every CTA of the cluster is through with its ring
    uint64_t* part = idle + 1;         // the sums' shares have arrived
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* warning = tmem_slot + 2;  // a CTA of the cluster has given up
    // what the epilogue multiplies and adds: fetched while the main loop runs
    float* channel_factor = reinterpret_cast<float*>(tmem_slot + 4);
    float* channel_bias = channel_factor + 128;
    float* token_factor = channel_bias + 128;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 8 / C::HALVES);
        }
        for (int s = 0; s < NS / 2; ++s) {
            mbar_init(&ready[s], 8 / C::HALVES);
            mbar_init(&slot_free[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], C::SUM_WARPS);
        }
        mbar_init(idle, (uint32_t)splits);
        mbar_init(part, 1);
        *abort_flag = 0;
        *warning = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (splits > 1) cluster_sync();  // every CTA's barriers exist before another's copies complete on them
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot, tmem_w = tmem + 2 * TN;
    griddep_launch_dependents();

    const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
    const int64_t tile = blockIdx.x / splits;
    const int64_t tm = tile % P.tiles_m, tw = tile / P.tiles_m;
    const int k0 = (int)((int64_t)P.k_steps * rank / splits), nk = (int)((int64_t)P.k_steps * (rank + 1) / splits) - k0;
    const int nslots = 2 * nk;
    const int64_t n0 = tw * 128;
    const Guard g{P.status, P.timeout_ns, abort_flag};
    if (!P.offsets && warp == 0 && lane == 0) {
        // warm L2 with the first stages of the weights while the previous kernel
        // in the stream finishes (a hint: L2 is where memory is coherent)
        for (int k = 0; k < nk && k < S; ++k) tma_prefetch_l2_2d(&tmB, (k0 + k) * S8_KSTEP, (int32_t)n0);
    }
    griddep_wait();
    int expert = 0, rows = 0;
    int64_t row0 = 0, atom_row = 0;
    bool live = true;
    if (P.offsets) {
        live = mx_expert_block(P.offsets, P.num_experts, P.epi.M, tn, tm, lane, &expert, &row0, &rows, &atom_row);
        live = live && rows > 0;
    } else {
        row0 = tm * tn;
        rows = (int)(P.epi.M - row0 < tn ? P.epi.M - row0 : tn);
    }

    bool ok = live;
    int32_t sum[C::COLS];  // (of the warps that add up)
    const int sum_half = (warp - 4) / 4;  // which of the columns
    if (warp < 4) {
        if constexpr (C::WIDE) regs_down<C::REGS_REST>();
        if (live && warp == 0) {
            int s = 0;
            uint32_t ph = 1;
            for (int i = 0; i < nk; ++i) {
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&empty[s], ph, g, SITE_PRODUCER_EMPTY));
                if (!ok) break;
                uint8_t* w = smem + (uint32_t)s * stage_bytes;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[s], stage_bytes);
                    if (P.b3d)
                        tma_load_3d(w, &tmB, &full[s], (k0 + i) * S8_KSTEP, (int32_t)n0, expert);
                    else
                        tma_load_2d(w, &tmB, &full[s], (k0 + i) * S8_KSTEP, (int32_t)n0);
                    tma_load_2d(w + C::W_BYTES, &tmA, &full[s], (k0 + i) * S8_KSTEP, (int32_t)row0);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        } else if (live && warp == 1) {
            const uint64_t xd0 = make_sw128_kmajor_desc(smem_u32(slots));
            int pair = 0;  // of slots
            uint32_t ph = 0, chunk = 0;
            for (int j0 = 0; ok && j0 < nslots; j0 += SLOT_CHUNK, ++chunk) {
                const uint32_t b = chunk & 1, d = tmem + TN * b;
                const int n = nslots - j0 < SLOT_CHUNK ? nslots - j0 : SLOT_CHUNK;
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&tempty[b], ((chunk >> 1) & 1) ^ 1, g, SITE_MMA_TMEM_EMPTY));
                for (int j = 0; ok && j < n; j += 2) {
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(&ready[pair], ph, g, SITE_MMA_OPERAND));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t xd = xd0 + (uint64_t)((uint32_t)pair * (slot_bytes / 8));
                    const uint32_t wa = tmem_w + 64 * pair;
                    if (elect_one()) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) umma_f16_ts(d, wa + 8 * q, xd + 2 * q, P.idesc, q ? 1u : (uint32_t)j);
#pragma unroll
                        for (int q = 0; q < 4; ++q) umma_f16_ts(d, wa + 32 + 8 * q, xd + slot_bytes / 16 + 2 * q, P.idesc, 1u);
                        umma_commit(&slot_free[pair]);
                        if (j == n - 2) umma_commit(&tfull[b]);
                    }
                    __syncwarp();
                    if (++pair == NS / 2) {
                        pair = 0;
                        ph ^= 1;
                    }
                }
            }
        } else if (live && warp > 1) {
            const EpiArith ar = epi_arith(P.epi);
            for (int i = threadIdx.x - 64; i < 128; i += 64) {
                channel_factor[i] = n0 + i < P.epi.N ? s8_channel_factor(P, expert, n0 + i) : 0.0f;
                channel_bias[i] = bias_at(ar, n0 + i);
            }
            for (int i = threadIdx.x - 64; i < rows; i += 64) token_factor[i] = s8_token_factor(P, row0 + i);
            if (P.epi.beta != 0.0f && n0 < P.epi.N)
                for (int r = threadIdx.x - 64; r < rows; r += 64) mx_prefetch_c(P.epi, row0 + r, n0, P.epi.N - n0 < 128 ? P.epi.N - n0 : 128);
        }
    } else if (warp < 4 + C::SUM_WARPS) {
        if constexpr (C::WIDE) regs_up<C::REGS_SUMS>();
        const uint32_t taddr = tmem + sum_half * C::COLS + ((uint32_t)(warp % 4 * 32) << 16);
        const int cols = rows - sum_half * C::COLS;
#pragma unroll
        for (int q = 0; q < C::COLS; ++q) sum[q] = 0;
        uint32_t chunk = 0;
        for (int j0 = 0; ok && j0 < nslots; j0 += SLOT_CHUNK, ++chunk) {
            const uint32_t b = chunk & 1;
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&tfull[b], (chunk >> 1) & 1, g, SITE_EPI_TMEM_FULL));
            if (!ok) break;
            tc_fence_after_sync();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < C::COLS; q += 16)
                if (q < cols) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(taddr + TN * b + q, v);
#pragma unroll
                    for (int r = 0; r < 16; ++r) sum[q + r] += __float2int_rn(__uint_as_float(v[r]));
                }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
        }
    } else {
        if constexpr (C::WIDE) regs_down<C::REGS_OPERANDS>();
        const int group = (warp - 4 - C::SUM_WARPS) / 4, half = C::HALVES == 1 ? group & 1 : 0, first = C::HALVES == 1 ? group / 2 : group;
        const uint32_t taddr = tmem_w + 32 * half + ((uint32_t)(warp % 4 * 32) << 16), out = smem_u32(slots) + half * slot_bytes;
        const HalfStage<TN / 8> codes(half, warp % 4 * 32 + lane, threadIdx.x & 127);
        // (The phase of slot_free before the one waited for has ended: this group has seen the
        // MMAs of K-step i - 2 - NS / 2 or later end.)
        int s = first, pair = first;
        uint32_t ph = 0, sph = 1;
        for (int i = first; ok && i < nk; i += 2) {
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[s], ph, g, SITE_DQ_RAW));
            if (!ok) break;
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&slot_free[pair], sph, g, SITE_DQ_EMPTY));
            if (!ok) break;
            tc_fence_after_sync();
            __syncwarp();
            const uint32_t w = smem_u32(smem) + (uint32_t)s * stage_bytes, ta = taddr + 64 * pair, to = out + 2 * pair * slot_bytes;
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) codes.convert(w, w + C::W_BYTES, ta + 32 * h, to + h * slot_bytes, tn, 64u * h);
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[s]);
                mbar_arrive(&ready[pair]);
            }
            s += 2;
            if (s >= S) {
                s -= S;
                ph ^= 1;
            }
            pair += 2;
            if (pair >= NS / 2) {
                pair -= NS / 2;
                sph ^= 1;
            }
        }
    }
    bool all_ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (live && !all_ok) {
        // gave up: let copies in flight land and issued MMAs finish before shared memory and TMEM go
        mx_settle();
    }
    if (live && warp >= 4 && warp < 4 + C::SUM_WARPS) {
        int32_t* mine = sums + sum_half * C::COLS * 128 + warp % 4 * 32 + lane;
#pragma unroll
        for (int q = 0; q < C::COLS; ++q)
            if (sum_half * C::COLS + q < rows) mine[q * 128] = sum[q];
    }
    if constexpr (C::WIDE) {  // the epilogue is everybody's again
        if (warp >= 4 && warp < 4 + C::SUM_WARPS)
            regs_down<C::REGS_LAUNCH>();
        else
            regs_up<C::REGS_LAUNCH>();
    }
    if (splits > 1) fence_proxy_async_smem();  // the sums are visible to the bulk copies
    __syncthreads();
    uint8_t* recv = smem + C::sum_bytes(tn);
    // every thread keeps to four channels
    const int64_t n = n0 + 4 * lane;
    EpiArith ar = epi_arith(P.epi);
    ar.alpha = 1.0f;
    S8Channels ch;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        ch.scale[j] = channel_factor[4 * lane + j];
        ch.bias[j] = channel_bias[4 * lane + j];
    }
    if (splits == 1) {
        if (all_ok)
            for (int m = warp; m < rows; m += C::THREADS / 32)
                s8_finish4(P, ar, ch, token_factor[m], row0 + m, n, reinterpret_cast<const int4*>(sums + m * 128)[lane]);
    } else if (live) {
        // (whether this CTA's part is right or not: the others wait for it)
        SumsLink link{idle, part, warning, smem_u32(sums), smem_u32(recv), splits, rank, rows, (rows + splits - 1) / splits, g};
        ok = mx_exchange(link, splits, threadIdx.x == 0);
        all_ok = __syncthreads_and(all_ok && ok ? 1 : 0) != 0;
        if (all_ok) {
            const int count = link.count(rank), first = link.first(rank);
            for (int m = warp; m < count; m += C::THREADS / 32) {
                int4 sum = make_int4(0, 0, 0, 0);
                for (int z = 0; z < splits; ++z) {
                    const int4 p = reinterpret_cast<const int4*>(recv + (uint32_t)(z * count + m) * 512u)[lane];
                    sum.x += p.x;
                    sum.y += p.y;
                    sum.z += p.z;
                    sum.w += p.w;
                }
                s8_finish4(P, ar, ch, token_factor[first + m], row0 + first + m, n, sum);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    // shared memory goes only when nobody will read or write it any more
    if (live && splits > 1) {
        SumsLink link{idle, part, warning, 0, 0, splits, rank, 0, 0, g};
        mx_exchange_leave(link);
    }
}

template <int TN>
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
        e = cudaFuncGetAttributes(&a, s8_gemm_kernel<TN>);
        if (e != cudaSuccess) return e;
        if (Cfg<TN>::WIDE && a.numRegs != Cfg<TN>::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(s8_gemm_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<TN>::BUDGET);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return cudaSuccess;
}

template <int TN>
cudaError_t launch_t(const S8Maps& m, const S8GemmParams& p, int grid, cudaStream_t st) {
    const cudaError_t e = configure<TN>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Cfg<TN>::THREADS);
    cfg.dynamicSmemBytes = Cfg<TN>::smem_bytes(p.tile_rows);
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
    return cudaLaunchKernelEx(&cfg, s8_gemm_kernel<TN>, m.a, m.b, p);
}

}  // namespace

cudaError_t launch_s8_gemm(int width, const S8Maps& m, const S8GemmParams& p, int grid, cudaStream_t st) {
    if (p.tile_rows < 16 || p.tile_rows > width || p.tile_rows % 16) return cudaErrorInvalidValue;
    switch (width) {
        case 32: return launch_t<32>(m, p, grid, st);
        case 128: return launch_t<128>(m, p, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

bool s8_gemm_usable(int width) {
    if ((width == 32 ? configure<32>() : configure<128>()) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

}  // namespace qg
