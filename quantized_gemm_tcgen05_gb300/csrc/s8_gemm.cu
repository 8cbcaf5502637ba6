// Int8 product on the tensor cores, one tile of 128 channels x up to TN tokens per
// cluster.
//
// A stage holds one K-step: 128 codes (one 128-byte swizzle row) of 128 channels
// and of the tile's tokens.  Two groups of four warps take the K-steps in turn and
// turn codes into f16 operands: the channels' into a slot of TMEM, the tokens' into
// a slot of shared memory.  The accumulator has two buffers of TN columns; after 8
// K-steps (1024 products) four warps add the full one to 32-bit sums in shared memory
// while the MMAs go on in the other.
//
// The tile's K-steps are shared out over the `splits` CTAs of a cluster, whose sums
// meet as in mx_exchange.h: every CTA finishes its share of the tokens.  Integer
// sums, so the order does not matter.
//
//   warp 0      TMA producer          warps 4-7   sums
//   warp 1      MMAs                  warps 8-15  f16 operands
//   warps 2-3   fetch the tile's C    all         epilogue
#include <atomic>

#include "mx_exchange.h"
#include "s8_tile.cuh"

namespace qg {

namespace {

constexpr int THREADS = 512;

template <int TN>
struct Cfg {
    static constexpr int CTAS = TN == 32 ? 2 : 1;   // per SM
    static constexpr int STAGES = 3;
    static constexpr int SLOTS = TN == 32 ? 3 : 2;  // f16 operands
    static constexpr uint32_t W_BYTES = 128 * 128, X_BYTES = TN * 128, STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr uint32_t SLOT_BYTES = TN * 256;
    static constexpr uint32_t RING_BYTES = STAGES * STAGE_BYTES + SLOTS * SLOT_BYTES;
    static constexpr uint32_t SUM_BYTES = TN * 512;  // [token][channel]
    static constexpr uint32_t AUX_BYTES = (2 * STAGES + 2 * SLOTS + 6) * 8 + 16;
    static constexpr uint32_t SMEM_BYTES = 1024 + RING_BYTES + SUM_BYTES + AUX_BYTES;
    static constexpr uint32_t TMEM_COLS = TN == 32 ? 256 : 512;
    static_assert(2 * TN + 64 * SLOTS <= TMEM_COLS && SMEM_BYTES <= 232448 && CTAS * (SMEM_BYTES + 1024) <= 233472, "");
    static_assert(STAGES >= SLOTS, "a free slot tells that the stage's last use is over");
    static_assert((TN + 8) * 512 <= RING_BYTES, "the shares received");
};

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
__global__ void __launch_bounds__(THREADS, Cfg<TN>::CTAS)
    s8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ S8GemmParams P) {
    using C = Cfg<TN>;
    constexpr int S = C::STAGES, NS = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* slots = smem + S * C::STAGE_BYTES;
    int32_t* sums = reinterpret_cast<int32_t*>(smem + C::RING_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING_BYTES + C::SUM_BYTES);
    uint64_t* empty = full + S;
    uint64_t* ready = empty + S;    // a slot's operands are there (4 warps)
    uint64_t* slot_free = ready + NS;
    uint64_t* tfull = slot_free + NS;  // an accumulator buffer is complete
    uint64_t* tempty = tfull + 2;      // ... and in the sums (4 warps)
    uint64_t* idle = tempty + 2;       // every CTA of the cluster is through with its ring
    uint64_t* part = idle + 1;         // the sums' shares have arrived
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* warning = tmem_slot + 2;  // a CTA of the cluster has given up

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int splits = P.splits, tn = P.tile_rows;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(&ready[s], 4);
            mbar_init(&slot_free[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 4);
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
    const int chunks = (nk + S8_CHUNK - 1) / S8_CHUNK;

    bool ok = live;
    if (live && warp == 0) {
        const uint32_t bytes = C::W_BYTES + (uint32_t)tn * 128u;
        int s = 0;
        uint32_t ph = 1;
        for (int i = 0; i < nk; ++i) {
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&empty[s], ph, g, SITE_PRODUCER_EMPTY));
            if (!ok) break;
            uint8_t* w = smem + (uint32_t)s * C::STAGE_BYTES;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], bytes);
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
        int slot = 0;
        uint32_t ph = 0;
        for (int i = 0; i < nk; ++i) {
            const int c = i / S8_CHUNK, b = c & 1;
            if (i % S8_CHUNK == 0) {
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&tempty[b], ((c >> 1) & 1) ^ 1, g, SITE_MMA_TMEM_EMPTY));
                if (!ok) break;
            }
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&ready[slot], ph, g, SITE_MMA_OPERAND));
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t xd = xd0 + (uint64_t)((uint32_t)slot * (C::SLOT_BYTES / 16));
            const uint32_t wa = tmem_w + 64 * slot, d = tmem + TN * b;
            const uint32_t acc = i % S8_CHUNK ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    umma_f16_ts(d, wa + 8 * q, xd + (uint64_t)((q / 4) * tn * 8 + 2 * (q % 4)), P.idesc, q ? 1u : acc);
                umma_commit(&slot_free[slot]);
                if (i % S8_CHUNK == S8_CHUNK - 1 || i == nk - 1) umma_commit(&tfull[b]);
            }
            __syncwarp();
            if (++slot == NS) {
                slot = 0;
                ph ^= 1;
            }
        }
    } else if (live && warp < 4) {
        if (P.epi.beta != 0.0f && n0 < P.epi.N)
            for (int r = threadIdx.x - 64; r < rows; r += 64) mx_prefetch_c(P.epi, row0 + r, n0, P.epi.N - n0 < 128 ? P.epi.N - n0 : 128);
    } else if (live && warp < 8) {
        const uint32_t quarter = (uint32_t)(warp % 4 * 32) << 16;
        int32_t* mine = sums + warp % 4 * 32 + lane;
        for (int c = 0; c < chunks; ++c) {
            const int b = c & 1;
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&tfull[b], (c >> 1) & 1, g, SITE_EPI_TMEM_FULL));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int j = 0; j < rows; j += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + TN * b + j + quarter, v);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int32_t x = __float2int_rn(__uint_as_float(v[q]));
                    int32_t* to = mine + (j + q) * 128;
                    *to = c ? *to + x : x;
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
        }
    } else if (live) {
        const int group = (warp - 8) / 4, thread = threadIdx.x & 127, row = warp % 4 * 32 + lane;
        const uint32_t quarter = (uint32_t)(warp % 4 * 32) << 16;
        for (int i = group; i < nk; i += 2) {
            const int s = i % S, slot = i % NS;
            // The slot first: it is free when the MMAs of K-step i - NS are done, and so
            // when K-step i - S has landed.  A wait for this phase of full[s] that came
            // before its last one had ended would not wait: stages are used by both
            // groups, and copies may land out of order.
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&slot_free[slot], ((i / NS) & 1) ^ 1, g, SITE_DQ_EMPTY));
            if (!ok) break;
            ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[s], (i / S) & 1, g, SITE_DQ_RAW));
            if (!ok) break;
            tc_fence_after_sync();
            __syncwarp();
            const uint8_t* w = smem + (uint32_t)s * C::STAGE_BYTES;
            s8_tokens_to_f16(w + C::W_BYTES, slots + slot * C::SLOT_BYTES, tn, thread);
            s8_weights_to_tmem(w, tmem_w + 64 * slot + quarter, row);
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[s]);
                mbar_arrive(&ready[slot]);
            }
        }
    }
    bool all_ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (live && !all_ok) {
        // gave up: let copies in flight land and issued MMAs finish before shared memory and TMEM go
        mx_settle();
    }
    // every thread keeps to four channels
    const int64_t n = n0 + 4 * lane;
    EpiArith ar = epi_arith(P.epi);
    ar.alpha = 1.0f;
    if (splits == 1) {
        if (all_ok) {
            const S8Channels ch = s8_channels(P, ar, expert, n);
            for (int m = warp; m < rows; m += THREADS / 32) s8_finish4(P, ar, ch, row0 + m, n, reinterpret_cast<const int4*>(sums + m * 128)[lane]);
        }
    } else if (live) {
        fence_proxy_async_smem();  // the sums are visible to the bulk copies
        __syncthreads();
        // (whether this CTA's part is right or not: the others wait for it)
        SumsLink link{idle, part, warning, smem_u32(sums), smem_u32(smem), splits, rank, rows, (rows + splits - 1) / splits, g};
        ok = mx_exchange(link, splits, threadIdx.x == 0);
        all_ok = __syncthreads_and(all_ok && ok ? 1 : 0) != 0;
        if (all_ok) {
            const S8Channels ch = s8_channels(P, ar, expert, n);
            const int count = link.count(rank), first = link.first(rank);
            for (int m = warp; m < count; m += THREADS / 32) {
                int4 sum = make_int4(0, 0, 0, 0);
                for (int z = 0; z < splits; ++z) {
                    const int4 p = reinterpret_cast<const int4*>(smem + (uint32_t)(z * count + m) * 512u)[lane];
                    sum.x += p.x;
                    sum.y += p.y;
                    sum.z += p.z;
                    sum.w += p.w;
                }
                s8_finish4(P, ar, ch, row0 + first + m, n, sum);
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
cudaError_t launch_t(const S8Maps& m, const S8GemmParams& p, int grid, cudaStream_t st) {
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(s8_gemm_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<TN>::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<TN>::SMEM_BYTES;
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

}  // namespace qg
