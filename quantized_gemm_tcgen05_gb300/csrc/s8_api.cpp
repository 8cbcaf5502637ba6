// The C ABI of the int8 products (include/gemm_s8.h): checks of arguments,
// choice of kernel, launch.  Host code only.
#include "gemm_s8.h"

#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "api_checks.h"
#include "mx_gemm.h"
#include "s8_params.h"

using namespace qg;

namespace {

// Rows of codes that the tensor-memory accelerator and 16-byte loads can read.
int check_s8(const gemm_layout_t* d, int64_t lines) {
    if (d->type != GEMM_S8) return GEMM_ERR_UNSUPPORTED;
    if (d->ld % 16) return GEMM_ERR_INVALID_ARG;
    if (d->num > 1 && (d->batch_stride % 16 || d->batch_stride < lines * d->ld)) return GEMM_ERR_INVALID_ARG;
    return offsets_fit(d, lines) ? GEMM_OK : GEMM_ERR_UNSUPPORTED;
}

int check_product(gemm_handle_t h, const gemm_op_t* op, float alpha, const void* A, const gemm_layout_t* Ad,
                  const float* SA, const void* B, const gemm_layout_t* Bd, const float* SB, float beta, const void* C,
                  const gemm_layout_t* Cd, void* D, const gemm_layout_t* Dd, const int32_t* offsets, int32_t experts,
                  S8GemmParams* out) {
    if (!op || !Ad || !Bd || !Dd) return GEMM_ERR_INVALID_ARG;
    const int32_t act = op->epilogue;
    if (act & ~(GEMM_EPILOGUE_BIAS | GEMM_EPILOGUE_RELU | GEMM_EPILOGUE_GELU)) return GEMM_ERR_INVALID_ARG;
    if ((act & GEMM_EPILOGUE_RELU) && (act & GEMM_EPILOGUE_GELU)) return GEMM_ERR_INVALID_ARG;
    if (act & GEMM_EPILOGUE_BIAS) {
        if (!op->bias) return GEMM_ERR_INVALID_ARG;
        const int64_t bs = float_size(op->bias_type);
        if (!bs) return GEMM_ERR_UNSUPPORTED;
        if (!aligned(op->bias, (uintptr_t)bs) || !handle_device_pointer(h, op->bias)) return GEMM_ERR_INVALID_ARG;
    }
    if (op->dispatch < GEMM_DISPATCH_DEFAULT || op->dispatch > GEMM_DISPATCH_REUSE) return GEMM_ERR_INVALID_ARG;
    if (op->splitk < 0 || op->streamk < -1 || op->streamk > 1) return GEMM_ERR_INVALID_ARG;
    if (op->splitk > 1 && op->streamk == 1) return GEMM_ERR_INVALID_ARG;
    if (op->streamk == 1 || op->quant_a_group || op->quant_b_group || op->b_zero) return GEMM_ERR_UNSUPPORTED;
    if (op->splitk > 1 && op->splitk != 2 && op->splitk != 4 && op->splitk != 8) return GEMM_ERR_UNSUPPORTED;
    S8GemmParams p;
    memset(&p, 0, sizeof p);
    const int64_t M = Ad->rows, K = Ad->cols, N = Bd->cols;
    int rc;
    if ((rc = check_matrix(Ad, GEMM_ROW_MAJOR, M, K))) return rc;
    if ((rc = check_matrix(Bd, GEMM_COL_MAJOR, K, N))) return rc;
    if ((rc = check_matrix(Dd, GEMM_ROW_MAJOR, M, N))) return rc;
    if ((rc = check_s8(Ad, M)) || (rc = check_s8(Bd, N))) return rc;
    if (K > S8_MAX_K) return GEMM_ERR_UNSUPPORTED;
    const int64_t ds = float_size(Dd->type);
    if (!ds || !offsets_fit(Dd, M)) return GEMM_ERR_UNSUPPORTED;
    if (Ad->num != 1 || Dd->num != 1) return experts ? GEMM_ERR_INVALID_ARG : GEMM_ERR_UNSUPPORTED;
    if (Bd->num != (experts ? experts : 1)) return experts || Bd->num == 1 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_UNSUPPORTED;
    EpiParams& e = p.epi;
    if (beta != 0.0f) {
        if (!C || !Cd) return GEMM_ERR_INVALID_ARG;
        if ((rc = check_matrix(Cd, GEMM_ROW_MAJOR, M, N))) return rc;
        if (Cd->type != Dd->type || !offsets_fit(Cd, M)) return GEMM_ERR_UNSUPPORTED;
        if (Cd->num != 1) return GEMM_ERR_INVALID_ARG;
        e.C = C;
        e.ldc = Cd->ld;
    }
    e.D = D;
    e.ldd = Dd->ld;
    e.M = M;
    e.N = N;
    e.alpha = alpha;
    e.beta = beta;
    e.d_type = Dd->type;
    e.flags = act;
    e.bias = (act & GEMM_EPILOGUE_BIAS) ? op->bias : nullptr;
    e.bias_type = op->bias_type;
    e.status = handle_status(h);
    if (M > 0 && N > 0) {
        e.d_extent = (M - 1) * e.ldd + N;
        e.c_extent = e.C ? (M - 1) * e.ldc + N : 0;
        if (!D || !aligned(D, (uintptr_t)ds) || !handle_device_pointer(h, D)) return GEMM_ERR_INVALID_ARG;
        if (e.C && (!aligned(C, (uintptr_t)ds) || !handle_device_pointer(h, C))) return GEMM_ERR_INVALID_ARG;
        if (K > 0) {
            if (!A || !B || !aligned(A, 16) || !aligned(B, 16)) return GEMM_ERR_INVALID_ARG;
            if (!handle_device_pointer(h, A) || !handle_device_pointer(h, B)) return GEMM_ERR_INVALID_ARG;
            for (const float* s : {SA, SB})
                if (s && (!aligned(s, 4) || !handle_device_pointer(h, s))) return GEMM_ERR_INVALID_ARG;
        }
    }
    p.A = static_cast<const int8_t*>(A);
    p.B = static_cast<const int8_t*>(B);
    p.lda = Ad->ld;
    p.ldb = Bd->ld;
    p.b_bs = Bd->num > 1 ? Bd->batch_stride : 0;
    p.sa = SA;
    p.sb = SB;
    p.K = K;
    p.offsets = offsets;
    p.num_experts = experts;
    *out = p;
    return GEMM_OK;
}

// Token tiles: exact, or an upper bound over the splits into experts.
int64_t token_tiles(const S8GemmParams& p, int64_t rows) {
    if (!p.num_experts) return ceil_div(p.epi.M, rows);
    return std::min(p.epi.M / rows + p.num_experts, p.epi.M);
}

enum S8Kernel { S8_GEMV, S8_TILE, S8_PAIR };
struct S8Choice {
    S8Kernel kernel;
    int width;   // S8_TILE: 32 or 128 tokens a tile at most
    int rows;    // tokens of a tile
    int splits;
};

// Rows an expert has on average, or all.
int64_t rows_each(const S8GemmParams& p) { return p.num_experts ? ceil_div(p.epi.M, p.num_experts) : p.epi.M; }

// Clusters of two that the CTA-pair kernel keeps resident (asked once per device).
int pair_clusters(gemm_handle_t h) {
    static std::atomic<int> known[64];
    std::atomic<int>& k = known[handle_device(h) & 63];
    int n = k.load();
    if (n == 0) {
        n = std::max(0, std::min(s8_pair_max_clusters(), handle_sm_count(h) / 2)) + 1;
        k.store(n);
    }
    return n - 1;
}

// GEMM_FORCE_KERNEL=s8_gemv / s8_t32 / s8_t128 / s8_pair (the names gemm_last_choice prints,
// up to the slash) pins the kernel, for tests and sweeps.
bool forced_kernel(S8Choice* c) {
    const char* f = getenv("GEMM_FORCE_KERNEL");
    if (!f || strncmp(f, "s8_", 3)) return false;
    if (!strncmp(f, "s8_gemv", 7)) c->kernel = S8_GEMV;
    else if (!strncmp(f, "s8_pair", 7)) c->kernel = S8_PAIR;
    else c->kernel = S8_TILE, c->width = strncmp(f, "s8_t32", 6) == 0 ? 32 : 128;
    return true;
}

// Estimated time of a choice, microseconds.  Measured on GB300 (152 SMs), back-to-back
// launches, cold operands:
//   one tile, up to 32 tokens    5 us for set-up, first data and epilogue; a K-step of
//     128 0.40 us, 0.50 where two CTAs share an SM, 0.08 more with 32 tokens than with 16;
//     K slices 3 us (8x4096x4096 9.3 us in eight, 16x4096x14336 16.1 in eight, 22 in four,
//     256x4096x4096 24.5, 512x4096x4096 47.5)
//   one tile, up to 128 tokens   7.5 us; a K-step 0.36 us and 0.0025 a token
//     (77x11002x4104 26.0, 128x14336x4096 28.7, 256x4096x4096 22.0 in two slices)
//   CTA pair                     9 us once; a K-step of a wave of tiles 0.51 us with 96
//     tokens, 0.53 with 128, 0.61 with 160, 0.65 with 192 (4096^3: 169, 132, 129, 116 us)
double estimate(const S8GemmParams& p, int sm_count, int clusters, const S8Choice& c) {
    const double n = (double)p.epi.N, k = (double)p.K;
    const int64_t steps = ceil_div(p.K, S8_KSTEP);
    // tiles of experts: half a tile each is expected to be cut off
    const double rows = (double)p.epi.M / c.rows + (p.num_experts ? 0.5 * (double)std::min<int64_t>(p.num_experts, p.epi.M) : 0.0);
    const double tokens = p.num_experts ? rows : (double)ceil_div(p.epi.M, c.rows);
    const double memory = 3.0 + n * k * (double)std::max<int64_t>(1, std::min<int64_t>(p.num_experts, p.epi.M)) / 6.0e6;
    if (c.kernel == S8_PAIR) {
        const double waves = ceil(tokens * (double)ceil_div(p.epi.N, 256) / clusters);
        const double step = c.rows <= 96 ? 0.51 : c.rows <= 128 ? 0.53 : c.rows <= 160 ? 0.61 : 0.65;
        return std::max(memory, 9.0 + waves * (double)steps * step);
    }
    const double ctas = tokens * (double)ceil_div(p.epi.N, 128) * c.splits;
    const double cut = c.splits > 1 ? 3.0 : 0.0, each = (double)ceil_div(steps, c.splits);
    if (c.width == 32) {
        const double step = (ctas > sm_count ? 0.50 : 0.40) + (c.rows > 16 ? 0.08 : 0.0);
        return std::max(memory, ceil(ctas / (2.0 * sm_count)) * (5.0 + each * step) + cut);
    }
    return std::max(memory, ceil(ctas / sm_count) * (7.5 + each * (0.36 + 0.0025 * c.rows)) + cut);
}

S8Choice choose(const S8GemmParams& p, int sm_count, int clusters, int forced_split) {
    const int64_t each = rows_each(p), steps = ceil_div(p.K, S8_KSTEP);
    S8Choice forced{S8_GEMV, 0, 0, 1}, best{S8_TILE, 32, 16, 1};
    const bool pinned = forced_kernel(&forced);
    if (pinned ? forced.kernel == S8_GEMV : each <= 1 && !forced_split) {
        // One token: 1x4096x14336 13.3 us, in tiles 15.4.  By experts with a row each on
        // average, popular ones first, each row reads its expert's weights: 8 rows by 32
        // experts of 2048 x 4096 13.6 us, in tiles 20.9; 8 by 8 of 4096 x 14336 64, 73; 32 by
        // 32 of 512 x 512 4.8, 6.1.  Tiles are quicker where many experts have several
        // rows: 32 by 32 of 2048 x 4096 30, here 41; 64 by 64 50, 71; 256 by 256 168, 282.
        best.kernel = S8_GEMV;
        best.rows = 1;
        return best;
    }
    double best_us = -1.0;
    auto consider = [&](const S8Choice& c) {
        const double us = estimate(p, sm_count, clusters, c);
        // a forced number of slices goes before time, as far as K has steps for it
        const bool better = forced_split && c.splits != best.splits ? c.splits > best.splits : us < best_us;
        if (best_us < 0 || better) {
            best_us = us;
            best = c;
        }
    };
    for (int width : {32, 128}) {
        if (pinned && (forced.kernel != S8_TILE || forced.width != width)) continue;
        if (!pinned && !s8_gemm_usable(width)) continue;  // the other serves the call
        const int rows = (int)(ceil_div(ceil_div(each, ceil_div(each, width)), 16) * 16);
        for (int splits : {1, 2, 4, 8}) {
            if (splits > steps || (forced_split && splits > forced_split)) continue;
            consider({S8_TILE, width, rows, splits});
        }
    }
    if (clusters > 0 && (pinned ? forced.kernel == S8_PAIR : !forced_split && each > 16))
        for (int rows : {96, 128, 160, 192}) consider({S8_PAIR, 0, (int)std::min<int64_t>(rows, ceil_div(each, 32) * 32), 1});
    return best;
}

// Tensor map over int8 codes: [matrices][lines][codes of a line], boxes of one
// K-step (128 codes, swizzled) x box_lines.
int map_s8(gemm_handle_t h, CUtensorMap* m, const void* ptr, int64_t k, int64_t lines, int64_t ld, int32_t num, int64_t bstride,
           int32_t box_lines) {
    const uint64_t dims[3] = {(uint64_t)k, (uint64_t)lines, (uint64_t)num};
    const uint64_t strides[2] = {(uint64_t)ld, (uint64_t)bstride};
    const uint32_t box[3] = {S8_KSTEP, (uint32_t)box_lines, 1};
    return handle_encode(h, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, num > 1 ? 3 : 2, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int run_product(gemm_handle_t h, const gemm_op_t* op, S8GemmParams& p, cudaStream_t st) {
    const int64_t M = p.epi.M, N = p.epi.N;
    if (M == 0 || N == 0) {
        handle_set_choice(h, "empty", M, N, p.K);
        return GEMM_OK;
    }
    if (p.K == 0) {  // no products: act(beta * C + bias), of the rows that K > 0 writes
        handle_set_choice(h, "scale_c", M, N, p.K);
        return status_of(launch_mx_no_k(p.epi, p.offsets, p.num_experts, st));
    }
    const int clusters = pair_clusters(h);
    const S8Choice c = choose(p, handle_sm_count(h), clusters, op->splitk);
    const char* grouped = p.num_experts ? "_grouped" : "";
    char name[64];
    p.tile_rows = c.rows;
    const int64_t tm = token_tiles(p, c.rows);
    if (c.kernel == S8_GEMV) {
        if (tm > 65535) return GEMM_ERR_UNSUPPORTED;
        p.tiles_m = (int32_t)tm;
        p.kslices = s8_gemv_slices(N, p.K, tm, handle_sm_count(h));
        snprintf(name, sizeof name, "s8%s_gemv/k%d", grouped, p.kslices);
        handle_set_choice(h, name, M, N, p.K);
        return status_of(launch_s8_gemv(p, st));
    }
    const bool pair = c.kernel == S8_PAIR;
    const int64_t tn = ceil_div(N, pair ? 256 : 128);
    if (tm * tn * c.splits > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    p.tiles_m = (int32_t)tm;
    p.tiles_n = (int32_t)tn;
    p.k_steps = (int32_t)ceil_div(p.K, S8_KSTEP);
    p.splits = c.splits;
    p.b3d = p.num_experts > 1;
    p.idesc = make_idesc_f16(0, 128, c.rows);
    const int64_t es = float_size(p.epi.d_type);
    auto four = [&](const void* q, int64_t ld) { return !q || (aligned(q, (uintptr_t)(4 * es)) && ld % 4 == 0); };
    p.vec4 = four(p.epi.D, p.epi.ldd) && four(p.epi.C, p.epi.ldc);
    p.status = handle_status(h);
    p.timeout_ns = handle_timeout_ns(h);
    S8Maps m;
    memset(&m, 0, sizeof m);
    int rc = map_s8(h, &m.a, p.A, p.K, M, p.lda, 1, 0, pair ? S8_PAIR_TOKENS / 2 : c.rows);
    if (rc == GEMM_OK) rc = map_s8(h, &m.b, p.B, p.K, N, p.ldb, p.num_experts > 1 ? p.num_experts : 1, p.b_bs, 128);
    if (rc != GEMM_OK) return rc;
    if (pair) {
        p.programs = (int32_t)std::min<int64_t>(clusters, tm * tn);
        snprintf(name, sizeof name, "s8%s_pair/rows%d", grouped, c.rows);
        handle_set_choice(h, name, M, N, p.K);
        return status_of(launch_s8_pair(m, p, p.programs, st));
    }
    snprintf(name, sizeof name, "s8%s_t%d/%s%d", grouped, c.width, c.splits > 1 ? "splitk" : "rows", c.splits > 1 ? c.splits : c.rows);
    handle_set_choice(h, name, M, N, p.K);
    return status_of(launch_s8_gemm(c.width, m, p, (int)(tm * tn * c.splits), st));
}

}  // namespace

extern "C" {

int gemm_run_s8(gemm_handle_t h, const gemm_op_t* op, float alpha, const void* A, const gemm_layout_t* Adesc,
                const float* SA, const void* B, const gemm_layout_t* Bdesc, const float* SB, float beta, const void* C,
                const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc, gemm_stream_t stream) {
    return guarded(h, [&] {
        S8GemmParams p;
        const int rc = check_product(h, op, alpha, A, Adesc, SA, B, Bdesc, SB, beta, C, Cdesc, D, Ddesc, nullptr, 0, &p);
        return rc ? rc : run_product(h, op, p, reinterpret_cast<cudaStream_t>(stream));
    });
}

int gemm_run_s8_grouped(gemm_handle_t h, const gemm_op_t* op, float alpha, const void* A, const gemm_layout_t* Adesc,
                        const float* SA, const void* B, const gemm_layout_t* Bdesc, const float* SB, float beta,
                        const void* C, const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc,
                        const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!expert_offsets_dev || num_experts < 1) return (int)GEMM_ERR_INVALID_ARG;
        int rc = check_experts(h, expert_offsets_dev, num_experts);
        if (rc) return rc;
        S8GemmParams p;
        rc = check_product(h, op, alpha, A, Adesc, SA, B, Bdesc, SB, beta, C, Cdesc, D, Ddesc, expert_offsets_dev,
                           num_experts, &p);
        return rc ? rc : run_product(h, op, p, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
