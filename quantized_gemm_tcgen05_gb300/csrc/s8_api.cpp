// The C ABI of the int8 products (include/gemm_s8.h): checks of arguments,
// choice of kernel, launch.  Host code only.
#include "gemm_s8.h"

#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

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

int run_product(gemm_handle_t h, const gemm_op_t* op, S8GemmParams& p, cudaStream_t st) {
    (void)op;
    const int64_t M = p.epi.M, N = p.epi.N;
    if (M == 0 || N == 0) {
        handle_set_choice(h, "empty", M, N, p.K);
        return GEMM_OK;
    }
    if (p.K == 0) {  // no products: act(beta * C + bias), of the rows that K > 0 writes
        handle_set_choice(h, "scale_c", M, N, p.K);
        return status_of(launch_mx_no_k(p.epi, p.offsets, p.num_experts, st));
    }
    const int64_t per = p.num_experts ? ceil_div(M, p.num_experts) : M;
    p.tile_rows = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 8;
    const int64_t tiles = token_tiles(p, p.tile_rows);
    if (tiles > 65535) return GEMM_ERR_UNSUPPORTED;
    p.tiles_m = (int32_t)tiles;
    p.kslices = s8_gemv_slices(N, p.K, tiles, handle_sm_count(h));
    char name[64];
    snprintf(name, sizeof name, "s8%s_gemv%d/k%d", p.num_experts ? "_grouped" : "", p.tile_rows, p.kslices);
    handle_set_choice(h, name, M, N, p.K);
    return status_of(launch_s8_gemv(p, handle_sm_count(h), st));
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
