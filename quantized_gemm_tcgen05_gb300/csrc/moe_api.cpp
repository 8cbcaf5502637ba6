// The C ABI of the operators around the grouped products (include/gemm_moe.h)
// and of row quantisation (include/gemm_s8.h): checks of arguments and launch.
// Host code only.
#include "gemm_moe.h"

#include <math.h>
#include <string.h>

#include <algorithm>

#include "api_checks.h"
#include "gemm_s8.h"
#include "moe_params.h"

using namespace qg;

static_assert((int)GEMM_ROUTE_SOFTMAX == (int)ROUTE_SOFTMAX && (int)GEMM_ROUTE_SIGMOID == (int)ROUTE_SIGMOID, "");
// counts of a block: one per expert, in octets
static_assert(GEMM_ROUTE_SCRATCH(1) == 8 * sizeof(uint16_t) * ROUTE_MAX_BLOCKS && GEMM_ROUTE_SCRATCH(9) == 2 * GEMM_ROUTE_SCRATCH(1), "");

namespace {

int64_t element_size(int32_t t) {
    return t == GEMM_S8 || t == GEMM_E4M3 || t == GEMM_E5M2 ? 1 : float_size(t);
}

bool usable(gemm_handle_t h, const void* p, int64_t align) {
    return p && aligned(p, (uintptr_t)align) && handle_device_pointer(h, p);
}

// Largest power of two, at most 16, that divides all of them.
int common_unit(std::initializer_list<uint64_t> v) {
    uint64_t all = 16;
    for (uint64_t x : v) all |= x;
    return (int)(all & (~all + 1));
}

// X to rows of Y: quantised where Y is int8 and X is not.
int rows_params(gemm_handle_t h, const void* X, const gemm_layout_t* Xd, const int32_t* map, int32_t topk, void* Y,
                const gemm_layout_t* Yd, float* S, RowsParams* p, bool* quantise) {
    if (!Xd || !Yd) return GEMM_ERR_INVALID_ARG;
    *quantise = Yd->type == GEMM_S8 && Xd->type != GEMM_S8;
    const int64_t xs = *quantise ? float_size(Xd->type) : element_size(Xd->type), ys = element_size(Yd->type);
    if (!xs || !ys || (!*quantise && Xd->type != Yd->type)) return GEMM_ERR_UNSUPPORTED;
    int rc;
    if ((rc = check_matrix(Xd, GEMM_ROW_MAJOR, Xd->rows, Xd->cols))) return rc;
    if ((rc = check_matrix(Yd, GEMM_ROW_MAJOR, map || topk > 1 ? Yd->rows : Xd->rows, Xd->cols))) return rc;
    if (Xd->num != Yd->num) return GEMM_ERR_INVALID_ARG;
    if (!offsets_fit(Xd, Xd->rows) || !offsets_fit(Yd, Yd->rows)) return GEMM_ERR_UNSUPPORTED;
    for (const gemm_layout_t* d : {Xd, Yd})
        if (d->num > 1 && d->batch_stride < (d->rows > 0 ? (d->rows - 1) * d->ld + d->cols : 0)) return GEMM_ERR_INVALID_ARG;
    if (Xd->num > 65535 || Xd->cols > INT32_MAX - 65536) return GEMM_ERR_UNSUPPORTED;
    memset(p, 0, sizeof *p);
    p->rows = Xd->rows;
    p->cols = (int32_t)Xd->cols;
    p->num = Xd->num;
    if (Xd->rows == 0 || Xd->cols == 0) return GEMM_OK;
    if (!usable(h, X, xs) || !usable(h, Y, ys)) return GEMM_ERR_INVALID_ARG;
    if (*quantise && !usable(h, S, 4)) return GEMM_ERR_INVALID_ARG;
    p->X = X;
    p->ldx = Xd->ld;
    p->x_bstride = Xd->num > 1 ? Xd->batch_stride : 0;
    p->x_end = past(X, (Xd->num - 1) * p->x_bstride + (Xd->rows - 1) * Xd->ld + Xd->cols, xs);
    p->Y = Y;
    p->ldy = Yd->ld;
    p->y_bstride = Yd->num > 1 ? Yd->batch_stride : 0;
    p->S = S;
    p->type = Xd->type;
    p->vec = std::min(row_alignment(X, Xd->ld, xs), row_alignment(X, p->x_bstride, xs));
    p->yvec = row_alignment(Y, Yd->ld, ys) > 0 && row_alignment(Y, p->y_bstride, ys) > 0;
    p->element = (int32_t)xs;
    p->copy_unit = common_unit({(uint64_t)(uintptr_t)X, (uint64_t)(uintptr_t)Y, (uint64_t)(Xd->ld * xs), (uint64_t)(Yd->ld * ys)});
    p->map = map;
    p->topk = topk;
    p->y_rows = Yd->rows;
    return GEMM_OK;
}

int check_map(gemm_handle_t h, const int32_t* rows, int64_t tokens, int32_t topk) {
    if (topk < 1 || topk > MOE_MAX_TOPK) return GEMM_ERR_INVALID_ARG;
    if (tokens > 0 && !usable(h, rows, 4)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_moe_route(gemm_handle_t h, const gemm_route_t* op, const void* L, const gemm_layout_t* Ldesc, int32_t* ids,
                   float* weights, int32_t* rows, int32_t* expert_offsets, const gemm_workspace_t* workspace,
                   gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!op || !Ldesc) return (int)GEMM_ERR_INVALID_ARG;
        if (op->score != GEMM_ROUTE_SOFTMAX && op->score != GEMM_ROUTE_SIGMOID) return (int)GEMM_ERR_UNSUPPORTED;
        const int64_t ls = float_size(Ldesc->type), tokens = Ldesc->rows, experts = Ldesc->cols;
        if (!ls) return (int)GEMM_ERR_UNSUPPORTED;
        int rc;
        if ((rc = check_matrix(Ldesc, GEMM_ROW_MAJOR, tokens, experts))) return rc;
        if (Ldesc->num != 1 || experts > MOE_MAX_EXPERTS || !offsets_fit(Ldesc, tokens)) return (int)GEMM_ERR_UNSUPPORTED;
        if (experts < 1 || op->topk < 1 || op->topk > experts) return (int)GEMM_ERR_INVALID_ARG;
        if (op->topk > MOE_MAX_TOPK) return (int)GEMM_ERR_UNSUPPORTED;
        if (op->groups < 0 || !isfinite(op->scale) || (op->renormalize != 0 && op->renormalize != 1))
            return (int)GEMM_ERR_INVALID_ARG;
        const int32_t groups = op->groups > 1 ? op->groups : 1;
        if (groups > 32) return (int)GEMM_ERR_UNSUPPORTED;
        if (groups > 1) {
            if (experts % groups || op->group_topk < 1 || op->group_topk > groups) return (int)GEMM_ERR_INVALID_ARG;
            if (op->group_best < 1 || op->group_best > 2) return (int)GEMM_ERR_INVALID_ARG;
        }
        if (tokens > ROUTE_MAX_TOKENS) return (int)GEMM_ERR_UNSUPPORTED;
        if (tokens > 0 && (rows != nullptr) != (expert_offsets != nullptr)) return (int)GEMM_ERR_INVALID_ARG;
        if (op->bias && !usable(h, op->bias, 4)) return (int)GEMM_ERR_INVALID_ARG;
        if (expert_offsets && !usable(h, expert_offsets, 4)) return (int)GEMM_ERR_INVALID_ARG;
        if (tokens > 0) {
            if (!usable(h, L, ls) || !usable(h, ids, 4) || !usable(h, weights, 4)) return (int)GEMM_ERR_INVALID_ARG;
            if (rows && !usable(h, rows, 4)) return (int)GEMM_ERR_INVALID_ARG;
        } else if (!expert_offsets) {
            return (int)GEMM_OK;
        }
        RouteParams p;
        memset(&p, 0, sizeof p);
        p.L = L;
        p.ld = Ldesc->ld;
        p.type = Ldesc->type;
        p.tokens = (int32_t)tokens;
        p.experts = (int32_t)experts;
        p.topk = op->topk;
        p.groups = groups;
        p.group_topk = op->group_topk;
        p.group_best = op->group_best;
        p.score = op->score;
        p.renormalize = op->renormalize;
        p.scale = op->scale;
        p.bias = op->bias;
        p.ids = ids;
        p.weights = weights;
        p.rows = rows;
        p.offsets = expert_offsets;
        const bool scratch = workspace && workspace->partials && workspace->partials_size >= GEMM_ROUTE_SCRATCH(experts);
        if (expert_offsets && (tokens <= ROUTE_FEW || (tokens <= ROUTE_ONE_BLOCK && !scratch))) {
            p.blocks = 1;
            p.tokens_per_block = ROUTE_ONE_BLOCK;
        } else {
            // a token a warp, a block an SM, then more tokens a warp
            int64_t per = std::max<int64_t>(ROUTE_FEW, ceil_div(tokens, std::min(handle_sm_count(h), ROUTE_MAX_BLOCKS)));
            if (per > 65535) per = ceil_div(tokens, ROUTE_MAX_BLOCKS);
            p.tokens_per_block = (int32_t)per;
            p.blocks = (int32_t)ceil_div(tokens, per);
        }
        if (expert_offsets && p.blocks > 1) {
            if (!scratch) return (int)GEMM_ERR_WORKSPACE;
            if (!usable(h, workspace->partials, 16)) return (int)GEMM_ERR_INVALID_ARG;
            p.counts = static_cast<uint16_t*>(workspace->partials);
            p.pitch = (int32_t)(ceil_div(experts, 8) * 8);
        }
        return status_of(launch_route(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

int gemm_s8_quantize(gemm_handle_t h, const void* X, const gemm_layout_t* Xdesc, void* Q, const gemm_layout_t* Qdesc,
                     float* S, gemm_stream_t stream) {
    return guarded(h, [&] {
        RowsParams p;
        bool quantise = false;
        const int rc = rows_params(h, X, Xdesc, nullptr, 1, Q, Qdesc, S, &p, &quantise);
        if (rc) return rc;
        if (!quantise) return (int)GEMM_ERR_UNSUPPORTED;
        if (p.rows == 0 || p.cols == 0) return (int)GEMM_OK;
        return status_of(launch_row_quantize(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

int gemm_moe_dispatch(gemm_handle_t h, const void* X, const gemm_layout_t* Xdesc, const int32_t* rows, int32_t topk,
                      void* Y, const gemm_layout_t* Ydesc, float* S, gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!Xdesc || !Ydesc) return (int)GEMM_ERR_INVALID_ARG;
        int rc = check_map(h, rows, Xdesc->rows, topk);
        if (rc) return rc;
        if (Xdesc->num != 1 || Ydesc->num != 1) return (int)GEMM_ERR_UNSUPPORTED;
        if (Xdesc->rows == 0 || Xdesc->cols == 0 || Ydesc->rows == 0) {
            // nothing to place; the layouts are looked at all the same
            RowsParams none;
            bool q;
            gemm_layout_t x = *Xdesc;
            x.rows = 0;
            rc = rows_params(h, X, &x, rows, 2, Y, Ydesc, S, &none, &q);
            return rc || q || !S ? rc : (int)GEMM_ERR_INVALID_ARG;
        }
        RowsParams p;
        bool quantise = false;
        if ((rc = rows_params(h, X, Xdesc, rows, topk, Y, Ydesc, S, &p, &quantise))) return rc;
        if (!quantise && S) return (int)GEMM_ERR_INVALID_ARG;  // nothing would be written there
        const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        return status_of(quantise ? launch_row_quantize(p, st) : launch_row_copy(p, st));
    });
}

int gemm_moe_combine(gemm_handle_t h, const void* Y, const gemm_layout_t* Ydesc, const int32_t* rows,
                     const float* weights, int32_t topk, float beta, const void* C, const gemm_layout_t* Cdesc, void* D,
                     const gemm_layout_t* Ddesc, gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!Ydesc || !Ddesc) return (int)GEMM_ERR_INVALID_ARG;
        const int64_t es = float_size(Ddesc->type), tokens = Ddesc->rows, cols = Ddesc->cols;
        if (!es || Ydesc->type != Ddesc->type) return (int)GEMM_ERR_UNSUPPORTED;
        int rc;
        if ((rc = check_matrix(Ddesc, GEMM_ROW_MAJOR, tokens, cols))) return rc;
        if ((rc = check_matrix(Ydesc, GEMM_ROW_MAJOR, Ydesc->rows, cols))) return rc;
        const bool use_c = beta != 0.0f;
        if (use_c) {
            if (!Cdesc) return (int)GEMM_ERR_INVALID_ARG;
            if ((rc = check_matrix(Cdesc, GEMM_ROW_MAJOR, tokens, cols))) return rc;
            if (Cdesc->type != Ddesc->type) return (int)GEMM_ERR_UNSUPPORTED;
        }
        if (Ydesc->num != 1 || Ddesc->num != 1 || (use_c && Cdesc->num != 1)) return (int)GEMM_ERR_UNSUPPORTED;
        if (!offsets_fit(Ydesc, Ydesc->rows) || !offsets_fit(Ddesc, tokens) || (use_c && !offsets_fit(Cdesc, tokens)))
            return (int)GEMM_ERR_UNSUPPORTED;
        if (cols > (int64_t)65535 * 2048) return (int)GEMM_ERR_UNSUPPORTED;
        if ((rc = check_map(h, rows, tokens, topk))) return rc;
        if (tokens == 0 || cols == 0) return (int)GEMM_OK;
        if (!usable(h, weights, 4) || !usable(h, D, es) || (use_c && !usable(h, C, es))) return (int)GEMM_ERR_INVALID_ARG;
        if (Ydesc->rows > 0 && !usable(h, Y, es)) return (int)GEMM_ERR_INVALID_ARG;
        CombineParams p;
        memset(&p, 0, sizeof p);
        p.Y = Y;
        p.y_rows = Ydesc->rows;
        p.ldy = Ydesc->ld;
        p.y_end = Ydesc->rows > 0 ? past(Y, (Ydesc->rows - 1) * Ydesc->ld + cols, es) : Y;
        if (use_c) {
            p.C = C;
            p.ldc = Cdesc->ld;
            p.c_end = past(C, (tokens - 1) * Cdesc->ld + cols, es);
        }
        p.D = D;
        p.ldd = Ddesc->ld;
        p.tokens = tokens;
        p.cols = (int32_t)cols;
        p.type = Ddesc->type;
        p.topk = topk;
        p.beta = beta;
        p.map = rows;
        p.weights = weights;
        p.vec = std::min({row_alignment(Ydesc->rows > 0 ? Y : nullptr, p.ldy, es), row_alignment(p.C, p.ldc, es), row_alignment(D, p.ldd, es)});
        return status_of(launch_combine(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
