// The C ABI of the 4-bit microscaled operators (include/gemm_mx.h): checks of
// arguments, tensor maps, choice of kernel, launch.  Host code only.
#include "gemm_mx.h"

#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "handle_internal.h"
#include "mx_gemm.h"

using namespace qg;

static_assert((int)GEMM_MXFP4 == (int)MXF_MXFP4 && (int)GEMM_NVFP4 == (int)MXF_NVFP4,
              "the C ABI's format codes are the kernels' codes");

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// How rows may be moved: 2 in 32-byte pieces, 1 in 16-byte ones, 0 by element.
int row_alignment(const void* p, int64_t ld, int64_t element) {
    if (!p) return 2;
    return aligned(p, 32) && ld * element % 32 == 0 ? 2 : aligned(p, 16) && ld * element % 16 == 0 ? 1 : 0;
}
const void* past(const void* p, int64_t n, int64_t element) {
    return p ? static_cast<const char*>(p) + n * element : nullptr;
}
bool known_format(int32_t f) { return f == GEMM_MXFP4 || f == GEMM_NVFP4; }
int64_t float_size(int32_t t) { return t == GEMM_F32 ? 4 : (t == GEMM_F16 || t == GEMM_BF16) ? 2 : 0; }

int check_matrix(const gemm_layout_t* d, int32_t order, int64_t rows, int64_t cols) {
    if (d->order != order) return GEMM_ERR_UNSUPPORTED;
    if (d->rows != rows || d->cols != cols || d->num < 1) return GEMM_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX) return GEMM_ERR_INVALID_ARG;
    const int64_t inner = order == GEMM_ROW_MAJOR ? cols : rows;
    if (d->ld < (inner > 0 ? inner : 1) || d->ld > ((int64_t)1 << 40)) return GEMM_ERR_INVALID_ARG;
    if (d->num > 1 && (d->batch_stride < 0 || d->batch_stride > ((int64_t)1 << 50))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// Packed codes: 16-byte rows, matrices one after another when there are several.
int check_codes(const gemm_layout_t* d, int64_t lines) {
    if (d->type != GEMM_E2M1) return GEMM_ERR_UNSUPPORTED;
    if (d->ld % 32) return GEMM_ERR_INVALID_ARG;
    if (d->num > 1 && (d->batch_stride % 32 || d->batch_stride < lines * d->ld)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

int64_t scale_bytes(int32_t format, int64_t rows, int64_t cols, int32_t experts) {
    const int64_t tiles = experts > 0 ? rows / MX_ATOM_ROWS + experts : ceil_div(rows, MX_ATOM_ROWS);
    return tiles * mx_atoms(format, cols) * MX_ATOM_BYTES;
}

bool tensor_scale_ok(int32_t format, float g) {
    if (format == GEMM_MXFP4) return g == 1.0f;
    return g >= 0x1p-64f && g <= 0x1p64f;  // false for NaN
}

int check_experts(gemm_handle_t h, const int32_t* offsets, int32_t experts) {
    if (!offsets && experts == 0) return GEMM_OK;
    if (!offsets || experts < 1 || experts > 4096) return GEMM_ERR_INVALID_ARG;
    if (!aligned(offsets, 4) || !handle_device_pointer(h, offsets)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_CUDA;
}

// The widest row a quantising grid covers: 512 columns a block, 65535 blocks.
constexpr int64_t QUANT_MAX_COLS = 65535ll * 512;

int quant_params(gemm_handle_t h, int32_t format, float g, const gemm_layout_t* v, const gemm_layout_t* q,
                 const void* vals, const void* codes, const void* S, size_t S_size, const int32_t* offsets,
                 int32_t experts, bool e4m3, MxQuantParams* p) {
    if (!v || !q) return GEMM_ERR_INVALID_ARG;
    if (!known_format(format)) return GEMM_ERR_UNSUPPORTED;
    const int64_t es = e4m3 && v->type == GEMM_E4M3 ? 1 : float_size(v->type);
    if (!es) return GEMM_ERR_UNSUPPORTED;
    int rc;
    if ((rc = check_matrix(v, GEMM_ROW_MAJOR, v->rows, v->cols))) return rc;
    if ((rc = check_matrix(q, GEMM_ROW_MAJOR, v->rows, v->cols))) return rc;
    if ((rc = check_codes(q, v->rows))) return rc;
    if (q->num != v->num) return GEMM_ERR_INVALID_ARG;
    if (v->num > 1 && v->batch_stride < (v->rows > 0 ? (v->rows - 1) * v->ld + v->cols : 0)) return GEMM_ERR_INVALID_ARG;
    if (!tensor_scale_ok(format, g)) return GEMM_ERR_INVALID_ARG;
    if ((rc = check_experts(h, offsets, experts))) return rc;
    if (experts && v->num != 1) return GEMM_ERR_INVALID_ARG;
    if (v->rows > INT32_MAX - 64 || v->cols > QUANT_MAX_COLS || v->num > 65535) return GEMM_ERR_UNSUPPORTED;
    const int64_t need = scale_bytes(format, v->rows, v->cols, experts);
    memset(p, 0, sizeof *p);
    p->rows = v->rows;
    p->cols = v->cols;
    if (v->rows == 0 || v->cols == 0) return GEMM_OK;
    if (!vals || !codes || !S) return GEMM_ERR_INVALID_ARG;
    if (!aligned(vals, (uintptr_t)es) || !aligned(codes, 16) || !aligned(S, 16)) return GEMM_ERR_INVALID_ARG;
    if (S_size / (uint64_t)v->num < (uint64_t)need) return GEMM_ERR_INVALID_ARG;
    if (!handle_device_pointer(h, vals) || !handle_device_pointer(h, codes) || !handle_device_pointer(h, S))
        return GEMM_ERR_INVALID_ARG;
    p->ldx = v->ld;
    p->x_bstride = v->num > 1 ? v->batch_stride : 0;
    p->ldq = q->ld / 2;
    p->q_bstride = v->num > 1 ? q->batch_stride / 2 : 0;
    p->s_bstride = need;
    p->num = v->num;
    p->type = v->type;
    p->format = format;
    p->vec = std::min(row_alignment(vals, v->ld, es), row_alignment(vals, p->x_bstride, es));
    p->atoms = (int32_t)mx_atoms(format, v->cols);
    p->c = mx_scale_const(g);
    p->offsets = offsets;
    p->num_experts = experts;
    return GEMM_OK;
}

// Tensor map over packed codes: [matrices][lines][bytes of a line], boxes of
// one K-step (128 bytes, swizzled) x box_lines.
int map_codes(gemm_handle_t h, CUtensorMap* m, const void* ptr, int64_t k, int64_t lines, int64_t ld, int32_t num,
              int64_t bstride, int32_t box_lines) {
    const uint64_t dims[3] = {(uint64_t)ceil_div(k, 2), (uint64_t)lines, (uint64_t)num};
    const uint64_t strides[2] = {(uint64_t)ld / 2, (uint64_t)bstride / 2};
    const uint32_t box[3] = {128, (uint32_t)box_lines, 1};
    return handle_encode(h, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, num > 1 ? 3 : 2, ptr, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tensor map over scales: [matrices][atom rows][bytes of an atom row], as
// 8-byte elements; a box is the atoms of one K-step of box_rows atom rows.
// Past the last atom and the last atom row the copies read zeros.
int map_scales(gemm_handle_t h, CUtensorMap* m, const void* ptr, int32_t format, int64_t k, int64_t atom_rows,
               int32_t num, int32_t box_rows) {
    const int64_t atoms = mx_atoms(format, k);
    const uint64_t dims[3] = {(uint64_t)(atoms * MX_ATOM_BYTES / 8), (uint64_t)atom_rows, (uint64_t)num};
    const uint64_t strides[2] = {(uint64_t)(atoms * MX_ATOM_BYTES), (uint64_t)(atoms * MX_ATOM_BYTES * atom_rows)};
    const uint32_t box[3] = {format == GEMM_NVFP4 ? 256u : 128u, (uint32_t)box_rows, 1};
    return handle_encode(h, m, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, num > 1 ? 3 : 2, ptr, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct MxProduct {
    int32_t format;
    int64_t M, N, K;
    const void *A, *SA, *B, *SB;
    int64_t lda, ldb, b_bs;
    EpiParams epi;
    const float* expert_alpha;
    const int32_t* offsets;
    int32_t experts;  // 0: dense
};

int check_product(gemm_handle_t h, const gemm_op_t* op, int32_t format, float alpha, const float* expert_alpha,
                  const void* A, const gemm_layout_t* Ad, const void* SA, size_t SA_size, const void* B,
                  const gemm_layout_t* Bd, const void* SB, size_t SB_size, float beta, const void* C,
                  const gemm_layout_t* Cd, void* D, const gemm_layout_t* Dd, const int32_t* offsets, int32_t experts,
                  MxProduct* out) {
    if (!op || !Ad || !Bd || !Dd) return GEMM_ERR_INVALID_ARG;
    if (!known_format(format)) return GEMM_ERR_UNSUPPORTED;
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
    MxProduct p;
    memset(&p, 0, sizeof p);
    p.format = format;
    p.M = Ad->rows;
    p.K = Ad->cols;
    p.N = Bd->cols;
    int rc;
    if ((rc = check_matrix(Ad, GEMM_ROW_MAJOR, p.M, p.K))) return rc;
    if ((rc = check_matrix(Bd, GEMM_COL_MAJOR, p.K, p.N))) return rc;
    if ((rc = check_matrix(Dd, GEMM_ROW_MAJOR, p.M, p.N))) return rc;
    if ((rc = check_codes(Ad, p.M)) || (rc = check_codes(Bd, p.N))) return rc;
    const int64_t ds = float_size(Dd->type);
    if (!ds) return GEMM_ERR_UNSUPPORTED;
    if (Ad->num != 1 || Dd->num != 1) return experts ? GEMM_ERR_INVALID_ARG : GEMM_ERR_UNSUPPORTED;
    if (Bd->num != (experts ? experts : 1)) return GEMM_ERR_INVALID_ARG;
    EpiParams& e = p.epi;
    if (beta != 0.0f) {
        if (!C || !Cd) return GEMM_ERR_INVALID_ARG;
        if ((rc = check_matrix(Cd, GEMM_ROW_MAJOR, p.M, p.N))) return rc;
        if (Cd->type != Dd->type) return GEMM_ERR_UNSUPPORTED;
        if (Cd->num != 1) return GEMM_ERR_INVALID_ARG;
        e.C = C;
        e.ldc = Cd->ld;
    }
    e.D = D;
    e.ldd = Dd->ld;
    e.M = p.M;
    e.N = p.N;
    e.alpha = alpha;
    e.beta = beta;
    e.d_type = Dd->type;
    e.flags = act;
    e.bias = (act & GEMM_EPILOGUE_BIAS) ? op->bias : nullptr;
    e.bias_type = op->bias_type;
    e.status = handle_status(h);
    if (p.M > 0 && p.N > 0) {
        e.d_extent = (p.M - 1) * e.ldd + p.N;
        e.c_extent = e.C ? (p.M - 1) * e.ldc + p.N : 0;
        if (!D || !aligned(D, (uintptr_t)ds) || !handle_device_pointer(h, D)) return GEMM_ERR_INVALID_ARG;
        if (e.C && (!aligned(C, (uintptr_t)ds) || !handle_device_pointer(h, C))) return GEMM_ERR_INVALID_ARG;
        if (p.K > 0) {
            if (!A || !B || !SA || !SB) return GEMM_ERR_INVALID_ARG;
            if (!aligned(A, 16) || !aligned(B, 16) || !aligned(SA, 16) || !aligned(SB, 16)) return GEMM_ERR_INVALID_ARG;
            if (!handle_device_pointer(h, A) || !handle_device_pointer(h, B) || !handle_device_pointer(h, SA) ||
                !handle_device_pointer(h, SB))
                return GEMM_ERR_INVALID_ARG;
            if (SA_size < (uint64_t)scale_bytes(format, p.M, p.K, experts)) return GEMM_ERR_INVALID_ARG;
            if (SB_size / (uint64_t)Bd->num < (uint64_t)scale_bytes(format, p.N, p.K, 0)) return GEMM_ERR_INVALID_ARG;
        }
        if (expert_alpha && (!aligned(expert_alpha, 4) || !handle_device_pointer(h, expert_alpha)))
            return GEMM_ERR_INVALID_ARG;
    }
    p.A = A;
    p.SA = SA;
    p.B = B;
    p.SB = SB;
    p.lda = Ad->ld;
    p.ldb = Bd->ld;
    p.b_bs = Bd->num > 1 ? Bd->batch_stride : 0;
    p.expert_alpha = expert_alpha;
    p.offsets = offsets;
    p.experts = experts;
    *out = p;
    return GEMM_OK;
}

// Output tiles along M: exact, or an upper bound over the splits into experts.
int64_t tiles_along_m(const MxProduct& p, int bm) {
    if (!p.experts) return ceil_div(p.M, bm);
    const int64_t most = p.M / bm + p.experts;
    return most < p.M ? most : p.M;
}

struct MxChoice {
    int bn, splits, pair;
};

// Rows of A that a stage of the one-tile kernel holds.
int rows_staged(const MxProduct& p) { return (int)(p.M < 128 ? ceil_div(p.M, 8) * 8 : 128); }

// Clusters of two that the CTA-pair kernel keeps resident (asked once per device).
int pair_clusters(gemm_handle_t h, int32_t format) {
    static std::atomic<int> known[64][2];
    std::atomic<int>& k = known[handle_device(h) & 63][format == GEMM_NVFP4];
    int n = k.load();
    if (n == 0) {
        n = std::max(0, std::min(mx_pair_max_clusters(format), handle_sm_count(h) / 2)) + 1;
        k.store(n);
    }
    return n - 1;
}

// GEMM_FORCE_KERNEL=mx_bn64 / mx_bn128 / mx2_bn256 (the names gemm_last_choice
// prints, up to the slash) pins the kernel, for tests and sweeps.
bool forced_kernel(MxChoice* c) {
    const char* f = getenv("GEMM_FORCE_KERNEL");
    if (!f || strncmp(f, "mx", 2)) return false;
    c->pair = strncmp(f, "mx2_bn256", 9) == 0;
    c->bn = c->pair ? 256 : strncmp(f, "mx_bn64", 7) == 0 ? 64 : 128;
    return true;
}

// Estimated time of a choice, microseconds.  Measured on GB300 (152 SMs),
// back-to-back launches:
//   one-tile kernel  2.5 us for launch, first data and exit (1x64x64), 0.30 us (64
//     columns) or 0.33 (128) a K-step of 256 while the issuing warp is the bound,
//     else the bytes of the stages of the CTAs that share an SM at 132 bytes a nanosecond; 1.2 us for
//     every further wave of CTAs, 0.25 us for every CTA on an SM; K slices: 1.4 us
//     and 0.025 us a row of a 64-column tile (1x4096x4096: 7.7 us whole, 6.2 in
//     two, 5.6 in four; 128x4096x4096: 9.0 whole, 10.3 in two)
//   CTA pair         3.9 us, 0.37 us a K-step, 0.42 when every cluster is busy
//     (512x4096x4096: 10.5 us against 9.4 in 64-column tiles; 1024x4096x4096:
//     11.0 against 18; 4096^3: 31 against 65)
// No choice takes less than its operands at 6.5 TB/s; among choices that memory
// bounds, the one with less else to do is ahead.
double estimate(const MxProduct& p, int sm_count, int clusters, const MxChoice& c) {
    const int64_t steps = ceil_div(p.K, MX_KSTEP);
    const double bytes = 0.56 * (double)p.K * ((double)p.M + (double)p.N * (p.experts ? std::min<int64_t>(p.experts, p.M) : 1));
    const double memory = 2.5 + bytes / 6.5e6;
    if (c.pair) {
        const int64_t tiles = tiles_along_m(p, 256) * ceil_div(p.N, 256);
        const double waves = (double)ceil_div(tiles, clusters);
        const double own = 3.9 + waves * steps * (tiles < clusters ? 0.37 : 0.42);
        return std::max(memory, own) + 0.2 * own;
    }
    const int a_rows = rows_staged(p);
    const int64_t ctas = tiles_along_m(p, 128) * ceil_div(p.N, c.bn) * c.splits;
    const double stage = 128.0 * (a_rows + c.bn) + (p.format == GEMM_NVFP4 ? 4096 : 2048);
    const double step = std::max(c.bn == 64 ? 0.30 : 0.33, (ctas > sm_count ? 2 : 1) * stage / 132e3);
    const double waves = (double)ceil_div(ctas, 2 * (int64_t)sm_count);
    const double rows = (double)std::min<int64_t>(p.M, 128);
    const double tail = (c.splits > 1 ? 1.4 + 0.025 * rows * c.bn / 64 : 0.0) + 0.25 * ceil_div(ctas, sm_count);
    const double own = 1.3 + waves * (1.2 + ceil_div(steps, c.splits) * step);
    return std::max(memory, own) + 0.2 * own + tail;
}

MxChoice choose(const MxProduct& p, int sm_count, int clusters, int forced_split) {
    const int64_t steps = ceil_div(p.K, MX_KSTEP);
    const int a_rows = rows_staged(p);
    MxChoice forced{0, 1, 0}, best{64, 1, 0};
    const bool pinned = forced_kernel(&forced);
    double best_us = -1.0;
    for (int bn : {64, 128}) {
        if (pinned && (forced.pair || forced.bn != bn)) continue;
        for (int splits : {1, 2, 4, 8}) {
            if (forced_split && splits != std::min(forced_split, 8)) {
                // a forced count is cut down to what K and shared memory allow
                const bool cut = splits < forced_split &&
                                 (2 * splits > steps || !mx_gemm_stages(bn, p.format, a_rows, 2 * splits));
                if (!cut) continue;
            }
            if (splits > steps || !mx_gemm_stages(bn, p.format, a_rows, splits)) continue;
            const MxChoice c{bn, splits, 0};
            const double us = estimate(p, sm_count, clusters, c);
            // a forced count goes before time: one width may allow it where another does not
            const bool better = forced_split && splits != best.splits ? splits > best.splits : us < best_us;
            if (best_us < 0 || better) {
                best_us = us;
                best = c;
            }
        }
    }
    if (clusters > 0 && (pinned ? forced.pair != 0 : !forced_split && p.M > 128)) {
        const MxChoice c{256, 1, 1};
        if (pinned || estimate(p, sm_count, clusters, c) < best_us) best = c;
    }
    return best;
}

int run_product(gemm_handle_t h, const gemm_op_t* op, MxProduct& p, cudaStream_t st) {
    if (p.M == 0 || p.N == 0) {
        handle_set_choice(h, "empty", p.M, p.N, p.K);
        return GEMM_OK;
    }
    if (p.K == 0) {  // no products: act(beta * C + bias), of the rows that K > 0 writes
        handle_set_choice(h, "scale_c", p.M, p.N, p.K);
        return status_of(launch_mx_no_k(p.epi, p.offsets, p.experts, st));
    }
    const int clusters = pair_clusters(h, p.format);
    const MxChoice c = choose(p, handle_sm_count(h), clusters, op->splitk);
    MxGemmParams k;
    memset(&k, 0, sizeof k);
    k.epi = p.epi;
    k.expert_alpha = p.expert_alpha;
    k.offsets = p.offsets;
    k.num_experts = p.experts;
    const int64_t tm = tiles_along_m(p, c.pair ? 256 : 128), tn = ceil_div(p.N, c.bn);
    if (tm * tn * c.splits > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    k.tiles_m = (int32_t)tm;
    k.tiles_n = (int32_t)tn;
    k.k_steps = (int32_t)ceil_div(p.K, MX_KSTEP);
    k.splits = c.splits;
    k.a_rows = c.pair ? 128 : rows_staged(p);
    k.stages = c.pair ? 0 : mx_gemm_stages(c.bn, p.format, k.a_rows, c.splits);
    k.b3d = p.experts > 1;
    k.idesc = make_idesc_mx(p.format == GEMM_NVFP4, c.pair ? 256 : 128, c.bn);
    const int64_t ds = float_size(p.epi.d_type);
    k.vec32 = aligned(p.epi.D, 32) && p.epi.ldd * ds % 32 == 0 &&
              (!p.epi.C || (aligned(p.epi.C, 32) && p.epi.ldc * ds % 32 == 0));
    k.status = handle_status(h);
    k.timeout_ns = handle_timeout_ns(h);
    MxMaps m;
    memset(&m, 0, sizeof m);
    const int32_t nb = p.experts > 1 ? p.experts : 1;
    const int64_t a_atom_rows = p.experts ? p.M / MX_ATOM_ROWS + p.experts : ceil_div(p.M, MX_ATOM_ROWS);
    int rc = map_codes(h, &m.a, p.A, p.K, p.M, p.lda, 1, 0, k.a_rows);
    if (rc == GEMM_OK) rc = map_codes(h, &m.b, p.B, p.K, p.N, p.ldb, nb, p.b_bs, c.pair ? 128 : c.bn);
    if (rc == GEMM_OK) rc = map_scales(h, &m.sa, p.SA, p.format, p.K, a_atom_rows, 1, 1);
    if (rc == GEMM_OK) rc = map_scales(h, &m.sb, p.SB, p.format, p.K, ceil_div(p.N, MX_ATOM_ROWS), nb, c.pair ? 2 : 1);
    if (rc != GEMM_OK) return rc;
    char name[64];
    if (c.pair || c.splits == 1)
        snprintf(name, sizeof name, "mx%s%s_bn%d/dp", c.pair ? "2" : "", p.experts ? "_grouped" : "", c.bn);
    else
        snprintf(name, sizeof name, "mx%s_bn%d/splitk%d", p.experts ? "_grouped" : "", c.bn, c.splits);
    handle_set_choice(h, name, p.M, p.N, p.K);
    if (c.pair) {
        k.programs = (int32_t)std::min<int64_t>(clusters, tm * tn);
        return status_of(launch_mx_pair(p.format, m, k, k.programs, st));
    }
    return status_of(launch_mx_gemm(c.bn, p.format, m, k, (int)(tm * tn * c.splits), st));
}

// Nothing throws across the C ABI.
template <typename F>
int guarded(gemm_handle_t h, F&& f) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    try {
        const int rc = handle_bind(h);
        return rc ? rc : f();
    } catch (...) {
        return GEMM_ERR_CUDA;
    }
}

}  // namespace

extern "C" {

int gemm_mx_scale_size(int32_t format, int64_t rows, int64_t cols, int32_t num_experts, size_t* bytes) {
    if (!bytes || rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX || num_experts < 0 || num_experts > 4096)
        return GEMM_ERR_INVALID_ARG;
    if (!known_format(format)) return GEMM_ERR_UNSUPPORTED;
    *bytes = (size_t)scale_bytes(format, rows, cols, num_experts);
    return GEMM_OK;
}

int gemm_mx_quantize(gemm_handle_t h, int32_t format, float tensor_scale, const void* X, const gemm_layout_t* Xdesc,
                     void* Q, const gemm_layout_t* Qdesc, void* S, size_t S_size, const int32_t* expert_offsets_dev,
                     int32_t num_experts, gemm_stream_t stream) {
    return guarded(h, [&] {
        MxQuantParams p;
        const int rc = quant_params(h, format, tensor_scale, Xdesc, Qdesc, X, Q, S, S_size, expert_offsets_dev,
                                    num_experts, false, &p);
        if (rc || p.rows == 0 || p.cols == 0) return rc;
        p.X = X;
        p.x_end = past(X, (p.num - 1) * p.x_bstride + (p.rows - 1) * p.ldx + p.cols, float_size(Xdesc->type));
        p.Y = Q;
        p.S = static_cast<uint8_t*>(S);
        return status_of(launch_mx_quantize(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

int gemm_mx_dequantize(gemm_handle_t h, int32_t format, float tensor_scale, const void* Q, const gemm_layout_t* Qdesc,
                       const void* S, size_t S_size, void* D, const gemm_layout_t* Ddesc,
                       const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream) {
    return guarded(h, [&] {
        MxQuantParams p;
        const int rc = quant_params(h, format, tensor_scale, Ddesc, Qdesc, D, Q, S, S_size, expert_offsets_dev,
                                    num_experts, true, &p);
        if (rc || p.rows == 0 || p.cols == 0) return rc;
        p.X = Q;
        p.Y = D;
        p.S = const_cast<uint8_t*>(static_cast<const uint8_t*>(S));
        return status_of(launch_mx_dequantize(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

int gemm_run_mx(gemm_handle_t h, const gemm_op_t* op, int32_t format, float alpha, const void* A,
                const gemm_layout_t* Adesc, const void* SA, size_t SA_size, const void* B, const gemm_layout_t* Bdesc,
                const void* SB, size_t SB_size, float beta, const void* C, const gemm_layout_t* Cdesc, void* D,
                const gemm_layout_t* Ddesc, gemm_stream_t stream) {
    return guarded(h, [&] {
        MxProduct p;
        const int rc = check_product(h, op, format, alpha, nullptr, A, Adesc, SA, SA_size, B, Bdesc, SB, SB_size, beta,
                                     C, Cdesc, D, Ddesc, nullptr, 0, &p);
        return rc ? rc : run_product(h, op, p, reinterpret_cast<cudaStream_t>(stream));
    });
}

int gemm_run_mx_grouped(gemm_handle_t h, const gemm_op_t* op, int32_t format, float alpha, const float* expert_alpha,
                        const void* A, const gemm_layout_t* Adesc, const void* SA, size_t SA_size, const void* B,
                        const gemm_layout_t* Bdesc, const void* SB, size_t SB_size, float beta, const void* C,
                        const gemm_layout_t* Cdesc, void* D, const gemm_layout_t* Ddesc,
                        const int32_t* expert_offsets_dev, int32_t num_experts, gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!expert_offsets_dev || num_experts < 1) return (int)GEMM_ERR_INVALID_ARG;
        int rc = check_experts(h, expert_offsets_dev, num_experts);
        if (rc) return rc;
        MxProduct p;
        rc = check_product(h, op, format, alpha, expert_alpha, A, Adesc, SA, SA_size, B, Bdesc, SB, SB_size, beta, C,
                           Cdesc, D, Ddesc, expert_offsets_dev, num_experts, &p);
        return rc ? rc : run_product(h, op, p, reinterpret_cast<cudaStream_t>(stream));
    });
}

int gemm_mx_norm_quantize(gemm_handle_t h, const gemm_mx_norm_t* op, const void* F, const gemm_layout_t* Fdesc,
                          const void* R, const gemm_layout_t* Rdesc, void* O, const gemm_layout_t* Odesc, void* Q,
                          const gemm_layout_t* Qdesc, void* S, size_t S_size, gemm_stream_t stream) {
    return guarded(h, [&] {
        if (!op || !Rdesc || !Qdesc || (F && !Fdesc) || (O && !Odesc) || (F && !O)) return (int)GEMM_ERR_INVALID_ARG;
        if (!known_format(op->format)) return (int)GEMM_ERR_UNSUPPORTED;
        const int64_t rows = Rdesc->rows, cols = Rdesc->cols, es = float_size(Rdesc->type);
        if (!es) return (int)GEMM_ERR_UNSUPPORTED;
        int rc;
        if ((rc = check_matrix(Rdesc, GEMM_ROW_MAJOR, rows, cols))) return rc;
        if (F && (rc = check_matrix(Fdesc, GEMM_ROW_MAJOR, rows, cols))) return rc;
        if (O && (rc = check_matrix(Odesc, GEMM_ROW_MAJOR, rows, cols))) return rc;
        if ((rc = check_matrix(Qdesc, GEMM_ROW_MAJOR, rows, cols)) || (rc = check_codes(Qdesc, rows))) return rc;
        if ((F && Fdesc->type != Rdesc->type) || (O && Odesc->type != Rdesc->type)) return (int)GEMM_ERR_UNSUPPORTED;
        if (Rdesc->num != 1 || Qdesc->num != 1 || (F && Fdesc->num != 1) || (O && Odesc->num != 1))
            return (int)GEMM_ERR_UNSUPPORTED;
        if (cols > 32768) return (int)GEMM_ERR_UNSUPPORTED;
        if (!tensor_scale_ok(op->format, op->tensor_scale)) return (int)GEMM_ERR_INVALID_ARG;
        if (!(op->eps >= 0.0f) || !isfinite(op->eps) || !isfinite(op->residual_scale)) return (int)GEMM_ERR_INVALID_ARG;
        const int64_t ws = float_size(op->weight_type), gs = float_size(op->gate_type);
        const bool weights = op->post_weight || op->pre_weight;
        if ((weights && !ws) || (op->gate && !gs)) return (int)GEMM_ERR_UNSUPPORTED;
        if (!F && (op->post_weight || op->gate)) return (int)GEMM_ERR_INVALID_ARG;
        if (op->gate && op->gate_ld != 0 && (op->gate_ld < cols || op->gate_ld > ((int64_t)1 << 40)))
            return (int)GEMM_ERR_INVALID_ARG;
        if ((rc = check_experts(h, op->expert_offsets, op->num_experts))) return rc;
        if (rows == 0 || cols == 0) return (int)GEMM_OK;
        auto bad = [&](const void* ptr, int64_t n) { return !aligned(ptr, (uintptr_t)n) || !handle_device_pointer(h, ptr); };
        if (!R || !Q || !S || bad(R, es) || bad(Q, 16) || bad(S, 16)) return (int)GEMM_ERR_INVALID_ARG;
        if ((F && bad(F, es)) || (O && bad(O, es))) return (int)GEMM_ERR_INVALID_ARG;
        if ((op->post_weight && bad(op->post_weight, ws)) || (op->pre_weight && bad(op->pre_weight, ws)) ||
            (op->gate && bad(op->gate, gs)))
            return (int)GEMM_ERR_INVALID_ARG;
        if (S_size < (uint64_t)scale_bytes(op->format, rows, cols, op->num_experts)) return (int)GEMM_ERR_INVALID_ARG;
        MxNormParams p;
        memset(&p, 0, sizeof p);
        p.F = F;
        p.R = R;
        p.O = O;
        p.Q = static_cast<uint8_t*>(Q);
        p.S = static_cast<uint8_t*>(S);
        p.rows = rows;
        p.cols = cols;
        p.ldf = F ? Fdesc->ld : 0;
        p.ldr = Rdesc->ld;
        p.ldo = O ? Odesc->ld : 0;
        p.ldq = Qdesc->ld / 2;
        p.type = Rdesc->type;
        p.format = op->format;
        p.vec = std::min({row_alignment(F, p.ldf, es), row_alignment(R, p.ldr, es), row_alignment(O, p.ldo, es)});
        p.wvec = std::min(row_alignment(op->post_weight, 0, ws), row_alignment(op->pre_weight, 0, ws));
        p.gvec = row_alignment(op->gate, op->gate_ld, gs);
        p.atoms = (int32_t)mx_atoms(op->format, cols);
        p.sm_count = handle_sm_count(h);
        p.offsets = op->expert_offsets;
        p.num_experts = op->num_experts;
        p.eps = op->eps;
        p.residual_scale = op->residual_scale;
        p.c = mx_scale_const(op->tensor_scale);
        p.post = op->post_weight;
        p.pre = op->pre_weight;
        p.gate = op->gate;
        p.weight_type = op->weight_type;
        p.gate_type = op->gate_type;
        p.gate_ld = op->gate_ld;
        p.f_end = past(F, (rows - 1) * p.ldf + cols, es);
        p.r_end = past(R, (rows - 1) * p.ldr + cols, es);
        p.post_end = past(p.post, cols, ws);
        p.pre_end = past(p.pre, cols, ws);
        p.gate_end = past(p.gate, (rows - 1) * p.gate_ld + cols, gs);
        return status_of(launch_mx_norm(p, reinterpret_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
