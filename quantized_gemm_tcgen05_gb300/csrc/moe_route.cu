// Routing: every token's topk experts, their weights, and the rows of the
// (token, slot) pairs sorted by expert.
//
// A warp takes a token; lane i holds experts i, i + 32, ...  Scores are numbers
// turned into unsigned keys of the same order (0: never chosen), so that a round
// of the choice is a warp-wide integer maximum.
//
// The choice is defined in 64 bits.  Without a bias it is the logits' own order,
// which fp32 holds exactly.  With one (and for groups' scores) it is that of sums
// whose error fp32 leaves open.  Three tries, each only where the one before
// cannot tell:
//   1. keys of 22 bits with the expert's number below them: a round is one maximum,
//      and needs no second one for the index;
//   2. keys of 32 bits (a few tokens in a hundred);
//   3. scores in 64 bits (one in a thousand).  All tokens that way would take ten
//      times the time: there are two 64-bit units an SM.
// What bounds it is the number of instructions: 4001 x 256 logits are 4 MB.
#include "common.cuh"
#include "moe_params.h"

namespace qg {

namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;

// Keys: unsigned integers in the order of the numbers, 0 below all of them.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 counts as 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ float number_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ double number_of(uint64_t k) { return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k)); }

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(FULL, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(FULL, (uint32_t)(k >> 32));
    return (uint64_t)hi << 32 | __reduce_max_sync(FULL, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
}
template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(FULL, x, d);
    return x;
}

__device__ __forceinline__ float exp_t(float x) { return expf(x); }
__device__ __forceinline__ double exp_t(double x) { return exp(x); }

template <typename T>
struct KeyType;
template <>
struct KeyType<float> {
    using type = uint32_t;
};
template <>
struct KeyType<double> {
    using type = uint64_t;
};

// A bound of the fp32 error of a token's scores s, without the part that grows with
// c.  Sigmoid: the exponential is off by 2 units, s (1 - s) 2^-22 <= 2^-24, a sum and a
// quotient by half a unit each: below 2e-7.  Softmax: the exponential's argument is off
// by up to 2^-24 |l - max| (x e^-x is at most 0.37), the exponential by 2 units, a sum of
// E <= 1024 of them by 37 roundings at most, the quotient by one: below 3e-6 s.
__device__ __forceinline__ float score_error(int32_t score, float largest) { return score == ROUTE_SOFTMAX ? 4e-6f * largest : 4e-7f; }
// ... of c = s + bias.
__device__ __forceinline__ float choice_error(float err, float c) { return err + 1.2e-7f * fabsf(c); }

// Choose for one token.  l: this lane's logits (-inf past the last expert).
// Slot j's expert lands in lane j's `id` (-1: none).  Returns false where fp32
// cannot tell (T = float only).  V: experts a lane.
template <int V, typename T>
__device__ __forceinline__ bool choose(const RouteParams& p, const float (&l)[V], float top, int lane, int& id) {
    using K = typename KeyType<T>::type;
    constexpr bool EXACT = sizeof(T) == 8;
    const bool by_logit = !p.bias;
    K key[V];
    bool sure = true;
    float err = 0.0f;
    if (!by_logit || p.groups > 1) {
        T s[V];
        if (p.score == ROUTE_SOFTMAX) {
            T sum = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = l[v] > -INFINITY ? exp_t((T)l[v] - (T)top) : (T)0;
                sum += s[v];
            }
            sum = warp_sum(sum);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = s[v] / sum;
            err = score_error(p.score, (float)((T)1 / sum));
        } else {
            err = score_error(p.score, 1.0f);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = (T)1 / ((T)1 + exp_t(-(T)l[v]));
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 32 + lane;
            const float b = p.bias && e < p.experts ? p.bias[e] : 0.0f;
            const T c = s[v] + (T)b;
            key[v] = l[v] > -INFINITY && b > -INFINITY ? key_of(c) : (K)0;
        }
    }
    if (p.groups > 1) {
        // group g's score in lane g, as a key
        const int size = p.experts / p.groups;
        int group[V];
#pragma unroll
        for (int v = 0; v < V; ++v) group[v] = (v * 32 + lane) / size;
        K mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            K first = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (group[v] == g && key[v] > first) first = key[v];
            const K a = warp_max(first);
            K score = a;
            if (p.group_best > 1 && a) {
                // without one expert that has it
                const unsigned have = __ballot_sync(FULL, first == a);
                const bool holder = (int)__ffs((int)have) - 1 == lane;
                K second = 0;
                bool skipped = !holder;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (group[v] != g) continue;
                    if (!skipped && key[v] == a)
                        skipped = true;
                    else if (key[v] > second)
                        second = key[v];
                }
                const K b = warp_max(second);
                if (b) score = key_of(number_of(a) + number_of(b));
            }
            if (lane == g) mine = score;
        }
        int better = 0;
        for (int g = 0; g < p.groups; ++g) {
            const K other = __shfl_sync(FULL, mine, g);
            better += other > mine || (other == mine && g < lane);
        }
        const bool kept = lane < p.groups && better < p.group_topk;
        const unsigned kept_mask = __ballot_sync(FULL, kept);
        if constexpr (!EXACT) {
            // the worst one kept against the best one left out
            const uint32_t worst = __reduce_min_sync(FULL, kept ? (uint32_t)mine : 0xFFFFFFFFu);
            const uint32_t best = __reduce_max_sync(FULL, !kept && lane < p.groups ? (uint32_t)mine : 0u);
            if (best) {
                const float w = number_of(worst), b = number_of(best);
                if (w - b < 4.0f * choice_error(err, w)) sure = false;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = group[v];
            if (!(g < 32 && kept_mask >> g & 1)) key[v] = 0;
            else if (by_logit) key[v] = key[v] ? key_of((T)l[v]) : (K)0;
        }
    } else if (by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l[v] > -INFINITY ? key_of((T)l[v]) : (K)0;
    }
    id = -1;
    K before = 0;
    int before_id = -1;
    const bool check = !EXACT && !by_logit;
    for (int j = 0; j < p.topk + (check ? 1 : 0); ++j) {
        K best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] >= best && key[v]) {
                best = key[v];
                at = v * 32 + lane;
            }
        const K m = warp_max(best);
        if (!m) break;
        const int e = (int)__reduce_min_sync(FULL, best == m ? (unsigned)at : 0x7FFFFFFFu);
        if constexpr (!EXACT) {
            if (check && before) {
                const float x = number_of(before), y = number_of(m);
                if (x - y < 2.0f * choice_error(err, fmaxf(fabsf(x), fabsf(y)))) {
                    // equal logits with equal biases have equal scores in any arithmetic
                    float la = 0.0f, lb = 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (v == before_id / 32) la = l[v];
                        if (v == e / 32) lb = l[v];
                    }
                    la = __shfl_sync(FULL, la, before_id % 32);
                    lb = __shfl_sync(FULL, lb, e % 32);
                    if (la != lb || p.bias[before_id] != p.bias[e]) sure = false;
                }
            }
        }
        before = m;
        before_id = e;
        if (j < p.topk && lane == j) id = e;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 32 + lane == e) key[v] = 0;
    }
    return sure;
}

// The same with keys of 22 bits above 1023 - expert: the keys differ, the largest
// one names its expert, and of equal ones the lowest index comes first.  16-bit
// logits lose nothing that way; else 2^-13 of a number are missing.
template <int V>
__device__ __forceinline__ bool choose_fast(const RouteParams& p, const float (&l)[V], float top, const float* bias, bool exact_keys,
                                            int lane, int& id) {
    constexpr float CUT = 1.3e-4f;
    const bool by_logit = !p.bias;
    uint32_t key[V];
    bool sure = true;
    float err = 0.0f;
    auto packed = [&](float c, int v) { return (key_of(c) & ~1023u) | (uint32_t)(1023 - (v * 32 + lane)); };
    auto number = [](uint32_t k) { return number_of(k & ~1023u); };
    if (!by_logit || p.groups > 1) {
        float s[V];
        if (p.score == ROUTE_SOFTMAX) {
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = l[v] > -INFINITY ? expf(l[v] - top) : 0.0f;
                sum += s[v];
            }
            const float r = 1.0f / warp_sum(sum);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= r;
            err = score_error(p.score, r);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-l[v]));
            err = score_error(p.score, 1.0f);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = by_logit ? 0.0f : bias[v * 32 + lane];
            key[v] = l[v] > -INFINITY && b > -INFINITY ? packed(s[v] + b, v) : 0u;
        }
    }
    if (p.groups > 1) {
        // group g's two largest keys in lane g
        const int size = p.experts / p.groups;
        const bool two = p.group_best > 1;
        uint32_t m1 = 0, m2 = 0;
        unsigned kept_mask;
        auto merge = [&](uint32_t a, uint32_t b) {
            m2 = m1 > a ? (m2 > a ? m2 : a) : (m1 > b ? m1 : b);
            m1 = m1 > a ? m1 : a;
        };
        if (size % 32 == 0) {  // a group is all lanes of some registers
            int g = 0, left = size;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t a = warp_max(key[v]), b = two ? warp_max(key[v] == a ? 0u : key[v]) : 0u;
                if (lane == g) merge(a, b);
                if ((left -= 32) == 0) {
                    left = size;
                    ++g;
                }
            }
        } else {
            int group[V];
#pragma unroll
            for (int v = 0; v < V; ++v) group[v] = (v * 32 + lane) / size;
            for (int g = 0; g < p.groups; ++g) {
                uint32_t first = 0, second = 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (group[v] == g) first = first > key[v] ? first : key[v];
                const uint32_t a = warp_max(first);
                if (two) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (group[v] == g && key[v] != a) second = second > key[v] ? second : key[v];
                    second = warp_max(second);
                }
                if (lane == g) merge(a, second);
            }
        }
        const float score = number(m1) + (two && m2 ? number(m2) : 0.0f);
        const float spread = CUT * (fabsf(number(m1)) + (two && m2 ? fabsf(number(m2)) : 0.0f)) + 2.0f * choice_error(err, score);
        const uint32_t mine = lane < p.groups && m1 ? key_of(score) : 0u;
        int better = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t other = __shfl_sync(FULL, mine, g);
            better += other > mine || (other == mine && g < lane);
        }
        const bool kept = lane < p.groups && better < p.group_topk;
        kept_mask = __ballot_sync(FULL, kept);
        const uint32_t low = __reduce_min_sync(FULL, kept ? key_of(score - spread) : 0xFFFFFFFFu);
        const uint32_t high = warp_max(!kept && mine ? key_of(score + spread) : 0u);
        // (a NaN, of infinities, counts as a number here: then the next try decides)
        if (__any_sync(FULL, lane < p.groups && m1 && !(fabsf(score) < INFINITY))) sure = false;
        if (high && __any_sync(FULL, kept && mine) && !(low > high)) sure = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = size % 32 == 0 ? v * 32 / size : (v * 32 + lane) / size;
            if (!(g < 32 && kept_mask >> g & 1)) key[v] = 0;
            else if (by_logit && key[v]) key[v] = packed(l[v], v);
        }
    } else if (by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l[v] > -INFINITY ? packed(l[v], v) : 0u;
    }
    uint32_t best = 0, before = 0;
    id = -1;
    const int rounds = p.topk + (exact_keys ? 0 : 1);
    for (int j = 0; j < rounds; ++j) {
        // the largest key below the last one
        best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t k = j == 0 || key[v] < before ? key[v] : 0u;
            best = best > k ? best : k;
        }
        const uint32_t m = warp_max(best);
        if (!m) break;
        if (!exact_keys && j > 0) {
            if (by_logit) {
                sure &= (before >> 10) != (m >> 10);
            } else {
                const float x = number(before), y = number(m), most = fmaxf(fabsf(x), fabsf(y));
                sure &= x - y > CUT * most + 2.0f * choice_error(err, most);
            }
        }
        before = m;
        if (lane == j && j < p.topk) id = 1023 - (int)(m & 1023u);
    }
    return sure;
}

template <int V>
__device__ __forceinline__ void load_logits(const RouteParams& p, int t, int lane, float (&l)[V]) {
    const int64_t at = t * p.ld + lane;
    auto load = [&](auto of) {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = v * 32 + lane < p.experts ? of(at + v * 32) : -INFINITY;
    };
    if (p.type == DT_F32)
        load([&](int64_t i) { return static_cast<const float*>(p.L)[i]; });
    else if (p.type == DT_BF16)
        load([&](int64_t i) { return __bfloat162float(static_cast<const __nv_bfloat16*>(p.L)[i]); });
    else
        load([&](int64_t i) { return __half2float(static_cast<const __half*>(p.L)[i]); });
}

// The second and the third try.  (The logits are read again: an array handed to a
// function would live in memory.)
template <int V, typename T>
__device__ __noinline__ int choose_again(const RouteParams& p, int t, float top, int lane, bool& sure) {
    float l[V];
    load_logits<V>(p, t, lane, l);
    int id;
    sure = choose<V, T>(p, l, top, lane, id);
    return id;
}
template <int V>
__device__ __forceinline__ int choose_carefully(const RouteParams& p, int t, float top, int lane) {
    bool sure;
    const int id = choose_again<V, float>(p, t, top, lane, sure);
    return sure ? id : choose_again<V, double>(p, t, top, lane, sure);
}

// Where the experts' rows start: exclusive sums of `count` (block-wide; threads
// >= experts).  start[experts] is the number of rows.
__device__ __forceinline__ void exclusive_sums(const int32_t* count, int32_t* start, int experts, int32_t* carry) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t base = 0;
    for (int e0 = 0; e0 < experts; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        const int32_t n = e < experts ? count[e] : 0;
        int32_t s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t u = __shfl_up_sync(FULL, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) carry[warp] = s;
        __syncthreads();
        int32_t below = base, total = 0;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) {
            if (w < warp) below += carry[w];
            total += carry[w];
        }
        if (e < experts) start[e] = below + s - n;
        base += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) start[experts] = base;
    __syncthreads();
}

// One warp: the rows of entries [first, last), in order; next[e]: expert e's next row.
__device__ __forceinline__ void place(const int32_t* ids, int32_t* rows, int64_t first, int64_t last, volatile int32_t* next,
                                      int lane) {
    for (int64_t i0 = first; i0 < last; i0 += 32) {
        const int64_t i = i0 + lane;
        const int32_t e = i < last ? ids[i] : -1;
        const unsigned same = __match_any_sync(FULL, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int32_t at = e >= 0 ? next[e] : 0;
        __syncwarp();
        if (e >= 0 && rank == 0) next[e] = at + __popc(same);
        __syncwarp();
        if (i < last) rows[i] = e >= 0 ? at + rank : -1;
    }
}

// Block b takes tokens b * tokens_per_block ..; with rows wanted it counts its
// entries by expert.  A single block then finishes the rows itself; several leave
// their counts to route_place_kernel.
template <int V>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_kernel(const __grid_constant__ RouteParams p) {
    __shared__ int32_t count[MOE_MAX_EXPERTS], start[MOE_MAX_EXPERTS + 1], carry[32];
    __shared__ float bias[32 * V];
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (p.offsets)
        for (int e = threadIdx.x; e < p.experts; e += blockDim.x) count[e] = 0;
    griddep_wait();
    bool bias_bad = false;
    if (p.bias)
        for (int e = threadIdx.x; e < 32 * V; e += blockDim.x) {
            bias[e] = e < p.experts ? p.bias[e] : 0.0f;
            bias_bad |= bias[e] != bias[e];
        }
    bias_bad = __syncthreads_or(bias_bad ? 1 : 0) != 0;
    const bool exact_keys = !p.bias && p.type != DT_F32;
    const int t0 = blockIdx.x * p.tokens_per_block;
    const int t1 = p.tokens - t0 < p.tokens_per_block ? p.tokens : t0 + p.tokens_per_block;
    for (int t = t0 + warp; t < t1; t += blockDim.x / 32) {
        float l[V];
        float top = -INFINITY;
        bool bad = bias_bad;
        load_logits<V>(p, t, lane, l);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bad |= l[v] != l[v];
            top = fmaxf(top, l[v]);
        }
        bad = __any_sync(FULL, bad || (p.score == ROUTE_SOFTMAX && top == INFINITY));
        top = number_of(warp_max(key_of(top)));
        int id = -1;
        float w = __uint_as_float(0x7FC00000u);
        if (!bad) {
            if (!choose_fast<V>(p, l, top, bias, exact_keys, lane, id)) id = choose_carefully<V>(p, t, top, lane);
            // weights: lane j has slot j
            const bool have = id >= 0;
            float x = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = __shfl_sync(FULL, l[v], id & 31);
                if (have && v == id / 32) x = u;
            }
            w = 0.0f;
            if (p.renormalize) {
                // relative to the largest chosen logit, so that nothing under- or overflows
                const float most = number_of(warp_max(key_of(x)));
                if (have) {
                    if (p.score == ROUTE_SOFTMAX)
                        w = expf(x - most);
                    else
                        w = x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - fminf(most, 0.0f)) / (1.0f + expf(x));
                }
                const float sum = warp_sum(w);
                if (have) w = w / sum * p.scale;
            } else {
                float sum = 1.0f;
                if (p.score == ROUTE_SOFTMAX) {
                    sum = 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) sum += l[v] > -INFINITY ? expf(l[v] - top) : 0.0f;
                    sum = warp_sum(sum);
                }
                if (have) w = (p.score == ROUTE_SOFTMAX ? expf(x - top) / sum : x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x) / (1.0f + expf(x))) * p.scale;
            }
        }
        if (lane < p.topk) {
            const int64_t i = (int64_t)t * p.topk + lane;
            p.ids[i] = id;
            p.weights[i] = w;
            if (p.offsets && id >= 0) atomicAdd(&count[id], 1);
        }
    }
    if (!p.offsets) return;
    __syncthreads();
    if (p.blocks > 1) {
        for (int e = threadIdx.x; e < p.experts; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.experts + e] = count[e];
        return;
    }
    exclusive_sums(count, start, p.experts, carry);
    for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = start[e];
    __syncthreads();
    if (warp == 0) place(p.ids, p.rows, 0, (int64_t)p.tokens * p.topk, start, lane);
}

// Block b's rows: expert e's start plus what the blocks before it hold of e, then
// one by one.  Every block adds up all counts (integers, so in any order).
__global__ void __launch_bounds__(512) route_place_kernel(const __grid_constant__ RouteParams p) {
    __shared__ int32_t count[MOE_MAX_EXPERTS], before[MOE_MAX_EXPERTS], start[MOE_MAX_EXPERTS + 1], carry[32];
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) count[e] = before[e] = 0;
    __syncthreads();
    griddep_wait();
    // a thread has one expert and every `parts`-th block
    const int threads = (int)blockDim.x;
    for (int e0 = 0; e0 < p.experts; e0 += threads) {
        const int here = p.experts - e0 < threads ? p.experts - e0 : threads, parts = threads / here;
        const int e = e0 + (int)threadIdx.x % here, part = (int)threadIdx.x / here;
        int32_t all = 0, below = 0;
        if (part < parts) {
#pragma unroll 8
            for (int b = part; b < p.blocks; b += parts) {
                const int32_t c = p.counts[(int64_t)b * p.experts + e];
                all += c;
                below += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&count[e], all);
            atomicAdd(&before[e], below);
        }
    }
    __syncthreads();
    exclusive_sums(count, start, p.experts, carry);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = start[e];
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) start[e] += before[e];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
        const int64_t t1 = p.tokens - t0 < p.tokens_per_block ? p.tokens : t0 + p.tokens_per_block;
        place(p.ids, p.rows, t0 * p.topk, t1 * p.topk, start, (int)threadIdx.x);
    }
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t st) {
    const int per = (p.experts + 31) / 32;
    auto go = [&](auto kernel) { return launch_pdl(kernel, p.blocks, 32 * ROUTE_WARPS, 0, st, p); };
    cudaError_t e = per <= 1 ? go(route_kernel<1>) : per <= 2 ? go(route_kernel<2>) : per <= 4 ? go(route_kernel<4>) : per <= 8 ? go(route_kernel<8>) : per <= 16 ? go(route_kernel<16>) : go(route_kernel<32>);
    if (e != cudaSuccess || !p.offsets || p.blocks == 1) return e;
    return launch_pdl(route_place_kernel, p.blocks, 512, 0, st, p);
}

}  // namespace qg
