// Routing: every token's topk experts, their weights, and the rows of the
// (token, slot) pairs sorted by expert.
//
// A warp takes a token; lane i holds experts i, i + 32, ...  Scores are numbers
// turned into unsigned keys of the same order (0: never chosen), so that a round
// of the choice is a warp-wide integer maximum.
//
// The choice is defined in 64 bits.  Without a bias it is the logits' own order,
// which fp32 holds exactly.  With one (and for groups' scores) it is that of sums
// whose error fp32 leaves open.  So, each only where the one before cannot tell:
//   1. keys of 22 bits with the expert's number below them: a round is one maximum
//      that names its expert;
//   2. where neighbours in that order are too near, a lane takes each of the
//      candidates and compares 32-bit keys (a token in ten or twenty);
//   3. ... and 64-bit scores (one in a thousand).
// All scores in 64 bits would take several times the time (16 tokens of 256 experts that
// all need them 46 us, else 9): this GPU has little 64-bit arithmetic.
// What bounds it: 4001 x 256 logits are 4 MB, 0.6 us, and take 18.7 to 25.7 us with bias and
// groups, 12.5 without.  With them the choice takes half of that: some 1900
// instructions a token of 256 experts, which the schedulers issue in 58% of their cycles;
// the rest is latency, above all the block's wait for its longest token (the stall
// sampled most is the barrier behind the loop).  The rows take the other half: a launch
// whose schedulers issue in 29% of the cycles, waiting for counts and for one warp a
// block that places its pairs.  16 x 8 tokens 3 us, one block.
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

// A bound of the fp32 error of a token's scores s, without the part that grows with
// c.  Sigmoid: the exponential is off by 2 units, s (1 - s) 2^-22 <= 2^-24, a sum and a
// quotient by half a unit each: below 2e-7.  Softmax: the exponential's argument is off
// by up to 2^-24 |l - max| (x e^-x is at most 0.37), the exponential by 2 units, a sum of
// E <= 1024 of them by 37 roundings at most, the quotient by one: below 3e-6 s.
__device__ __forceinline__ float score_error(int32_t score, float largest) { return score == ROUTE_SOFTMAX ? 4e-6f * largest : 4e-7f; }
// ... of c = s + bias.
__device__ __forceinline__ float choice_error(float err, float c) { return err + 1.2e-7f * fabsf(c); }

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

// A score in fp32 or in 64 bits.  total: softmax's sum.
template <typename T>
__device__ __forceinline__ T score_of(int32_t kind, float l, float top, T total) {
    return kind == ROUTE_SOFTMAX ? exp_t((T)l - (T)top) / total : (T)1 / ((T)1 + exp_t(-(T)l));
}

// Groups kept, as a mask, by keys of all choice scores.  sure: fp32's error leaves
// no doubt (err: that of one score; 0 for keys in 64 bits).
template <int V, typename K>
__device__ __forceinline__ unsigned keep_groups(const RouteParams& p, const K (&key)[V], float err, int lane, bool& sure) {
    const int size = p.experts / p.groups;
    const bool two = p.group_best > 1;
    K m1 = 0, m2 = 0;  // group g's two largest keys, in lane g
    auto merge = [&](K a, K b) {
        m2 = m1 > a ? (m2 > a ? m2 : a) : (m1 > b ? m1 : b);
        m1 = m1 > a ? m1 : a;
    };
    if (size % 32 == 0) {  // a group is all lanes of some registers
        int g = 0, left = size;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const K a = warp_max(key[v]);
            K b = 0;
            if (two) {
                const unsigned have = __ballot_sync(FULL, key[v] == a);
                b = __popc(have) > 1 ? a : warp_max(key[v] == a ? (K)0 : key[v]);
            }
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
            K first = 0, second = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (group[v] == g) {
                    second = key[v] > first ? first : (key[v] > second ? key[v] : second);
                    first = key[v] > first ? key[v] : first;
                }
            const K a = warp_max(first);
            K b = 0;
            if (two) {
                const unsigned have = __ballot_sync(FULL, first == a);
                b = __popc(have) > 1 ? a : warp_max(first == a ? second : first);
            }
            if (lane == g) merge(a, b);
        }
    }
    const auto score = two && m2 ? number_of(m1) + number_of(m2) : number_of(m1);
    const K mine = lane < p.groups && m1 ? key_of(score) : (K)0;
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
        const K other = __shfl_sync(FULL, mine, g);
        better += other > mine || (other == mine && g < lane);
    }
    const bool kept = lane < p.groups && better < p.group_topk;
    if (err > 0.0f) {
        // A group's score is off by what its one or two c are, each by its own size (they
        // may cancel), and by the sum's rounding.  Every group kept against the best one
        // left out, which may be any whose error reaches so high.
        const bool both = two && m2;
        const float size = fabsf((float)number_of(m1)) + (both ? fabsf((float)number_of(m2)) : 0.0f), x = (float)score;
        const float off = m1 ? choice_error(both ? 2.0f * err : err, size + fabsf(x)) : 0.0f;
        const K high = warp_max(!kept ? mine : (K)0);
        const float most = __uint_as_float(warp_max(!kept && mine ? __float_as_uint(off) : 0u));
        // (with a live one left out, all groups kept are live)
        if (high && __any_sync(FULL, kept && !(x - (float)number_of(high) > off + most))) sure = false;
    }
    return __ballot_sync(FULL, kept);
}

// The choice from 64-bit scores of all experts: slot j's expert in lane j.
template <int V>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int t, float top, int lane) {
    float l[V];
    uint64_t key[V];
    load_logits<V>(p, t, lane, l);
    double total = 0.0;
    if (p.score == ROUTE_SOFTMAX) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (l[v] > -INFINITY) total += exp((double)l[v] - (double)top);
        total = warp_sum(total);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float b = p.bias && v * 32 + lane < p.experts ? p.bias[v * 32 + lane] : 0.0f;
        key[v] = l[v] > -INFINITY && b > -INFINITY ? key_of(score_of<double>(p.score, l[v], top, total) + (double)b) : 0ull;
    }
    if (p.groups > 1) {
        bool sure = true;
        const unsigned kept = keep_groups<V>(p, key, 0.0f, lane, sure);
        const int size = p.experts / p.groups;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (v * 32 + lane) / size;
            if (!(g < 32 && kept >> g & 1)) key[v] = 0;
        }
    }
    if (!p.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] ? (uint64_t)key_of(l[v]) : 0ull;
    }
    int id = -1;
    for (int j = 0; j < p.topk; ++j) {
        uint64_t best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] >= best && key[v]) {
                best = key[v];
                at = v * 32 + lane;
            }
        const uint64_t m = warp_max(best);
        if (!m) break;
        const int e = (int)__reduce_min_sync(FULL, best == m ? (unsigned)at : 0x7FFFFFFFu);
        if (lane == j) id = e;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 32 + lane == e) key[v] = 0;
    }
    return id;
}

// Lane j < n has candidate `id` and its key: puts them into order, ties to the lowest
// index.
template <typename K>
__device__ __forceinline__ void sort_candidates(int n, int lane, int& id, K& key, float& l, float& b) {
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const K other = __shfl_sync(FULL, key, i);
        const int e = __shfl_sync(FULL, id, i);
        rank += other > key || (other == key && e < id);
    }
    int from = lane;
    for (int i = 0; i < n; ++i)
        if (__shfl_sync(FULL, rank, i) == lane) from = i;
    id = __shfl_sync(FULL, id, from);
    key = __shfl_sync(FULL, key, from);
    l = __shfl_sync(FULL, l, from);
    b = __shfl_sync(FULL, b, from);
}

// The order of n <= 32 candidates, among which the topk are.  Slot j's expert in
// lane j.
template <int V>
__device__ __noinline__ int choose_among(const RouteParams& p, int t, float top, float total, float err, int n, int id, int lane) {
    const bool mine = lane < n;
    float l = mine ? ld_elem(p.L, p.type, t * p.ld + id) : 0.0f;
    float b = mine && p.bias ? p.bias[id] : 0.0f;
    const float c = p.bias ? score_of<float>(p.score, l, top, total) + b : l;
    uint32_t key = mine ? key_of(c) : 0u;
    sort_candidates(n, lane, id, key, l, b);
    bool doubt = false;
    if (p.bias) {
        // against the next one: equal logits with equal biases have equal scores in any
        // arithmetic
        const float x = number_of(key), y = number_of(__shfl_down_sync(FULL, key, 1));
        // (all lanes take part in both exchanges)
        const float next_l = __shfl_down_sync(FULL, l, 1), next_b = __shfl_down_sync(FULL, b, 1);
        const bool same = l == next_l && b == next_b;
        const bool near = lane + 1 < n && !(x - y > 2.0f * choice_error(err, fmaxf(fabsf(x), fabsf(y))));
        // The last slot's run goes on for as long as neighbours are near, equal ones among
        // them: what stands in doubt anywhere in it may belong before it.  Behind a
        // neighbour that is certainly smaller nothing can.
        const unsigned run = __ballot_sync(FULL, near) >> (p.topk - 1);
        const int end = p.topk - 1 + __ffs((int)~run) - 1;  // (lane 31 has no next one)
        doubt = near && !same && lane < end;
    }
    if (__any_sync(FULL, doubt)) {
        double sum = 0.0;
        if (p.score == ROUTE_SOFTMAX) {
            float all[V];
            load_logits<V>(p, t, lane, all);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (all[v] > -INFINITY) sum += exp((double)all[v] - (double)top);
            sum = warp_sum(sum);
        }
        uint64_t exact = lane < n ? key_of(score_of<double>(p.score, l, top, sum) + (double)b) : 0ull;
        sort_candidates(n, lane, id, exact, l, b);
    }
    return lane < p.topk && lane < n ? id : -1;
}

// Choose for one token.  l: this lane's logits (-inf past the last expert).  Slot
// j's expert in lane j (-1: none).  V: experts a lane.
//
// Keys of 22 bits lie above 1023 - expert: all differ, and of equal ones the lowest
// index comes first.  16-bit logits lose nothing that way; else 2^-13 of a number
// are missing.
template <int V>
__device__ __forceinline__ int choose(const RouteParams& p, int t, const float (&l)[V], float top, const float* bias, bool exact_keys, int lane) {
    constexpr float CUT = 1.3e-4f;
    const bool by_logit = !p.bias;
    uint32_t key[V];
    float err = 0.0f, total = 1.0f;
    if (!by_logit || p.groups > 1) {
        float s[V];
        if (p.score == ROUTE_SOFTMAX) {
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = l[v] > -INFINITY ? expf(l[v] - top) : 0.0f;
                sum += s[v];
            }
            total = warp_sum(sum);
            const float r = 1.0f / total;
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
            key[v] = l[v] > -INFINITY && b > -INFINITY ? key_of(s[v] + b) : 0u;
        }
    }
    if (p.groups > 1) {
        bool sure = true;
        const unsigned kept = keep_groups<V>(p, key, err, lane, sure);
        if (!sure) return choose_exactly<V>(p, t, top, lane);
        const int size = p.experts / p.groups;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = size % 32 == 0 ? v * 32 / size : (v * 32 + lane) / size;
            if (!(g < 32 && kept >> g & 1)) key[v] = 0;
            else if (by_logit && key[v]) key[v] = key_of(l[v]);
        }
    } else if (by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l[v] > -INFINITY ? key_of(l[v]) : 0u;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] ? (key[v] & ~1023u) | (uint32_t)(1023 - (v * 32 + lane)) : 0u;
    int id = -1, n = 0;
    uint32_t before = 0xFFFFFFFFu, last = 0;  // last: the key of slot topk - 1
    bool doubt = false;
    for (int round = 0; round <= 32; ++round) {  // (ends before: n goes up)
        // the largest key below the one before
        uint32_t best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t k = key[v] < before ? key[v] : 0u;
            best = best > k ? best : k;
        }
        const uint32_t m = warp_max(best);
        if (!m) break;
        if (!exact_keys && n > 0) {
            // whether the order of two neighbours (beyond topk: of slot topk - 1 and this
            // one) is certain
            const uint32_t a = n <= p.topk ? before : last;
            bool certain;
            if (by_logit) {
                certain = a >> 10 != m >> 10;
            } else {
                const float x = number_of(a & ~1023u), y = number_of(m & ~1023u), most = fmaxf(fabsf(x), fabsf(y));
                certain = x - y > CUT * most + 2.0f * choice_error(err, most);
            }
            if (n >= p.topk && certain) break;
            doubt |= !certain;
        }
        if (n == 32) return choose_exactly<V>(p, t, top, lane);
        if (lane == n) id = 1023 - (int)(m & 1023u);
        before = m;
        if (++n == p.topk) {
            last = m;
            if (exact_keys) break;
        }
    }
    if (doubt) return choose_among<V>(p, t, top, total, err, n, id, lane);
    return lane < p.topk ? id : -1;
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

// One warp: the rows of n entries, in order; next[e]: expert e's next row; mask: a
// zero per expert.  near: the first `staged` entries, in shared memory.
__device__ __forceinline__ void place(const int32_t* ids, const int32_t* near, int staged, int32_t* rows, int n, volatile int32_t* next,
                                      volatile uint32_t* mask, int lane) {
    auto entry = [&](int i) { return i >= n ? -1 : i < staged ? near[i] : ids[i]; };
    int32_t e = entry(lane);
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int32_t after = entry(i + 32);  // on its way during this round
        // the lanes that have the same expert (an instruction that finds them takes ten
        // times as long)
        if (e >= 0) atomicOr(const_cast<uint32_t*>(&mask[e]), 1u << lane);
        __syncwarp();
        const uint32_t same = e >= 0 ? mask[e] : 0u;
        const int32_t at = e >= 0 ? next[e] : 0;
        const int rank = __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && rank == 0) {
            next[e] = at + __popc(same);
            mask[e] = 0;
        }
        __syncwarp();
        if (i < n) rows[i] = e >= 0 ? at + rank : -1;
        e = after;
    }
}

// Block b takes tokens b * tokens_per_block ..; with rows wanted it counts its
// entries by expert.  A single block then finishes the rows itself; several leave
// their counts to route_place_kernel.
template <int V>
__global__ void __launch_bounds__(V <= 8 ? 1024 : 512) route_kernel(const __grid_constant__ RouteParams p) {
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
            id = choose<V>(p, t, l, top, bias, exact_keys, lane);
            // weights: lane j has slot j
            const bool have = id >= 0;
            const float x = have ? ld_elem(p.L, p.type, t * p.ld + id) : -INFINITY;
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
        for (int e = threadIdx.x; e < p.pitch; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.pitch + e] = e < p.experts ? (uint16_t)count[e] : (uint16_t)0;
        return;
    }
    exclusive_sums(count, start, p.experts, carry);
    for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = start[e];
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) count[e] = 0;
    __syncthreads();
    if (warp == 0) place(p.ids, nullptr, 0, p.rows, p.tokens * p.topk, start, reinterpret_cast<uint32_t*>(count), lane);
}

// Block b's rows: expert e's start plus what the blocks before it hold of e, then
// one by one.  Every block adds up all counts (integers, so in any order).
constexpr int PLACE_THREADS = 512;
__global__ void __launch_bounds__(PLACE_THREADS) route_place_kernel(const __grid_constant__ RouteParams p) {
    // sums of a thread's share of the blocks, eight experts each: of all, and of those
    // before this one
    __shared__ __align__(16) int32_t share[2][PLACE_THREADS * 8];
    __shared__ int32_t count[MOE_MAX_EXPERTS], start[MOE_MAX_EXPERTS + 1], carry[32], near[PLACE_THREADS];
    griddep_launch_dependents();
    const int tid = (int)threadIdx.x;
    const int octets = p.pitch / 8, parts = PLACE_THREADS / octets, part = tid / octets, o = tid % octets;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
    const int64_t t1 = p.tokens - t0 < p.tokens_per_block ? p.tokens : t0 + p.tokens_per_block;
    const int n = (int)(t1 - t0) * p.topk;
    const int32_t* ids = p.ids + t0 * p.topk;
    griddep_wait();
    const int32_t first = tid < n ? ids[tid] : -1;
    int32_t all[8] = {}, below[8] = {};
    if (part < parts) {
#pragma unroll 8
        for (int b = part; b < p.blocks; b += parts) {
            const uint4 c = reinterpret_cast<const uint4*>(p.counts + (int64_t)b * p.pitch)[o];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            const bool earlier = b < (int)blockIdx.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t x = (int32_t)(w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
                all[i] += x;
                below[i] += earlier ? x : 0;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<int4*>(&share[0][tid * 8 + i]) = make_int4(all[i], all[i + 1], all[i + 2], all[i + 3]);
        *reinterpret_cast<int4*>(&share[1][tid * 8 + i]) = make_int4(below[i], below[i + 1], below[i + 2], below[i + 3]);
    }
    near[tid] = first;
    __syncthreads();
    int32_t before[2] = {0, 0};  // of experts tid and tid + 512
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = tid + k * PLACE_THREADS;
        if (e < p.experts) {
            int32_t sum = 0;
            for (int q = 0; q < parts; ++q) {
                sum += share[0][q * p.pitch + e];
                before[k] += share[1][q * p.pitch + e];
            }
            count[e] = sum;
        }
    }
    __syncthreads();
    exclusive_sums(count, start, p.experts, carry);
    if (blockIdx.x == 0)
        for (int e = tid; e <= p.experts; e += PLACE_THREADS) p.offsets[e] = start[e];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = tid + k * PLACE_THREADS;
        if (e < p.experts) {
            start[e] += before[k];
            count[e] = 0;
        }
    }
    __syncthreads();
    if (tid < 32) place(ids, near, PLACE_THREADS, p.rows + t0 * p.topk, n, start, reinterpret_cast<uint32_t*>(count), tid);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t st) {
    const int per = (p.experts + 31) / 32;
    auto go = [&](auto kernel) { return launch_pdl(kernel, p.blocks, p.blocks == 1 ? 512 : route_threads(p.experts), 0, st, p); };
    cudaError_t e = per <= 1 ? go(route_kernel<1>) : per <= 2 ? go(route_kernel<2>) : per <= 4 ? go(route_kernel<4>) : per <= 8 ? go(route_kernel<8>) : per <= 16 ? go(route_kernel<16>) : go(route_kernel<32>);
    if (e != cudaSuccess || !p.offsets || p.blocks == 1) return e;
    return launch_pdl(route_place_kernel, p.blocks, PLACE_THREADS, 0, st, p);
}

}  // namespace qg
