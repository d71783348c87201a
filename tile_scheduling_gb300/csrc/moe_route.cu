// Routing of tokens to experts, its gradient, and the plan that sorts the routed
// slots by expert.
//
//   s = sigmoid(x) or softmax(x),  c = s + bias  (-inf where x is -inf or NaN)
//   groups: score = the sum of a group's 1 or 2 largest c; the keep best groups stay
//   experts = the top_k largest c of those groups;  w_j = scale * s_j (/ sum_j s_j)
//
// Equal values go to the lower index.  The choice is reproducible to the bit from
// the definition: sigmoid is 1 / (1 + exp(-x)) with each operation rounded to fp32,
// and softmax divides exp(x - max) by a sum that folds the upper half of the
// (zero-padded, power of two, at least 32) expert axis onto the lower one until
// one value is left.
//
// One warp takes one token.  Expert e sits in lane e % 32, slot e / 32, so the
// halving sum is first a tree over a lane's slots, then a butterfly over lanes,
// and a round of the choice is one scan of a lane's slots and two warp
// reductions on order-preserving integer keys.
//
// A token's logits are a few hundred bytes, so instructions bound a batch: at 8191 tokens of
// 128 in bf16, six choices, a scheduler issues in 68 % of its cycles (the gradient: 50 %)
// and memory is at 3 % of its rate.  Launches back to back: that batch 6.2 us and its
// gradient 4.7; 16384 tokens of 256 fp32 logits, eight choices, softmax 16.5 us (18.7 MB,
// 1.1 TB/s) and 10.4, sigmoid 15.9 and 12.2; one token of 256 in eight groups 3.4.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr int kRouteWarps = 4;
constexpr int kMaxRouteExperts = 1024;
constexpr int kMaxTopK = 32;  // lane j of the warp holds choice j
constexpr uint32_t kAll = 0xffffffffu;

struct RouteParams {
    const void *logits;
    int64_t ldx;
    const float *bias;
    int32_t *experts;
    float *weights;
    const float *grad_w;
    void *grad_x;
    int64_t ldg;
    int64_t T;
    int32_t E, k;
    int32_t softmax, renorm;
    int32_t groups, keep, best, group_size;
    uint32_t group_div;  // e / group_size = e * group_div >> 22, exact for e < 1024
    float scale;
    unsigned long long *status;
};

template <class T>
__device__ __forceinline__ float load_logit(const T *x) {
    if constexpr (sizeof(T) == 4)
        return *x;
    else
        return __uint_as_float(uint32_t(*x) << 16);
}

// Unsigned keys in the order of the floats (no NaN; -0 as +0), above 0 for every
// number: 0 stands for "not to be chosen".
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// What a token's softmax scores share.
struct Norm {
    float top, sum;
};

// The score of one logit (x: not NaN, at most the largest number; -inf where masked).
__device__ __forceinline__ float score_of(float x, const Norm &n, bool softmax) {
    if (softmax) return n.sum > 0.f ? expf(x - n.top) / n.sum : 0.f;
    return 1.f / (1.f + expf(-x));
}
__device__ __forceinline__ float clean(float x) { return x > -INFINITY ? fminf(x, 3.402823466e38f) : -INFINITY; }

// Scores of one token: x[i] becomes s of expert i * 32 + lane (if `all`; else only what they
// share is formed); masked[i] tells the experts that cannot be chosen.  Returns whether any
// logit of the row is NaN.
template <int NS>
__device__ __forceinline__ bool scores(float (&x)[NS], bool (&masked)[NS], Norm &norm, bool softmax, bool all = true) {
    bool nan = false;
    norm.top = -3.402823466e38f;
    norm.sum = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        nan |= isnan(x[i]);
        masked[i] = !(x[i] > -INFINITY);
        x[i] = clean(x[i]);  // (+inf as the largest number)
        norm.top = fmaxf(norm.top, x[i]);
    }
    if (softmax) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) norm.top = fmaxf(norm.top, __shfl_xor_sync(kAll, norm.top, d));
        float sum[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            x[i] = expf(x[i] - norm.top);
            sum[i] = x[i];
        }
#pragma unroll
        for (int n = NS / 2; n > 0; n >>= 1) {
#pragma unroll
            for (int i = 0; i < n; ++i) sum[i] += sum[i + n];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[0] += __shfl_xor_sync(kAll, sum[0], d);
        norm.sum = sum[0];
        if (all) {
#pragma unroll
            for (int i = 0; i < NS; ++i) x[i] = sum[0] > 0.f ? x[i] / sum[0] : 0.f;
        }
    } else if (all) {
#pragma unroll
        for (int i = 0; i < NS; ++i) x[i] = score_of(x[i], norm, false);
    }
    return __any_sync(kAll, nan);
}

template <class T, int NS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T *const row = static_cast<const T *>(p.logits) + t * p.ldx;
    float s[NS];
    bool masked[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = i * 32 + lane;
        s[i] = e < p.E ? load_logit(row + e) : -INFINITY;
    }
    Norm norm;
    const bool nan = scores<NS>(s, masked, norm, p.softmax);
    uint32_t key[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = i * 32 + lane;
        float c = s[i];
        if (p.bias && e < p.E) c += __ldg(p.bias + e);
        key[i] = masked[i] || !(c > -INFINITY) ? 0u : key_of(c);
    }
    if (p.groups > 1) {
        // lane g holds the key of group g's score
        uint32_t gkey = 0;
        // the score's key, from this lane's two largest of the group
        auto group_key = [&](uint32_t k1, uint32_t k2) {
            const uint32_t m1 = __reduce_max_sync(kAll, k1);
            if (p.best != 2) return m1;
            const uint32_t owner = __reduce_min_sync(kAll, k1 == m1 ? static_cast<uint32_t>(lane) : kAll);
            const uint32_t m2 = __reduce_max_sync(kAll, lane == owner ? k2 : k1);
            return m2 ? key_of(value_of(m1) + value_of(m2)) : m1;
        };
        if (p.group_size == 32) {
            // a lane has one expert of each group: nothing to search, and the groups' reductions
            // overlap (one token, 256 experts in eight groups: 4.8 us, through the search 5.3)
#pragma unroll
            for (int g = 0; g < NS; ++g) {
                const uint32_t k = group_key(key[g], 0u);
                if (lane == g) gkey = k;
            }
        } else {
            for (int g = 0; g < p.groups; ++g) {
                const int lo = g * p.group_size, hi = lo + p.group_size;
                uint32_t k1 = 0, k2 = 0;  // this lane's two largest of the group
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int e = i * 32 + lane;
                    const uint32_t k = e >= lo && e < hi ? key[i] : 0u;
                    k2 = max(k2, min(k1, k));
                    k1 = max(k1, k);
                }
                const uint32_t k = group_key(k1, k2);
                if (lane == g) gkey = k;
            }
        }
        uint32_t kept = 0;  // bit g: group g stays
        for (int r = 0; r < p.keep; ++r) {
            const uint32_t m = __reduce_max_sync(kAll, gkey);
            if (!m) break;
            const int g = __ffs(__ballot_sync(kAll, gkey == m)) - 1;
            kept |= 1u << g;
            if (lane == g) gkey = 0;
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E && !((kept >> (e * p.group_div >> 22)) & 1u)) key[i] = 0;
        }
    }
    int32_t mine = -1;  // lane j: choice j
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(kAll, best);
        if (!best) break;
        uint32_t at = kAll;  // the lowest of this lane's experts with that key
#pragma unroll
        for (int i = NS - 1; i >= 0; --i)
            if (key[i] == best) at = i * 32 + lane;
        const uint32_t e = __reduce_min_sync(kAll, at);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (i * 32 + lane == e) key[i] = 0;
        if (lane == j) mine = static_cast<int32_t>(e);
    }
    // its score once more, from its logit: one load for a search through the lanes a choice
    float w = mine >= 0 ? score_of(clean(load_logit(row + mine)), norm, p.softmax) : 0.f;
    if (p.renorm) {
        float sum = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < p.k) {
        p.experts[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = nan ? __int_as_float(0x7fffffff) : w * p.scale;
    }
}

// The gradient recomputes the scores.  With g_j = scale * grad_w_j and p_j = s_j / S, S = sum_j s_j:
//   v_j = s_j * d s_j = (g_j - sum_i g_i p_i) * p_j (renorm), else g_j * s_j
//   sigmoid: dx = v * (1 - s);   softmax: dx_e = v_e - s_e * sum_i v_i   (renorm: the sum is 0)
// 1 - s is sigmoid(-x), which keeps its digits where s is close to 1.  Dividing s by S before
// anything multiplies it keeps v finite where S is so small that 1 / S would not be.
template <class T, int NS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const __grid_constant__ RouteParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T *const row = static_cast<const T *>(p.logits) + t * p.ldx;
    float s[NS], x[NS];
    bool masked[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = i * 32 + lane;
        s[i] = e < p.E ? load_logit(row + e) : -INFINITY;
        x[i] = s[i];
    }
    Norm norm;
    const bool every = p.softmax && !p.renorm;  // every expert's score stands in the gradient
    const bool nan = scores<NS>(s, masked, norm, p.softmax, every);
    int32_t mine = -1;
    float g = 0.f;
    if (lane < p.k) {
        mine = p.experts[t * p.k + lane];
        if (mine >= p.E) {
            if (atomicCAS(&p.status[0], 0ull, 7ull) == 0ull)
                atomicExch(&p.status[1], static_cast<unsigned long long>(t * p.k + lane));
            atomicAdd(&p.status[2], 1ull);
            mine = -1;
        }
        if (mine >= 0) g = p.grad_w[t * p.k + lane] * p.scale;
    }
    // lane j: the score of choice j, from its logit
    const float sj = mine >= 0 ? score_of(clean(load_logit(row + mine)), norm, p.softmax) : 0.f;
    float dsj = g * sj, mean = 0.f;
    if (p.renorm) {
        float sum = sj;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        const float share = sum > 0.f ? sj / sum : 0.f;
        float dot = g * share;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(kAll, dot, d);
        dsj = mine >= 0 ? (g - dot) * share : 0.f;
    } else if (p.softmax) {
        mean = dsj;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mean += __shfl_xor_sync(kAll, mean, d);
    }
    float dx[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) dx[i] = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const int e = __shfl_sync(kAll, mine, j);
        const float v = __shfl_sync(kAll, dsj, j);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (i * 32 + lane == e) dx[i] += v;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = i * 32 + lane;
        if (every)
            dx[i] -= s[i] * mean;
        else if (!p.softmax)
            dx[i] = masked[i] ? 0.f : dx[i] * (1.f / (1.f + expf(fminf(x[i], 3.402823466e38f))));
        if (nan) dx[i] = __int_as_float(0x7fffffff);
        if (e < p.E) {
            if constexpr (sizeof(T) == 4)
                static_cast<float *>(p.grad_x)[t * p.ldg + e] = dx[i];
            else
                static_cast<uint16_t *>(p.grad_x)[t * p.ldg + e] =
                    static_cast<uint16_t>(pack_bf16x2(__float_as_uint(dx[i]), 0u));
        }
    }
}

template <bool GRAD, class T>
cudaError_t route_launch(const RouteParams &p, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(cdiv(p.T, kRouteWarps))), block(32 * kRouteWarps);
    auto go = [&](auto ns) {
        constexpr int NS = decltype(ns)::value;
        if constexpr (GRAD)
            return launch_pdl(route_grad_kernel<T, NS>, grid, block, 0, st, p);
        else
            return launch_pdl(route_kernel<T, NS>, grid, block, 0, st, p);
    };
    if (p.E <= 32) return go(std::integral_constant<int, 1>{});
    if (p.E <= 64) return go(std::integral_constant<int, 2>{});
    if (p.E <= 128) return go(std::integral_constant<int, 4>{});
    if (p.E <= 256) return go(std::integral_constant<int, 8>{});
    if (p.E <= 512) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

ts_status route_check(RouteParams &p, const void *logits, int64_t T, int32_t E, int32_t k, int32_t dtype,
                      const ts_route_opts *opts) {
    const ts_route_opts z = {};
    const ts_route_opts *o = opts ? opts : &z;
    if (T < 0 || T > kMaxDim) return fail(TS_ERR_INVALID_ARG, "tokens = %lld", static_cast<long long>(T));
    if (E < 1 || k < 1 || k > E) return fail(TS_ERR_INVALID_ARG, "experts = %d, top_k = %d", E, k);
    if (E > kMaxRouteExperts || k > kMaxTopK)
        return fail(TS_ERR_UNSUPPORTED, "experts = %d (at most %d), top_k = %d (at most %d)", E, kMaxRouteExperts, k,
                    kMaxTopK);
    if (dtype != TS_OUT_BF16 && dtype != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "dtype %d", dtype);
    if (o->score != TS_SCORE_SOFTMAX && o->score != TS_SCORE_SIGMOID)
        return fail(TS_ERR_INVALID_ARG, "score %d", o->score);
    if (o->no_renorm != 0 && o->no_renorm != 1)
        return fail(TS_ERR_INVALID_ARG, "no_renorm = %d (0 or 1)", o->no_renorm);
    const int32_t groups = o->groups ? o->groups : 1, keep = o->keep_groups ? o->keep_groups : groups;
    const int32_t best = o->group_best ? o->group_best : 1;
    if (groups < 1 || E % groups) return fail(TS_ERR_INVALID_ARG, "%d experts do not form %d equal groups", E, groups);
    if (groups > 32) return fail(TS_ERR_UNSUPPORTED, "groups = %d (at most 32)", groups);
    if (keep < 1 || keep > groups || static_cast<int64_t>(keep) * (E / groups) < k)
        return fail(TS_ERR_INVALID_ARG, "keep_groups = %d leaves fewer than top_k = %d experts", keep, k);
    if (best != 1 && best != 2) return fail(TS_ERR_INVALID_ARG, "group_best = %d (1 or 2)", best);
    p.ldx = o->ldx ? o->ldx : E;
    p.ldg = o->ldg ? o->ldg : E;
    if (p.ldx < E || p.ldg < E) return fail(TS_ERR_INVALID_ARG, "leading dimensions must cover a row");
    if (T > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % (dtype == TS_OUT_F32 ? 4 : 2)))
        return fail(TS_ERR_INVALID_ARG, "logits is NULL or not aligned to its element size");
    p.logits = logits;
    p.T = T;
    p.E = E;
    p.k = k;
    p.softmax = o->score == TS_SCORE_SOFTMAX;
    p.renorm = !o->no_renorm;
    p.groups = groups;
    p.keep = keep;
    p.best = best;
    p.group_size = E / groups;
    p.group_div = ((1u << 22) + p.group_size - 1) / p.group_size;
    p.scale = o->scale != 0.f ? o->scale : 1.f;
    p.bias = o->bias;
    ts_status s = TS_OK;
    p.status = T > 0 ? device_status_word(&s) : nullptr;
    return s;
}

// ------------------------------------------------------------------- plan
// A stable counting sort of the slots by expert.  A CTA takes tiles of
// kPlanSlots consecutive slots, a warp kWarpSlots of them in order; equal
// experts of a warp's 32 slots rank by lane.  Latencies bound it (three integers move
// for a slot, and at 49146 slots the two kernels issue in 9 and 18 % of the cycles): 8
// slots 2.7 us, 49146 of 128 experts 7.5, 131072 of 256 12.0, 1048576 of 256 34.5, where
// a tile's 16 x E counts, cleared and walked twice for 1024 slots, add to it.
constexpr int kPlanWarps = 16;
constexpr int kWarpSlots = 64;
constexpr int kPlanSlots = kPlanWarps * kWarpSlots;
constexpr int kOneCtaSlots = 2 * kPlanSlots;  // up to here one CTA does it all
// Up to here every placing CTA sums the tiles' counts itself (two launches); past it that
// reads tiles^2 * E counts and a kernel of its own does it (three).  Two / three launches:
// 128 tiles of 256 experts 11.1 / 12.0 us, of 512 14.9 / 13.0, 256 tiles of 256 24.6 / 14.2.
constexpr int kFusedTiles = 64;

struct PlanParams {
    const int32_t *experts;
    int64_t *offsets;
    int32_t *order, *position;
    int32_t *counts;  // workspace: [tiles][E] counts, then (many tiles) those of the earlier tiles, and [E] sums
    int64_t n;
    int32_t E, tiles;
    unsigned long long *status;
};

// Expert of slot i, or -1 (dropped, past the end, or out of range: reported).
__device__ __forceinline__ int32_t plan_expert(const PlanParams &p, int64_t i, bool report) {
    const int32_t e = i < p.n ? p.experts[i] : -1;
    if (e < p.E) return e;
    if (report) {
        if (atomicCAS(&p.status[0], 0ull, 7ull) == 0ull) atomicExch(&p.status[1], static_cast<unsigned long long>(i));
        atomicAdd(&p.status[2], 1ull);
    }
    return -1;
}

// A thread's slots of a tile: their experts, and the lanes whose slot has the same one.
struct PlanSlots {
    int32_t e[kWarpSlots / 32];
    uint32_t same[kWarpSlots / 32];
};

// Per-warp counts of one tile's slots in hist[warp][E].
__device__ __forceinline__ PlanSlots plan_count(const PlanParams &p, int64_t first, int32_t *hist, bool report) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int32_t i = threadIdx.x; i < kPlanWarps * p.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int32_t *const h = hist + warp * p.E;
    PlanSlots s;
#pragma unroll
    for (int r = 0; r < kWarpSlots / 32; ++r)
        s.e[r] = plan_expert(p, first + warp * kWarpSlots + r * 32 + lane, report);
#pragma unroll
    for (int r = 0; r < kWarpSlots / 32; ++r) {
        s.same[r] = __match_any_sync(kAll, s.e[r]);
        if (s.e[r] >= 0 && lane == __ffs(s.same[r]) - 1) h[s.e[r]] += __popc(s.same[r]);
        __syncwarp();
    }
    __syncthreads();
    return s;
}

// Rows of one tile's slots: hist[warp][e] holds the first row of the warp's slots of e.
__device__ __forceinline__ void plan_place(const PlanParams &p, int64_t first, int32_t *hist, const PlanSlots &s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *const h = hist + warp * p.E;
#pragma unroll
    for (int r = 0; r < kWarpSlots / 32; ++r) {
        const int64_t i = first + warp * kWarpSlots + r * 32 + lane;
        int32_t row = -1;
        if (s.e[r] >= 0) row = h[s.e[r]] + __popc(s.same[r] & ((1u << lane) - 1u));
        __syncwarp();
        if (s.e[r] >= 0 && lane == __ffs(s.same[r]) - 1) h[s.e[r]] += __popc(s.same[r]);
        __syncwarp();
        if (i < p.n) {
            p.position[i] = row;
            if (row >= 0) p.order[row] = static_cast<int32_t>(i);
        }
    }
    __syncthreads();
}

// Turns a tile's counts of expert e, per warp, into the first row of each warp's slots;
// returns the row after the last.
__device__ __forceinline__ int32_t plan_first_rows(const PlanParams &p, int32_t e, int32_t row, int32_t *hist) {
    int32_t n[kPlanWarps];  // all read first: a read behind a write would wait for it
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) n[w] = hist[w * p.E + e];
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        hist[w * p.E + e] = row;
        row += n[w];
    }
    return row;
}

// Exclusive sum over the experts of tot[e] into tot itself and, if `write`, offsets
// (one warp's work: a lane sums its share of the experts, the lanes scan once).
__device__ __forceinline__ void plan_offsets(const PlanParams &p, int32_t *tot, bool write) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int32_t share = (p.E + 31) / 32, e0 = min(lane * share, p.E), e1 = min(e0 + share, p.E);
        int32_t own = 0;
#pragma unroll 4
        for (int32_t e = e0; e < e1; ++e) own += tot[e];
        int32_t run = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(kAll, run, d);
            if (lane >= d) run += o;
        }
        const int32_t all = __shfl_sync(kAll, run, 31);
        run -= own;
        for (int32_t e = e0; e < e1; ++e) {
            const int32_t n = tot[e];
            tot[e] = run;
            if (write) p.offsets[e] = run;
            run += n;
        }
        if (lane == 0) {
            if (write) p.offsets[p.E] = all;
            tot[p.E] = all;
        }
    }
    __syncthreads();
}

// Few slots: one CTA counts, sums and places.
__global__ void __launch_bounds__(32 * kPlanWarps) plan_one_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int32_t smem[];
    int32_t *const hist = smem, *const next = smem + kPlanWarps * p.E;  // next[e]: next free row
    grid_dep_wait();
    grid_dep_launch();
    for (int32_t e = threadIdx.x; e <= p.E; e += blockDim.x) next[e] = 0;
    __syncthreads();  // without a slot there is no tile, and no other barrier before the sums
    for (int32_t t = 0; t < p.tiles; ++t) {
        plan_count(p, static_cast<int64_t>(t) * kPlanSlots, hist, true);
        for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
            int32_t c = next[e];
            for (int w = 0; w < kPlanWarps; ++w) c += hist[w * p.E + e];
            next[e] = c;
        }
        __syncthreads();
    }
    plan_offsets(p, next, true);
    const int32_t valid = next[p.E];
    for (int32_t t = 0; t < p.tiles; ++t) {
        const PlanSlots s = plan_count(p, static_cast<int64_t>(t) * kPlanSlots, hist, false);
        for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) next[e] = plan_first_rows(p, e, next[e], hist);
        __syncthreads();
        plan_place(p, static_cast<int64_t>(t) * kPlanSlots, hist, s);
    }
    for (int64_t r = valid + threadIdx.x; r < p.n; r += blockDim.x) p.order[r] = -1;
}

__global__ void __launch_bounds__(32 * kPlanWarps) plan_count_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int32_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    plan_count(p, static_cast<int64_t>(blockIdx.x) * kPlanSlots, smem, true);
    for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
        int32_t c = 0;
        for (int w = 0; w < kPlanWarps; ++w) c += smem[w * p.E + e];
        p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = c;
    }
}

// Many tiles: a CTA turns the counts of 32 experts into the slots of each in the earlier
// tiles, and sums them.  A lane takes an expert, a warp a run of tiles.
__global__ void __launch_bounds__(1024) plan_scan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ int32_t part[32][33];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t e = static_cast<int32_t>(blockIdx.x) * 32 + lane;
    const int32_t run = (p.tiles + 31) / 32, t0 = min(warp * run, p.tiles), t1 = min(t0 + run, p.tiles);
    int32_t *const column = p.counts + e;
    int32_t c = 0;
    if (e < p.E) {
#pragma unroll 8
        for (int32_t t = t0; t < t1; ++t) c += column[static_cast<int64_t>(t) * p.E];
    }
    part[warp][lane] = c;
    __syncthreads();
    if (e >= p.E) return;
    c = 0;
    for (int w = 0; w < warp; ++w) c += part[w][lane];
    if (warp == 31) column[static_cast<int64_t>(p.tiles) * p.E] = c + part[31][lane];
    for (int32_t t = t0; t < t1; t += 8) {
        int32_t n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = t + i < t1 ? column[static_cast<int64_t>(t + i) * p.E] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t + i < t1) column[static_cast<int64_t>(t + i) * p.E] = c;
            c += n[i];
        }
    }
}

template <bool FUSED>
__global__ void __launch_bounds__(32 * kPlanWarps) plan_place_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int32_t smem[];
    // slots of each expert in all tiles, then its first row; and in the earlier tiles
    __shared__ int32_t tot[kMaxRouteExperts + 1], before[kMaxRouteExperts];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanSlots;
    if constexpr (FUSED) {
        for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) tot[e] = before[e] = 0;
        __syncthreads();
        // the CTA's threads share the tiles of an expert, so that a few loads each, in flight
        // together, cover them
        const int32_t parts = max(static_cast<int32_t>(blockDim.x) / p.E, 1);
        for (int32_t i = threadIdx.x; i < parts * p.E; i += blockDim.x) {
            const int32_t e = i % p.E;
            int32_t all = 0, bef = 0;
#pragma unroll 8
            for (int32_t t = i / p.E; t < p.tiles; t += parts) {
                const int32_t n = p.counts[static_cast<int64_t>(t) * p.E + e];
                if (t < static_cast<int32_t>(blockIdx.x)) bef += n;
                all += n;
            }
            atomicAdd(&tot[e], all);
            atomicAdd(&before[e], bef);
        }
    } else {
        for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
            tot[e] = p.counts[static_cast<int64_t>(p.tiles) * p.E + e];
            before[e] = p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e];
        }
    }
    const PlanSlots s = plan_count(p, first, smem, false);
    plan_offsets(p, tot, blockIdx.x == 0);
    for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) plan_first_rows(p, e, tot[e] + before[e], smem);
    __syncthreads();
    plan_place(p, first, smem, s);
    const int64_t valid = tot[p.E];
    for (int64_t r = first + threadIdx.x; r < first + kPlanSlots && r < p.n; r += blockDim.x)
        if (r >= valid) p.order[r] = -1;
}

}  // namespace
}  // namespace ts

extern "C" {

ts_status ts_moe_route(const void *logits, int32_t *experts, float *weights, int64_t T, int32_t E, int32_t top_k,
                       int32_t dtype, const ts_route_opts *opts, void *stream) {
    using namespace ts;
    RouteParams p = {};
    ts_status s = route_check(p, logits, T, E, top_k, dtype, opts);
    if (s != TS_OK || T == 0) return s;
    if (!experts || !weights || reinterpret_cast<uintptr_t>(experts) % 4 || reinterpret_cast<uintptr_t>(weights) % 4 ||
        reinterpret_cast<uintptr_t>(p.bias) % 4)
        return fail(TS_ERR_INVALID_ARG, "experts, weights or bias is NULL or not aligned to 4 bytes");
    p.experts = experts;
    p.weights = weights;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == TS_OUT_F32 ? route_launch<false, float>(p, st) : route_launch<false, uint16_t>(p, st);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "routing launch");
}

ts_status ts_moe_route_grad(const void *logits, const int32_t *experts, const float *grad_weights, void *grad_logits,
                            int64_t T, int32_t E, int32_t top_k, int32_t dtype, const ts_route_opts *opts,
                            void *stream) {
    using namespace ts;
    RouteParams p = {};
    ts_status s = route_check(p, logits, T, E, top_k, dtype, opts);
    if (s != TS_OK || T == 0) return s;
    if (!experts || !grad_weights || !grad_logits || reinterpret_cast<uintptr_t>(experts) % 4 ||
        reinterpret_cast<uintptr_t>(grad_weights) % 4 ||
        reinterpret_cast<uintptr_t>(grad_logits) % (dtype == TS_OUT_F32 ? 4 : 2))
        return fail(TS_ERR_INVALID_ARG, "experts, grad_weights or grad_logits is NULL or misaligned");
    p.experts = const_cast<int32_t *>(experts);
    p.grad_w = grad_weights;
    p.grad_x = grad_logits;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == TS_OUT_F32 ? route_launch<true, float>(p, st) : route_launch<true, uint16_t>(p, st);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "routing gradient launch");
}

int64_t ts_moe_plan_workspace(int64_t slots, int32_t E) {
    using namespace ts;
    if (slots <= kOneCtaSlots || E < 1) return 0;
    return (cdiv(slots, kPlanSlots) + 1) * E * static_cast<int64_t>(sizeof(int32_t));
}

ts_status ts_moe_plan(const int32_t *experts, int64_t *offsets, int32_t *order, int32_t *position, int64_t slots,
                      int32_t E, void *workspace, int64_t workspace_bytes, void *stream) {
    using namespace ts;
    if (slots < 0 || slots > kMaxDim) return fail(TS_ERR_INVALID_ARG, "slots = %lld", static_cast<long long>(slots));
    if (E < 1) return fail(TS_ERR_INVALID_ARG, "experts = %d", E);
    if (E > kMaxRouteExperts) return fail(TS_ERR_UNSUPPORTED, "experts = %d (at most %d)", E, kMaxRouteExperts);
    if (!offsets || (slots > 0 && (!experts || !order || !position)))
        return fail(TS_ERR_INVALID_ARG, "experts, offsets, order or position is NULL");
    if (reinterpret_cast<uintptr_t>(offsets) % 8 || reinterpret_cast<uintptr_t>(experts) % 4 ||
        reinterpret_cast<uintptr_t>(order) % 4 || reinterpret_cast<uintptr_t>(position) % 4)
        return fail(TS_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
    const int64_t need = ts_moe_plan_workspace(slots, E);
    if (need > 0 && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 4))
        return fail(TS_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", static_cast<long long>(workspace_bytes),
                    static_cast<long long>(need));
    PlanParams p = {};
    ts_status s;
    p.status = device_status_word(&s);
    if (!p.status) return s;
    p.experts = experts;
    p.offsets = offsets;
    p.order = order;
    p.position = position;
    p.counts = static_cast<int32_t *>(workspace);
    p.n = slots;
    p.E = E;
    p.tiles = static_cast<int32_t>(cdiv(slots, kPlanSlots));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 block(32 * kPlanWarps);
    const size_t hist = static_cast<size_t>(kPlanWarps) * E * 4;
    // up to 1024 experts take 68 KB, with 8 KB of static arrays: above the default limit of 48
    static std::atomic<uint64_t> raised{0};  // devices
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    cudaError_t e = cudaSuccess;
    if (hist > 32 * 1024 && !(raised.load(std::memory_order_acquire) & bit)) {
        for (auto *k : {plan_one_kernel, plan_count_kernel, plan_place_kernel<true>, plan_place_kernel<false>})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kPlanWarps * kMaxRouteExperts * 4 + 4 * (kMaxRouteExperts + 1));
        if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_acq_rel);
    }
    if (e == cudaSuccess && need == 0) {
        e = launch_pdl(plan_one_kernel, dim3(1), block, hist + 4 * (E + 1), st, p);
    } else if (e == cudaSuccess) {
        const dim3 grid(static_cast<unsigned>(p.tiles));
        e = launch_pdl(plan_count_kernel, grid, block, hist, st, p);
        if (e == cudaSuccess && p.tiles <= kFusedTiles) {
            e = launch_pdl(plan_place_kernel<true>, grid, block, hist, st, p);
        } else if (e == cudaSuccess) {
            e = launch_pdl(plan_scan_kernel, dim3(static_cast<unsigned>(cdiv(E, 32))), dim3(1024), 0, st, p);
            if (e == cudaSuccess) e = launch_pdl(plan_place_kernel<false>, grid, block, hist, st, p);
        }
    }
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "plan launch");
}

}  // extern "C"
