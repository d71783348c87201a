// The way back from the experts: each token's weighted sum of its experts' rows,
// and its gradient.
//
//   out[t] = sum_j w[t][j] * y[position[t][j]]            (slots with position < 0 are dropped)
//   grad_y[position[t][j]] = w[t][j] * grad_out[t],   grad_w[t][j] = <grad_out[t], y[position[t][j]]>
//
// Both are bound by memory: each row of y moves once.  8192 tokens, four slots, rows of
// 4096 bf16: 54 us (335 MB, 6.2 TB/s), the gradient 98 us (604 MB, 6.1 TB/s); 32 tokens of
// eight slots 2.7 us.  Sums run in fp32, a token's slots in order, so results do not depend
// on timing.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr int kThreads = 256, kGradThreads = 512, kGradSlots = 4;

struct CombineParams {
    const void *y, *grad_out;
    void *out, *grad_y;
    float *grad_w;
    const float *w;  // nullptr: every weight is 1
    const int32_t *position;
    int64_t T, N, R;
    int64_t ldy, ldo, ldg;  // rows of y, of out (or grad_out), of grad_y
    int32_t k;
    unsigned long long *status;
};

// A thread's values of a row as they lie in memory, in units of U bytes: what the rows'
// starts are aligned to.  Units of 16 bytes: one.  Smaller: several, 32 units apart, so
// that a warp's loads and stores of one unit each still fill whole sectors (8192 tokens,
// eight slots of bf16, combine and gradient: 4096 values 107 and 182 us, 4092 128 and 203,
// 4094 141 and 221, 4095 167 and 282; 4095 with eight neighbours a thread 278 and 727).
template <class T, int U>
struct Vals {
    static constexpr int UE = U / sizeof(T), COUNT = U == 2 ? 4 : 16 / sizeof(T), UNITS = COUNT / UE;
    static constexpr bool PACKED = sizeof(T) == 2 && UE > 1;  // two bf16 a word, else a value a word
    static constexpr int UW = PACKED ? UE / 2 : UE;           // words of a unit
    uint32_t w[UNITS * UW];

    // a thread's first column among those of its CTA
    static __device__ __forceinline__ int64_t first(int thread) {
        return int64_t(thread & ~31) * COUNT + (thread & 31) * UE;
    }
    // those of row x from column c on; the ones past the N-th read as 0
    __device__ __forceinline__ void load(const T *x, int64_t c, int64_t N) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t at = c + u * (32 * UE);
            uint32_t *const o = w + u * UW;
            if constexpr (UE == 1) {
                const T v = at < N ? x[at] : T(0);
                if constexpr (sizeof(T) == 4)
                    o[0] = __float_as_uint(v);
                else
                    o[0] = v;
            } else if (at + UE <= N) {
                if constexpr (U == 16) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(x + at));
                    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
                } else if constexpr (U == 8) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(x + at);
                    o[0] = v.x, o[1] = v.y;
                } else {
                    o[0] = *reinterpret_cast<const uint32_t *>(x + at);
                }
            } else {
#pragma unroll
                for (int i = 0; i < UW; ++i) o[i] = 0u;
#pragma unroll
                for (int i = 0; i < UE; ++i)
                    if (at + i < N) {
                        if constexpr (sizeof(T) == 4)
                            o[i] = __float_as_uint(x[at + i]);
                        else
                            o[i >> 1] |= uint32_t(x[at + i]) << (16 * (i & 1));
                    }
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        if constexpr (!PACKED) return __uint_as_float(w[i] << 16);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    static __device__ __forceinline__ void store(T *x, int64_t c, int64_t N, const float (&v)[COUNT]) {
        uint32_t r[UNITS * UW];
#pragma unroll
        for (int i = 0; i < UNITS * UW; ++i) {
            if constexpr (sizeof(T) == 4)
                r[i] = __float_as_uint(v[i]);
            else if constexpr (PACKED)
                r[i] = pack_bf16x2(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
            else
                r[i] = pack_bf16x2(__float_as_uint(v[i]), 0u);
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t at = c + u * (32 * UE);
            const uint32_t *const o = r + u * UW;
            if constexpr (UE == 1) {
                if (at < N) {
                    if constexpr (sizeof(T) == 4)
                        x[at] = __uint_as_float(o[0]);
                    else
                        x[at] = static_cast<T>(o[0]);
                }
            } else if (at + UE <= N) {
                if constexpr (U == 16)
                    __stcs(reinterpret_cast<uint4 *>(x + at), make_uint4(o[0], o[1], o[2], o[3]));
                else if constexpr (U == 8)
                    *reinterpret_cast<uint2 *>(x + at) = make_uint2(o[0], o[1]);
                else
                    *reinterpret_cast<uint32_t *>(x + at) = o[0];
            } else {
#pragma unroll
                for (int i = 0; i < UE; ++i)
                    if (at + i < N) {
                        if constexpr (sizeof(T) == 4)
                            x[at + i] = __uint_as_float(o[i]);
                        else
                            x[at + i] = static_cast<T>(o[i >> 1] >> (16 * (i & 1)));
                    }
            }
        }
    }
};

// The row of y that slot (t, j) takes, or -1.
__device__ __forceinline__ int32_t slot_row(const CombineParams &p, int64_t t, int32_t j) {
    if (j >= p.k) return -1;
    const int32_t at = p.position[t * p.k + j];
    if (at >= p.R) {
        if (threadIdx.x == 0) {
            if (atomicCAS(&p.status[0], 0ull, 6ull) == 0ull)
                atomicExch(&p.status[1], static_cast<unsigned long long>(t * p.k + j));
            atomicAdd(&p.status[2], 1ull);
        }
        return -1;
    }
    return at;
}

// One CTA per token and kThreads threads' columns.  KS: slots whose rows are in
// flight together (raw, four registers each, so that several CTAs fit an SM).
template <class T, int KS, int U>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p) {
    using Row = Vals<T, U>;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t = blockIdx.x;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x * Row::COUNT + Row::first(threadIdx.x);
    float sum[Row::COUNT];
#pragma unroll
    for (int i = 0; i < Row::COUNT; ++i) sum[i] = 0.f;
    for (int32_t j0 = 0; j0 < p.k; j0 += KS) {
        Row v[KS];
        float w[KS];
        int32_t at[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            at[j] = slot_row(p, t, j0 + j);
            w[j] = at[j] >= 0 && p.w ? p.w[t * p.k + j0 + j] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
            if (at[j] >= 0) v[j].load(static_cast<const T *>(p.y) + at[j] * p.ldy, c, p.N);
#pragma unroll
        for (int j = 0; j < KS; ++j)
            if (at[j] >= 0) {
#pragma unroll
                for (int i = 0; i < Row::COUNT; ++i) sum[i] = fmaf(w[j], v[j][i], sum[i]);
            }
    }
    if (c < p.N) Row::store(static_cast<T *>(p.out) + t * p.ldo, c, p.N, sum);
}

// One CTA per token: grad_out's row is read for each group of four slots (from L2 after
// the first; eight at once would leave room for one CTA on an SM), the slots' dot products
// are reduced in fixed order.
//
// Registers: 56 (three CTAs of 384 threads: 4096 tokens, four slots of 2880 36.1 us, 43.5
// with 64); with a limit of 64 single values take 56 too, and less time (4095: 282 us, 368).
template <class T, int U>
__global__ void __maxnreg__(U == 2 ? 64 : 56) combine_grad_kernel(const __grid_constant__ CombineParams p) {
    using Row = Vals<T, U>;
    __shared__ float part[kGradSlots][kGradThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    constexpr int KS = kGradSlots;
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int32_t j0 = 0; j0 < p.k; j0 += KS) {
        int32_t at[KS];
        float w[KS], dot[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            at[j] = slot_row(p, t, j0 + j);
            w[j] = at[j] >= 0 && p.w ? p.w[t * p.k + j0 + j] : 1.f;
            dot[j] = 0.f;
        }
#pragma unroll 1
        for (int64_t c = Row::first(threadIdx.x); c < p.N; c += static_cast<int64_t>(blockDim.x) * Row::COUNT) {
            Row g, y[KS];
            g.load(static_cast<const T *>(p.grad_out) + t * p.ldo, c, p.N);
#pragma unroll
            for (int j = 0; j < KS; ++j)
                if (at[j] >= 0) y[j].load(static_cast<const T *>(p.y) + at[j] * p.ldy, c, p.N);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                if (at[j] < 0) continue;
                float o[Row::COUNT];
#pragma unroll
                for (int i = 0; i < Row::COUNT; ++i) {
                    const float x = g[i];
                    dot[j] = fmaf(x, y[j][i], dot[j]);
                    o[i] = w[j] * x;
                }
                Row::store(static_cast<T *>(p.grad_y) + at[j] * p.ldg, c, p.N, o);
            }
        }
        if (p.grad_w) {
#pragma unroll
            for (int j = 0; j < KS; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                if (lane == 0) part[j][warp] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < KS && j0 + static_cast<int>(threadIdx.x) < p.k) {
                float s = 0.f;
                for (unsigned i = 0; i < blockDim.x / 32; ++i) s += part[threadIdx.x][i];
                p.grad_w[t * p.k + j0 + threadIdx.x] = s;  // 0 for a dropped slot
            }
            __syncthreads();
        }
    }
}

// Threads of a CTA: the row's vectors shared evenly by as few rounds (or CTAs) as `most`
// threads need, in warps: 1795 tokens, four slots of 2360 bf16 8.9 us; with `most` threads
// and a last CTA that is mostly idle 13.4.
int cta_threads(int64_t N, int per, int most) {
    const int64_t vectors = cdiv(N, per);
    return static_cast<int>(cdiv(cdiv(vectors, cdiv(vectors, most)), 32) * 32);
}

// Bytes (16, 8, 4 or the element) that both the base and the pitch of rows are multiples of.
int row_unit(const void *x, int64_t ld, int esize) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(ld * esize);
    int u = 16;
    while (u > esize && bits % u) u /= 2;
    return u;
}
int values_of(int unit, int esize) { return unit == 2 ? 4 : 16 / esize; }

// Calls f with the unit as a compile-time constant.
template <class F>
cudaError_t with_unit(int unit, F &&f) {
    switch (unit) {
        case 16: return f(std::integral_constant<int, 16>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 2>{});
    }
}

template <class T>
cudaError_t combine_launch(const CombineParams &p, int unit, dim3 grid, dim3 block, cudaStream_t st) {
    return with_unit(unit, [&](auto u) {
        constexpr int U = decltype(u)::value < static_cast<int>(sizeof(T)) ? static_cast<int>(sizeof(T)) : decltype(u)::value;
        return launch_pdl(p.k <= 4 ? combine_kernel<T, 4, U> : combine_kernel<T, 8, U>, grid, block, 0, st, p);
    });
}

template <class T>
cudaError_t combine_grad_launch(const CombineParams &p, int unit, dim3 grid, dim3 block, cudaStream_t st) {
    return with_unit(unit, [&](auto u) {
        constexpr int U = decltype(u)::value < static_cast<int>(sizeof(T)) ? static_cast<int>(sizeof(T)) : decltype(u)::value;
        return launch_pdl(combine_grad_kernel<T, U>, grid, block, 0, st, p);
    });
}

ts_status combine_check(int64_t T, int32_t k, int64_t N, int64_t R, int32_t dtype, int64_t ldy, int64_t ldo,
                        int64_t ldg) {
    if (T < 0 || N < 0 || R < 0 || T > kMaxDim || N > kMaxDim || R > kMaxDim)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^31-1] (T=%lld N=%lld R=%lld)",
                    static_cast<long long>(T), static_cast<long long>(N), static_cast<long long>(R));
    if (k < 0 || k > 1024) return fail(TS_ERR_INVALID_ARG, "top_k = %d (0 to 1024)", k);
    if (dtype != TS_OUT_BF16 && dtype != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "dtype %d", dtype);
    if (ldy < N || ldo < N || ldg < N)
        return fail(TS_ERR_INVALID_ARG, "leading dimensions must cover a row (%lld, %lld, %lld)",
                    static_cast<long long>(ldy), static_cast<long long>(ldo), static_cast<long long>(ldg));
    return TS_OK;
}

}  // namespace
}  // namespace ts

extern "C" {

ts_status ts_moe_combine(const void *y, const int32_t *position, const float *weights, void *out, int64_t T,
                         int32_t top_k, int64_t N, int64_t R, int32_t dtype, int64_t ldy, int64_t ldo, void *stream) {
    using namespace ts;
    ldy = ldy ? ldy : N;
    ldo = ldo ? ldo : N;
    ts_status s = combine_check(T, top_k, N, R, dtype, ldy, ldo, N);
    if (s != TS_OK) return s;
    if (T == 0 || N == 0) return TS_OK;
    const int esize = dtype == TS_OUT_F32 ? 4 : 2;
    if (!out || (top_k > 0 && !position) || (R > 0 && !y))
        return fail(TS_ERR_INVALID_ARG, "y, position or out is NULL");
    if (reinterpret_cast<uintptr_t>(out) % esize || reinterpret_cast<uintptr_t>(y) % esize ||
        reinterpret_cast<uintptr_t>(position) % 4 || reinterpret_cast<uintptr_t>(weights) % 4)
        return fail(TS_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
    if (R > 0 && ranges_overlap(out, ((T - 1) * ldo + N) * esize, y, ((R - 1) * ldy + N) * esize))
        return fail(TS_ERR_INVALID_ARG, "out overlaps y");
    CombineParams p = {};
    p.status = device_status_word(&s);
    if (!p.status) return s;
    p.y = y;
    p.out = out;
    p.w = weights;
    p.position = position;
    p.T = T;
    p.N = N;
    p.R = R;
    p.ldy = ldy;
    p.ldo = ldo;
    p.k = top_k;
    const int unit = std::min(row_unit(y, ldy, esize), row_unit(out, ldo, esize));
    const int per = values_of(unit, esize), threads = cta_threads(N, per, kThreads);
    if (cdiv(N, threads * per) > 65535) return fail(TS_ERR_UNSUPPORTED, "rows of %lld values", static_cast<long long>(N));
    const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(cdiv(N, threads * per))), block(threads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == TS_OUT_F32 ? combine_launch<float>(p, unit, grid, block, st)
                                        : combine_launch<uint16_t>(p, unit, grid, block, st);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "combine launch");
}

ts_status ts_moe_combine_grad(const void *grad_out, const void *y, const int32_t *position, const float *weights,
                              void *grad_y, float *grad_weights, int64_t T, int32_t top_k, int64_t N, int64_t R,
                              int32_t dtype, int64_t ldy, int64_t ldo, int64_t ldg, void *stream) {
    using namespace ts;
    ldy = ldy ? ldy : N;
    ldo = ldo ? ldo : N;
    ldg = ldg ? ldg : N;
    ts_status s = combine_check(T, top_k, N, R, dtype, ldy, ldo, ldg);
    if (s != TS_OK) return s;
    if (T == 0 || top_k == 0) return TS_OK;
    const int esize = dtype == TS_OUT_F32 ? 4 : 2;
    if (!position || (N > 0 && !grad_out) || (R > 0 && N > 0 && (!y || !grad_y)))
        return fail(TS_ERR_INVALID_ARG, "grad_out, y, position or grad_y is NULL");
    if (reinterpret_cast<uintptr_t>(grad_out) % esize || reinterpret_cast<uintptr_t>(y) % esize ||
        reinterpret_cast<uintptr_t>(grad_y) % esize || reinterpret_cast<uintptr_t>(position) % 4 ||
        reinterpret_cast<uintptr_t>(weights) % 4 || reinterpret_cast<uintptr_t>(grad_weights) % 4)
        return fail(TS_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
    if (R > 0 && N > 0) {
        const int64_t gbytes = ((R - 1) * ldg + N) * esize;
        if (ranges_overlap(grad_y, gbytes, grad_out, ((T - 1) * ldo + N) * esize) ||
            ranges_overlap(grad_y, gbytes, y, ((R - 1) * ldy + N) * esize))
            return fail(TS_ERR_INVALID_ARG, "grad_y overlaps grad_out or y");
    }
    CombineParams p = {};
    p.status = device_status_word(&s);
    if (!p.status) return s;
    p.y = y;
    p.grad_out = grad_out;
    p.grad_y = grad_y;
    p.grad_w = grad_weights;
    p.w = weights;
    p.position = position;
    p.T = T;
    p.N = N;
    p.R = R;
    p.ldy = ldy;
    p.ldo = ldo;
    p.ldg = ldg;
    p.k = top_k;
    const int unit =
        std::min({row_unit(y, ldy, esize), row_unit(grad_out, ldo, esize), row_unit(grad_y, ldg, esize)});
    const dim3 grid(static_cast<unsigned>(T)),
        block(cta_threads(std::max<int64_t>(N, 1), values_of(unit, esize), kGradThreads));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == TS_OUT_F32 ? combine_grad_launch<float>(p, unit, grid, block, st)
                                        : combine_grad_launch<uint16_t>(p, unit, grid, block, st);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "combine gradient launch");
}

}  // extern "C"
