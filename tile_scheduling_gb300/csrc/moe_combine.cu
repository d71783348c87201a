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

// A thread's values of a row as they lie in memory.  VEC (the rows start on 16-byte
// boundaries): the 16 bytes from column c on, in one load.  Else four values 32 columns
// apart, so that a warp's loads and stores of one value each still fill whole sectors
// (8192 tokens, eight slots, 4095 bf16 values: 169 us and 290 for the gradient; with eight
// neighbours a thread 278 and 727; rows of 4096, VEC, 107 and 187).
template <class T, bool VEC>
struct Vals {
    static constexpr int COUNT = VEC ? 16 / sizeof(T) : 4;
    uint32_t w[4];

    // a thread's first column among those of its CTA
    static __device__ __forceinline__ int64_t first(int thread) {
        return VEC ? int64_t(thread) * COUNT : int64_t(thread & ~31) * COUNT + (thread & 31);
    }
    // those of row x from column c on; the ones past the N-th read as 0
    __device__ __forceinline__ void load(const T *x, int64_t c, int64_t N) {
        if constexpr (VEC) {
            if (c + COUNT <= N) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(x + c));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                return;
            }
            w[0] = w[1] = w[2] = w[3] = 0u;
#pragma unroll
            for (int i = 0; i < COUNT; ++i)
                if (c + i < N) {
                    if constexpr (sizeof(T) == 4)
                        w[i] = __float_as_uint(x[c + i]);
                    else
                        w[i >> 1] |= uint32_t(x[c + i]) << (16 * (i & 1));
                }
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const T v = c + 32 * i < N ? x[c + 32 * i] : T(0);
                if constexpr (sizeof(T) == 4)
                    w[i] = __float_as_uint(v);
                else
                    w[i] = v;
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        if constexpr (!VEC) return __uint_as_float(w[i] << 16);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    static __device__ __forceinline__ void store(T *x, int64_t c, int64_t N, const float (&v)[COUNT]) {
        if constexpr (VEC) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4)
                    o[i] = __float_as_uint(v[i]);
                else
                    o[i] = pack_bf16x2(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
            }
            if (c + COUNT <= N) {
                __stcs(reinterpret_cast<uint4 *>(x + c), make_uint4(o[0], o[1], o[2], o[3]));
                return;
            }
#pragma unroll
            for (int i = 0; i < COUNT; ++i)
                if (c + i < N) {
                    if constexpr (sizeof(T) == 4)
                        x[c + i] = v[i];
                    else
                        x[c + i] = static_cast<T>(o[i >> 1] >> (16 * (i & 1)));
                }
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i)
                if (c + 32 * i < N) {
                    if constexpr (sizeof(T) == 4)
                        x[c + 32 * i] = v[i];
                    else
                        x[c + 32 * i] = static_cast<T>(pack_bf16x2(__float_as_uint(v[i]), 0u));
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
template <class T, int KS, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p) {
    using Row = Vals<T, VEC>;
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
template <class T, bool VEC>
__global__ void __launch_bounds__(kGradThreads, 2) combine_grad_kernel(const __grid_constant__ CombineParams p) {
    using Row = Vals<T, VEC>;
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

bool row16(const void *x, int64_t ld, int esize) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ld * esize) % 16 == 0;
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
    const bool vec = row16(y, ldy, esize) && row16(out, ldo, esize);
    const int per = vec ? 16 / esize : 4, threads = cta_threads(N, per, kThreads);
    if (cdiv(N, threads * per) > 65535) return fail(TS_ERR_UNSUPPORTED, "rows of %lld values", static_cast<long long>(N));
    const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(cdiv(N, threads * per))), block(threads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto *k4, auto *k8) { return launch_pdl(top_k <= 4 ? k4 : k8, grid, block, 0, st, p); };
    cudaError_t e = dtype == TS_OUT_F32
                        ? (vec ? go(combine_kernel<float, 4, true>, combine_kernel<float, 8, true>)
                               : go(combine_kernel<float, 4, false>, combine_kernel<float, 8, false>))
                        : (vec ? go(combine_kernel<uint16_t, 4, true>, combine_kernel<uint16_t, 8, true>)
                               : go(combine_kernel<uint16_t, 4, false>, combine_kernel<uint16_t, 8, false>));
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
    const bool vec = row16(y, ldy, esize) && row16(grad_out, ldo, esize) && row16(grad_y, ldg, esize);
    const dim3 grid(static_cast<unsigned>(T)),
        block(cta_threads(std::max<int64_t>(N, 1), vec ? 16 / esize : 4, kGradThreads));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto *kernel) { return launch_pdl(kernel, grid, block, 0, st, p); };
    cudaError_t e = dtype == TS_OUT_F32
                        ? (vec ? go(combine_grad_kernel<float, true>) : go(combine_grad_kernel<float, false>))
                        : (vec ? go(combine_grad_kernel<uint16_t, true>) : go(combine_grad_kernel<uint16_t, false>));
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "combine gradient launch");
}

}  // extern "C"
