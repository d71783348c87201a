// Orthogonalised updates: parameters, and the passes that normalise a matrix, shared by the chain of
// launches and the one-launch form.
#pragma once
#include <cuda_runtime.h>

#include "common.h"
#include "linear_params.h"
#include "ptx.cuh"

namespace ts {

constexpr float kOrthScale = 4096.f;

struct OrthParams {
    const void *G;
    int64_t ldg, g_matrix;
    void *X;              // fp16 times kOrthScale, or bf16 itself (no steps)
    int64_t ldx, x_matrix;
    float *partial;       // [batch][chunks][3]
    int64_t R, C, vecs;   // vecs: vectors of a row
    FastDiv div_vecs;
    int32_t chunks, to_bf16;
    float eps;
};

template <class T, int V>
__device__ __forceinline__ void load_row(const T *p, int count, float (&f)[V]) {
    if (V > 1 && count == V) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i % V] = __uint_as_float(w[i]);
            } else {
                f[2 * i % V] = __uint_as_float(w[i] << 16);
                f[(2 * i + 1) % V] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f[i] = 0.f;
        if (i < count) {
            if constexpr (sizeof(T) == 4)
                f[i] = __ldg(p + i);
            else
                f[i] = __uint_as_float(uint32_t(__ldg(p + i)) << 16);
        }
    }
}

// f(values, row, first column, how many) for the vectors of rows [r0, r1), four of a thread in flight (single
// values: sixteen).
template <int THREADS, class T, int V, class F>
__device__ __forceinline__ void each_vector(const OrthParams &p, const T *g, int64_t r0, int64_t r1, F &&f) {
    constexpr int UN = V > 1 ? 4 : 16;
    const int64_t total = (r1 - r0) * p.vecs;
    for (int64_t i0 = threadIdx.x; i0 < total; i0 += UN * THREADS) {
        float v[UN][V];
        int32_t r[UN], c[UN], count[UN];  // R and C are at most 2^20
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t i = i0 + u * THREADS;
            count[u] = 0;
            if (i < total) {
                // a CTA's share has fewer than 2^31 vectors: see where the host chooses the shares
                const int32_t row = fast_div(static_cast<int32_t>(i), p.div_vecs);
                r[u] = static_cast<int32_t>(r0) + row;
                c[u] = static_cast<int32_t>(i - row * p.vecs) * V;
                count[u] = min(V, static_cast<int32_t>(p.C) - c[u]);
                load_row<T, V>(g + r[u] * p.ldg + c[u], count[u], v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (count[u]) f(v[u], r[u], c[u], count[u]);
    }
}

// The block's sums of three values, in thread 0, in a fixed order.
template <int THREADS, class T>
__device__ __forceinline__ void block_sum3(T &a, T &b, T &c) {
    __shared__ T s[3][THREADS / 32];
    __syncthreads();  // the last sums have been read
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, d);
        b += __shfl_xor_sync(0xffffffffu, b, d);
        c += __shfl_xor_sync(0xffffffffu, c, d);
    }
    if (threadIdx.x % 32 == 0) {
        s[0][threadIdx.x / 32] = a;
        s[1][threadIdx.x / 32] = b;
        s[2][threadIdx.x / 32] = c;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < THREADS / 32; ++w) {
            a += s[0][w];
            b += s[1][w];
            c += s[2][w];
        }
}

// Sums of squares in three ranges, after Blue ("A Portable Fortran Program to Find the Euclidean
// Norm of a Vector", 1978): as they are, and scaled for values whose squares leave fp32's range.
// A matrix has at most 2^40 values (checked on the host).  Scaled by kBigScale = 2^-100 the squares of
// values up to 2^128 sum to at most 2^96.  The third sum is used where the first is below 2^-60, so that
// values are below 2^-30: scaled by kTinyScale = 2^90 their squares sum to less than 2^120, and the
// least fp32 value's square is 2^-118.
constexpr float kBigScale = 0x1p-100f, kTinyScale = 0x1p90f;
// One of p.chunks shares of matrix z, by THREADS threads.
template <class T, bool VEC, int THREADS>
__device__ __forceinline__ void orth_norm(const OrthParams &p, int64_t z, int64_t chunk) {
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
    const T *g = static_cast<const T *>(p.G) + z * p.g_matrix;
    float mid = 0.f, big = 0.f, tiny = 0.f;
    const int64_t r0 = p.R * chunk / p.chunks, r1 = p.R * (chunk + 1) / p.chunks;
    float top = 0.f;
    each_vector<THREADS, T, V>(p, g, r0, r1, [&](const float (&f)[V], int32_t, int32_t, int) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            mid = fmaf(f[k], f[k], mid);
            top = fmaxf(top, fabsf(f[k]));
        }
    });
    // The other two only where this share may matter to them.  The sum of large values is used where the
    // plain sum is infinite, 2^128 or more: shares of values up to 2^30 add less than 2^60 * 2^40 = 2^100 to
    // that, a share of 2^-28, and cannot overflow it.  The sum of tiny ones is used where the plain sum is
    // below 2^-60, and so every share's.
    __shared__ int again;
    block_sum3<THREADS>(mid, big, tiny);
    if (threadIdx.x == 0) again = mid < 0x1p-50f;
    if (__syncthreads_or(top > 0x1p30f) || again) {
        float none = 0.f;
        each_vector<THREADS, T, V>(p, g, r0, r1, [&](const float (&f)[V], int32_t, int32_t, int) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float b = f[k] * kBigScale, t = f[k] * kTinyScale;
                big = fmaf(b, b, big);
                tiny = fmaf(t, t, tiny);
            }
        });
        block_sum3<THREADS>(none, big, tiny);
    }
    if (threadIdx.x == 0) {
        float *const q = p.partial + (z * p.chunks + chunk) * 3;
        __stcg(q, mid);
        __stcg(q + 1, big);
        __stcg(q + 2, tiny);
    }
}

// X = G / (|G|_F + eps), a share of matrix z
template <class T, bool VEC, int THREADS>
__device__ __forceinline__ void orth_scale(const OrthParams &p, int64_t z, int64_t chunk) {
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
    __shared__ float factors[2];
    {
        float mid = 0.f, big = 0.f, tiny = 0.f;
        const float *q = p.partial + z * p.chunks * 3;
        for (int c = threadIdx.x; c < p.chunks; c += THREADS) {
            mid += __ldcg(q + 3 * c);
            big += __ldcg(q + 3 * c + 1);
            tiny += __ldcg(q + 3 * c + 2);
        }
        block_sum3<THREADS>(mid, big, tiny);
        if (threadIdx.x == 0) {
            // The plain sum where it neither overflowed (then it is infinite) nor lost what is below 2^-75
            // (then it is small); a NaN stays one.  x = g * first * second; one of them is a power of two that
            // brings g, the norm and eps into fp32's range.
            const float scale = p.to_bf16 ? 1.f : kOrthScale;
            float first = 1.f, second;
            if (isinf(mid)) {
                first = scale / (sqrtf(big) + p.eps * kBigScale);
                second = kBigScale;
            } else if (mid < 0x1p-60f) {
                const float norm = sqrtf(tiny), sum = norm / kTinyScale + p.eps;
                if (sum < 0x1p-100f) first = kTinyScale;  // whose reciprocal might overflow
                second = scale / (sum < 0x1p-100f ? norm + p.eps * kTinyScale : sum);
            } else {
                second = scale / (sqrtf(mid) + p.eps);
            }
            factors[0] = first;
            factors[1] = second;
        }
        __syncthreads();
    }
    const float first = factors[0], second = factors[1];
    const T *g = static_cast<const T *>(p.G) + z * p.g_matrix;
    uint16_t *x = static_cast<uint16_t *>(p.X) + z * p.x_matrix;
    const bool whole = (p.ldx % V) == 0 && (p.x_matrix % V) == 0 && reinterpret_cast<uintptr_t>(p.X) % (2 * V) == 0;
    const int64_t r0 = p.R * chunk / p.chunks, r1 = p.R * (chunk + 1) / p.chunks;
    each_vector<THREADS, T, V>(p, g, r0, r1, [&](const float (&f)[V], int32_t r, int32_t c, int count) {
        uint16_t o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float v = f[k] * first * second;
            o[k] = p.to_bf16 ? static_cast<uint16_t>(pack_bf16x2(__float_as_uint(v), 0u))
                             : static_cast<uint16_t>(pack_f16x2(__float_as_uint(v), 0u));
        }
        uint16_t *const at = x + r * p.ldx + c;
        if (V > 1 && whole && count == V) {
            uint32_t w[(V + 1) / 2];
#pragma unroll
            for (int k = 0; k < V / 2; ++k) w[k] = o[2 * k] | (uint32_t(o[2 * k + 1]) << 16);
            if constexpr (V == 8)
                *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < count) at[k] = o[k];
        }
    });
}

// What both forms run on: the iteration's matrices in the workspace and its coefficients.
struct OrthRun {
    OrthParams prep;
    bool f32, vec;            // type of G, and whether its rows start on 16-byte boundaries
    int64_t batch, R, C, n;   // n: the shorter side
    int32_t steps;
    float a, b, c;
    uint16_t *X[2], *A, *B;   // fp16 times kOrthScale: [batch][R][ldx], [batch][ldn][ldn]
    int64_t ldx, ldn;
    void *O;                  // bf16
    int64_t ldo, o_matrix;
    int32_t *barrier;         // the one-launch form's counter of arrivals
    double timeout_s;
    cudaStream_t stream;
};
// The one-launch form: its tiles (128 rows by bn columns; of a symmetric product and of X), and the launch.
struct OrthTiles {
    int bn;
    int64_t sym, x;
};
OrthTiles orth_one_tiles(const OrthRun &r, int64_t sms);
ts_status orth_one(const OrthRun &r);

}  // namespace ts
