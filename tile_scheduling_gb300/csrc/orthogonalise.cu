// Orthogonalised updates by Newton-Schulz products:
//
//   X = G / (|G|_F + eps);   steps times:  A = X X^T,  X = a X + (b A + c A^2) X
//
// (with X^T X and X on the left where G has more rows than columns: the short side's n x n matrix
// either way).  Each step applies p(s) = a s + b s^3 + c s^5 to the singular values of X.
//
// The products run on the tensor cores with fp16 operands: every value is bounded (singular values
// stay below 1.3 for the usual coefficients), so fp16's range is enough and its 11 bits round eight
// times finer than bf16 at the same rate.  X, A and b A + c A^2 are held as 4096 times their value,
// which keeps entries as small as 2^-26 normal: an entry of a normalised 4096 x 4096 matrix is
// about 2^-12.  Simulated against 64 bits on 64^2 to 2048^2 matrices, the result is off by 2e-3 of
// its norm, 1.7e-3 of which is the rounding to bf16; with bf16 operands it is 1e-2.
//
// A and b A + c A^2 are symmetric: half of their tiles are computed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.h"
#include "linear_params.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr float kOrthScale = 4096.f;
constexpr int kOrthThreads = 256;
constexpr int64_t kOrthChunks = 608;  // CTAs that share a matrix, at most: four for each SM

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

// f(values, row, first column, how many) for the vectors of rows [r0, r1), four of a thread in flight.
template <class T, int V, class F>
__device__ __forceinline__ void each_vector(const OrthParams &p, const T *g, int64_t r0, int64_t r1, F &&f) {
    constexpr int UN = 4;
    const int64_t total = (r1 - r0) * p.vecs;
    for (int64_t i0 = threadIdx.x; i0 < total; i0 += UN * kOrthThreads) {
        float v[UN][V];
        int64_t r[UN], c[UN];
        int count[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t i = i0 + u * kOrthThreads;
            count[u] = 0;
            if (i < total) {
                // a CTA's share has fewer than 2^31 vectors (checked on the host)
                const int32_t row = fast_div(static_cast<int32_t>(i), p.div_vecs);
                r[u] = r0 + row;
                c[u] = (i - row * p.vecs) * V;
                count[u] = static_cast<int>(min(static_cast<int64_t>(V), p.C - c[u]));
                load_row<T, V>(g + r[u] * p.ldg + c[u], count[u], v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (count[u]) f(v[u], r[u], c[u], count[u]);
    }
}

// The block's sums of three values, in thread 0, in a fixed order.
template <class T>
__device__ __forceinline__ void block_sum3(T &a, T &b, T &c) {
    __shared__ T s[3][kOrthThreads / 32];
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
        for (int w = 1; w < kOrthThreads / 32; ++w) {
            a += s[0][w];
            b += s[1][w];
            c += s[2][w];
        }
}

// Sums of squares in three ranges, after Blue ("A Portable Fortran Program to Find the Euclidean
// Norm of a Vector", 1978): as they are, and scaled by 2^-70 and 2^70 for values whose squares
// leave fp32's range.
template <class T, bool VEC>
__global__ void __launch_bounds__(kOrthThreads) orth_norm_kernel(const __grid_constant__ OrthParams p) {
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
    grid_dep_wait();
    grid_dep_launch();
    const T *g = static_cast<const T *>(p.G) + blockIdx.y * p.g_matrix;
    float mid = 0.f, big = 0.f, tiny = 0.f;
    const int64_t r0 = p.R * blockIdx.x / p.chunks, r1 = p.R * (blockIdx.x + 1) / p.chunks;
    each_vector<T, V>(p, g, r0, r1, [&](const float (&f)[V], int64_t, int64_t, int) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float b = f[k] * 0x1p-70f, t = f[k] * 0x1p70f;
            mid = fmaf(f[k], f[k], mid);
            big = fmaf(b, b, big);
            tiny = fmaf(t, t, tiny);
        }
    });
    block_sum3(mid, big, tiny);
    if (threadIdx.x == 0) {
        float *const q = p.partial + (static_cast<int64_t>(blockIdx.y) * p.chunks + blockIdx.x) * 3;
        q[0] = mid;
        q[1] = big;
        q[2] = tiny;
    }
}

// X = G / (|G|_F + eps)
template <class T, bool VEC>
__global__ void __launch_bounds__(kOrthThreads) orth_scale_kernel(const __grid_constant__ OrthParams p) {
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
    grid_dep_wait();
    grid_dep_launch();
    __shared__ double sums[3];
    {
        double mid = 0.0, big = 0.0, tiny = 0.0;
        const float *q = p.partial + static_cast<int64_t>(blockIdx.y) * p.chunks * 3;
        for (int c = threadIdx.x; c < p.chunks; c += kOrthThreads) {
            mid += static_cast<double>(q[3 * c]);
            big += static_cast<double>(q[3 * c + 1]);
            tiny += static_cast<double>(q[3 * c + 2]);
        }
        block_sum3(mid, big, tiny);
        if (threadIdx.x == 0) {
            sums[0] = mid;
            sums[1] = big;
            sums[2] = tiny;
        }
        __syncthreads();
    }
    // the middle sum where it neither overflowed (then it is infinite) nor lost what is below
    // 2^-75 (then it is small); a NaN stays one
    double sq = sums[0];
    if (sums[1] >= 0x1p-20)
        sq = sums[1] * 0x1p140;
    else if (sums[0] < 0x1p-60)
        sq = sums[2] * 0x1p-140;
    // a power of two apart, so that neither the norm's reciprocal nor the product leaves fp32's range
    const double inv = 1.0 / (sqrt(sq) + static_cast<double>(p.eps));
    int e;
    const float f0 = static_cast<float>(frexp(inv, &e));
    const int e1 = isfinite(inv) ? e / 2 : 0, e2 = isfinite(inv) ? e - e1 : 0;
    const float s1 = f0 * (p.to_bf16 ? 1.f : kOrthScale) * exp2f(static_cast<float>(e1)), s2 = exp2f(static_cast<float>(e2));
    const T *g = static_cast<const T *>(p.G) + blockIdx.y * p.g_matrix;
    uint16_t *x = static_cast<uint16_t *>(p.X) + blockIdx.y * p.x_matrix;
    const bool whole = (p.ldx % V) == 0 && (p.x_matrix % V) == 0 && reinterpret_cast<uintptr_t>(p.X) % (2 * V) == 0;
    const int64_t r0 = p.R * blockIdx.x / gridDim.x, r1 = p.R * (blockIdx.x + 1) / gridDim.x;
    each_vector<T, V>(p, g, r0, r1, [&](const float (&f)[V], int64_t r, int64_t c, int count) {
        uint16_t o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float v = f[k] * s2 * s1;
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

// Where the iteration's matrices lie in the workspace, in bytes.
struct OrthPlan {
    int64_t ldx, ldn, n, x_bytes, n_bytes, partial_bytes, chunks;
    int64_t x(int i) const { return i * x_bytes; }
    int64_t a() const { return 2 * x_bytes; }
    int64_t b() const { return 2 * x_bytes + n_bytes; }
    int64_t partial() const { return 2 * x_bytes + 2 * n_bytes; }
    int64_t total() const { return partial() + partial_bytes; }
};

OrthPlan plan_orth(int64_t batch, int64_t R, int64_t C, int steps) {
    OrthPlan o;
    auto round = [](int64_t v) { return cdiv(v, 256) * 256; };
    o.n = std::min(R, C);
    o.ldx = cdiv(C, 8) * 8;
    o.ldn = cdiv(o.n, 8) * 8;
    o.x_bytes = steps > 0 ? round(batch * R * o.ldx * 2) : 0;
    o.n_bytes = steps > 0 ? round(batch * o.n * o.ldn * 2) : 0;
    o.chunks = std::max<int64_t>(1, std::min<int64_t>({kOrthChunks, R, cdiv(R * C, 8192)}));
    o.partial_bytes = round(batch * o.chunks * 3 * 4);
    return o;
}

constexpr int64_t kMaxSide = 1 << 20, kMaxBatch = 65535;

}  // namespace
}  // namespace ts

extern "C" {

int64_t ts_orthogonalise_workspace(int64_t batch, int64_t R, int64_t C, int32_t steps) {
    using namespace ts;
    if (batch <= 0 || R <= 0 || C <= 0 || steps < 0 || batch > kMaxBatch || R > kMaxSide || C > kMaxSide ||
        batch * R > (int64_t(1) << 40) / C)
        return 0;
    return plan_orth(batch, R, C, steps).total();
}

ts_status ts_orthogonalise(const void *G, void *O, int64_t batch, int64_t R, int64_t C, int32_t g_type,
                           const ts_orth_opts *opts, void *workspace, int64_t workspace_bytes, void *stream) {
    using namespace ts;
    ts_orth_opts z;
    std::memset(&z, 0, sizeof z);
    const ts_orth_opts *o = opts ? opts : &z;
    if (batch < 0 || R < 0 || C < 0 || R > kMaxSide || C > kMaxSide)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^20] (batch=%lld R=%lld C=%lld)",
                    static_cast<long long>(batch), static_cast<long long>(R), static_cast<long long>(C));
    if (batch > kMaxBatch)
        return fail(TS_ERR_UNSUPPORTED, "%lld matrices exceed the limit of %lld", static_cast<long long>(batch),
                    static_cast<long long>(kMaxBatch));
    if (C > 0 && batch * R > (int64_t(1) << 40) / C) return fail(TS_ERR_UNSUPPORTED, "too many elements");
    if (g_type != TS_OUT_BF16 && g_type != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "g_type %d", g_type);
    const int32_t steps = o->steps == 0 ? 5 : o->steps < 0 ? 0 : o->steps;
    if (steps > 64) return fail(TS_ERR_INVALID_ARG, "steps = %d (at most 64)", steps);
    if (!(o->eps >= 0.f) || std::isinf(o->eps)) return fail(TS_ERR_INVALID_ARG, "eps must be a finite number, not negative");
    if (!std::isfinite(o->a) || !std::isfinite(o->b) || !std::isfinite(o->c))
        return fail(TS_ERR_INVALID_ARG, "coefficients must be finite");
    if (!(o->timeout_s >= 0)) return fail(TS_ERR_INVALID_ARG, "negative option");
    const bool given = o->a != 0.f || o->b != 0.f || o->c != 0.f;
    const float a = given ? o->a : 3.4445f, b = given ? o->b : -4.7750f, cc = given ? o->c : 2.0315f;
    const int64_t ldg = o->ldg ? o->ldg : C, ldo = o->ldo ? o->ldo : C, pitch = int64_t(1) << 30;
    if (ldg < C || ldo < C || ldg > pitch || ldo > pitch)
        return fail(TS_ERR_INVALID_ARG, "row strides must cover a row (ldg=%lld ldo=%lld)", static_cast<long long>(ldg),
                    static_cast<long long>(ldo));
    const int64_t g_matrix = o->g_matrix ? o->g_matrix : R * ldg, o_matrix = o->o_matrix ? o->o_matrix : R * ldo;
    if (batch > 1 && (g_matrix < (R - 1) * ldg + C || o_matrix < (R - 1) * ldo + C || g_matrix > (int64_t(1) << 37) ||
                      o_matrix > (int64_t(1) << 37)))
        return fail(TS_ERR_INVALID_ARG, "matrices overlap or are too far apart (g_matrix=%lld o_matrix=%lld)",
                    static_cast<long long>(g_matrix), static_cast<long long>(o_matrix));
    if (batch == 0 || R == 0 || C == 0) return TS_OK;
    if (!G || !O) return fail(TS_ERR_INVALID_ARG, "G or O is NULL");
    const int gsize = g_type == TS_OUT_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(G) % gsize || reinterpret_cast<uintptr_t>(O) % 2)
        return fail(TS_ERR_INVALID_ARG, "G or O is not aligned to its element size");
    const int64_t gbytes = ((batch - 1) * g_matrix + (R - 1) * ldg + C) * gsize, obytes = ((batch - 1) * o_matrix + (R - 1) * ldo + C) * 2;
    const OrthPlan plan = plan_orth(batch, R, C, steps);
    if (!workspace || workspace_bytes < plan.total())
        return fail(TS_ERR_INVALID_ARG, "the workspace must hold %lld bytes", static_cast<long long>(plan.total()));
    if (reinterpret_cast<uintptr_t>(workspace) % 256)
        return fail(TS_ERR_INVALID_ARG, "the workspace must start on a 256-byte boundary");
    if (ranges_overlap(G, gbytes, O, obytes)) return fail(TS_ERR_INVALID_ARG, "O overlaps G");
    if (ranges_overlap(workspace, plan.total(), G, gbytes) || ranges_overlap(workspace, plan.total(), O, obytes))
        return fail(TS_ERR_INVALID_ARG, "the workspace overlaps G or O");

    char *const ws = static_cast<char *>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool vec = reinterpret_cast<uintptr_t>(G) % 16 == 0 && (R <= 1 || (ldg * gsize) % 16 == 0) &&
                     (batch <= 1 || (g_matrix * gsize) % 16 == 0);
    const int V = vec ? 16 / gsize : 1;
    OrthParams p;
    std::memset(&p, 0, sizeof p);
    p.G = G;
    p.ldg = ldg;
    p.g_matrix = g_matrix;
    p.X = steps > 0 ? ws : static_cast<char *>(O);
    p.ldx = steps > 0 ? plan.ldx : ldo;
    p.x_matrix = steps > 0 ? R * plan.ldx : o_matrix;
    p.partial = reinterpret_cast<float *>(ws + plan.partial());
    p.R = R;
    p.C = C;
    p.vecs = cdiv(C, V);
    p.div_vecs = fast_div_for(p.vecs);
    p.chunks = static_cast<int32_t>(plan.chunks);
    p.to_bf16 = steps == 0;
    p.eps = o->eps > 0.f ? o->eps : 1e-7f;
    const dim3 norm_grid(static_cast<unsigned>(plan.chunks), static_cast<unsigned>(batch));
    const dim3 block(kOrthThreads);
    cudaError_t e;
    auto prepare = [&](auto norm, auto scale) {
        e = launch_pdl(norm, norm_grid, block, 0, st, p);
        if (e == cudaSuccess) e = launch_pdl(scale, norm_grid, block, 0, st, p);
    };
    if (gsize == 4)
        vec ? prepare(orth_norm_kernel<float, true>, orth_scale_kernel<float, true>)
            : prepare(orth_norm_kernel<float, false>, orth_scale_kernel<float, false>);
    else
        vec ? prepare(orth_norm_kernel<uint16_t, true>, orth_scale_kernel<uint16_t, true>)
            : prepare(orth_norm_kernel<uint16_t, false>, orth_scale_kernel<uint16_t, false>);
    if (e != cudaSuccess) return cuda_fail(e, "normalisation launch");

    const bool tall = R > C;
    const int64_t n = plan.n, x_matrix = R * plan.ldx, n_matrix = n * plan.ldn;
    void *const A = ws + plan.a(), *const B = ws + plan.b();
    LinCall base;
    std::memset(&base, 0, sizeof base);
    base.f16 = 1;
    base.out = base.aux_type = OUT_F16;
    base.batch = batch;
    base.timeout_s = o->timeout_s;
    base.stream = st;
    for (int32_t i = 0; i < steps; ++i) {
        const void *X = ws + plan.x(i & 1);
        const bool last = i + 1 == steps;
        // A = X X^T: 4096 A from the product of 4096 X with itself
        LinCall c = base;
        c.A = c.B = X;
        c.lda = c.ldb = plan.ldx;
        c.a_matrix = c.b_matrix = x_matrix;
        c.a_mn = c.b_mn = tall;
        c.D = A;
        c.ldd = plan.ldn;
        c.d_matrix = n_matrix;
        c.M = c.N = n;
        c.K = tall ? R : C;
        c.sym = 1;
        c.alpha = 1.f / kOrthScale;
        ts_status s = linear_product(c);
        if (s != TS_OK) return s;
        // B = b A + c A^2
        c = base;
        c.A = c.B = c.aux = A;
        c.lda = c.ldb = c.ld_aux = plan.ldn;
        c.a_matrix = c.b_matrix = c.aux_matrix = n_matrix;
        c.D = B;
        c.ldd = plan.ldn;
        c.d_matrix = n_matrix;
        c.M = c.N = c.K = n;
        c.sym = 1;
        c.alpha = cc / kOrthScale;
        c.beta = b;
        s = linear_product(c);
        if (s != TS_OK) return s;
        // X = a X + B X, or a X + X B
        c = base;
        c.A = tall ? X : B;
        c.lda = tall ? plan.ldx : plan.ldn;
        c.a_matrix = tall ? x_matrix : n_matrix;
        c.B = tall ? B : X;
        c.ldb = tall ? plan.ldn : plan.ldx;
        c.b_matrix = tall ? n_matrix : x_matrix;
        c.b_mn = !tall;
        c.aux = X;
        c.ld_aux = plan.ldx;
        c.aux_matrix = x_matrix;
        c.D = last ? O : ws + plan.x((i + 1) & 1);
        c.ldd = last ? ldo : plan.ldx;
        c.d_matrix = last ? o_matrix : x_matrix;
        c.M = R;
        c.N = C;
        c.K = n;
        c.out = last ? OUT_BF16 : OUT_F16;
        c.alpha = last ? 1.f / (kOrthScale * kOrthScale) : 1.f / kOrthScale;
        c.beta = last ? a / kOrthScale : a;
        s = linear_product(c);
        if (s != TS_OK) return s;
    }
    return TS_OK;
}

}  // extern "C"
