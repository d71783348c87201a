// The gradient of a linear layer's activation and bias:
//
//   grad_z = grad_y * act'(preact),   grad_bias[n] = sum_m grad_z[m][n]
//
// One pass over the data.  A cluster takes a strip of columns, 128 bytes of a row, and its CTAs
// share the rows; each thread holds the fp32 sums of its columns, which the CTA adds up through
// shared memory and the cluster's first CTA over the cluster, in a fixed order.  The sums take the
// values before they are rounded to grad_z's type.  Bound by memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "act.cuh"
#include "common.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int kActThreads = 256;
// On an SM: the 64 registers that leaves a thread are 6 too few for bf16 vectors, which spill 24 bytes (17 words
// loaded again in a loop over rows that waits for memory: 5.6 TB/s of 6.8).
constexpr int kActCtas = 4;
constexpr int kActUnroll = 4;      // rows of a thread in flight
constexpr int kMaxActCluster = 8;

struct ActParams {
    const void *gy, *z;
    void *gz;
    float *gb;
    int64_t ldy, ldz, ldg;
    int64_t M, N;
    int32_t act, cluster;
};

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

// V values, one access: as they lie, and unpacked
template <class T, int V>
struct Vec {
    uint4 u;
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V == 1)
            u.x = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t *>(p) : *reinterpret_cast<const uint16_t *>(p);
        else
            u = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
        const uint32_t w = i / 2 == 0 ? u.x : i / 2 == 1 ? u.y : i / 2 == 2 ? u.z : u.w;
        return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
    }
};
template <class T, int V>
__device__ __forceinline__ void store_v(T *p, const float (&f)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 4)
            *p = f[0];
        else
            *p = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(f[0]), 0u));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else
                w[i] = pack_bf16x2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// T: uint16_t (bf16) or float; VEC: rows start on 16-byte boundaries; LANES: threads along a row.
template <class T, bool VEC, int LANES>
__global__ void __launch_bounds__(kActThreads, kActCtas) act_grad_kernel(const __grid_constant__ ActParams p) {
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
    constexpr int STRIP = LANES * V, ROWS = kActThreads / LANES;
    __shared__ __align__(16) float part[ROWS][STRIP];
    grid_dep_wait();
    grid_dep_launch();
    const int rank = static_cast<int>(blockIdx.x) % p.cluster;
    const int64_t strip = blockIdx.x / p.cluster;
    const int tx = threadIdx.x % LANES, ty = threadIdx.x / LANES;
    const int64_t col = strip * STRIP + tx * V;
    const int64_t m0 = p.M * rank / p.cluster, m1 = p.M * (rank + 1) / p.cluster;
    const int count = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(V), p.N - col)));  // columns of this thread
    const T *gy = static_cast<const T *>(p.gy) + col, *z = static_cast<const T *>(p.z) + col;
    T *gz = static_cast<T *>(p.gz) + col;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    auto rows = [&](auto tag) {
        constexpr int A = decltype(tag)::value;
        if (count == V) {
            for (int64_t m = m0 + ty; m < m1; m += kActUnroll * ROWS) {
                Vec<T, V> g[kActUnroll], zz[kActUnroll];
#pragma unroll
                for (int k = 0; k < kActUnroll; ++k) {
                    const int64_t r = m + k * ROWS;
                    if (r < m1) {
                        g[k].load(gy + r * p.ldy);
                        if constexpr (A != ACT_NONE) zz[k].load(z + r * p.ldz);
                    }
                }
#pragma unroll
                for (int k = 0; k < kActUnroll; ++k) {
                    const int64_t r = m + k * ROWS;
                    if (r < m1) {
                        float o[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = g[k].get(i);
                        if constexpr (A != ACT_NONE) {
                            constexpr int W = V > 1 ? 1 : 0;  // a single value goes as a pair of itself
#pragma unroll
                            for (int i = 0; i < V; i += 1 + W) {
                                float other;
                                split(two(o[i], o[i + W]) * act_slope<A>(two(zz[k].get(i), zz[k].get(i + W))), o[i],
                                      W ? o[i + W] : other);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < V; ++i) sum[i] += o[i];
                        if (p.gz) store_v<T, V>(gz + r * p.ldg, o);
                    }
                }
            }
        } else if (count > 0) {  // the last, shorter vector of the rows
            for (int64_t m = m0 + ty; m < m1; m += ROWS) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (i < count) {
                        float g = to_f32(gy[m * p.ldy + i]);
                        if constexpr (A != ACT_NONE) {
                            float other;
                            split(two(g) * act_slope<A>(two(to_f32(z[m * p.ldz + i]))), g, other);
                        }
                        sum[i] += g;
                        if (p.gz) {
                            const float one[1] = {g};
                            store_v<T, 1>(gz + m * p.ldg + i, one);
                        }
                    }
                }
            }
        }
    };
    with_act(p.act, rows);
    if (!p.gb) return;
#pragma unroll
    for (int i = 0; i < V; ++i) part[ty][tx * V + i] = sum[i];
    __syncthreads();
    static_assert(STRIP <= kActThreads, "a thread sums a column");
    float total = 0.f;
    if (threadIdx.x < STRIP) {
        for (int r = 0; r < ROWS; ++r) total += part[r][threadIdx.x];
        part[0][threadIdx.x] = total;  // only this thread reads the column
    }
    if (p.cluster > 1) {
        cluster_sync();
        if (rank == 0 && threadIdx.x < STRIP) {
            const uint32_t at = smem_u32(&part[0][threadIdx.x]);
            for (int c = 1; c < p.cluster; ++c) total += ld_cluster_f32(mapa(at, c));
        }
        cluster_sync();  // no CTA leaves while the first reads its sums
    }
    if (rank == 0 && threadIdx.x < STRIP && strip * STRIP + threadIdx.x < p.N) p.gb[strip * STRIP + threadIdx.x] = total;
}

template <class T, bool VEC, int LANES>
cudaError_t launch_strips(ActParams &p, int64_t sms, cudaStream_t st) {
    constexpr int64_t STRIP = LANES * (VEC ? 16 / sizeof(T) : 1);
    // CTAs that share a strip's rows: while they all run at once, and have 64 rows each or more.  (One where there are
    // many strips: of eight values or more then, so that no grid has more than 2^28 CTAs.)
    const int64_t strips = cdiv(p.N, STRIP);
    p.cluster = static_cast<int32_t>(std::max<int64_t>(1, std::min({int64_t{kMaxActCluster}, p.M / 64, kActCtas * sms / strips})));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(strips * p.cluster), 1, 1);
    cfg.blockDim = dim3(kActThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, act_grad_kernel<T, VEC, LANES>, p);
}

template <class T, bool VEC>
cudaError_t launch_act_grad(ActParams &p, int64_t sms, cudaStream_t st) {
    // Strips of 128 bytes, or of 64 where those would be too few for two CTAs on each SM.  (Rows of 8192
    // columns: 70 us by 4 CTAs a strip, 77 by 8, which take two waves.)
    const int64_t strips = cdiv(p.N, 8 * (VEC ? 16 / sizeof(T) : 1));
    return strips * kMaxActCluster < 2 * sms ? launch_strips<T, VEC, 4>(p, sms, st) : launch_strips<T, VEC, 8>(p, sms, st);
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_act_grad(const void *grad_y, const void *preact, void *grad_z, float *grad_bias, int64_t M,
                                 int64_t N, int32_t dtype, int32_t act, int64_t ldy, int64_t ldp, int64_t ldg,
                                 void *stream) {
    using namespace ts;
    constexpr int64_t kMax = 0x7fffffffLL - 511, kPitch = int64_t(1) << 37;
    if (M < 0 || N < 0 || M > kMax || N > kMax)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^31 - 512] (M=%lld N=%lld)", static_cast<long long>(M),
                    static_cast<long long>(N));
    if (dtype != TS_OUT_BF16 && dtype != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "dtype %d", dtype);
    if (act < 0 || act >= kActs) return fail(TS_ERR_INVALID_ARG, "act %d", act);
    if ((act != TS_ACT_NONE) != (preact != nullptr))
        return fail(TS_ERR_INVALID_ARG, "an activation and its pre-activations are given together");
    if (!grad_z && !grad_bias) return fail(TS_ERR_INVALID_ARG, "neither grad_z nor grad_bias is given");
    ldy = ldy ? ldy : N;
    ldp = ldp ? ldp : N;
    ldg = ldg ? ldg : N;
    if (ldy < N || ldp < N || ldg < N || ldy > kPitch || ldp > kPitch || ldg > kPitch)
        return fail(TS_ERR_INVALID_ARG, "row strides must cover a row (%lld, %lld, %lld)", static_cast<long long>(ldy),
                    static_cast<long long>(ldp), static_cast<long long>(ldg));
    if (N == 0 || (M == 0 && !grad_bias)) return TS_OK;
    if (M > 0 && !grad_y) return fail(TS_ERR_INVALID_ARG, "grad_y is NULL");
    const int esize = dtype == TS_OUT_F32 ? 4 : 2;
    bool vec = true;
    for (const void *q : {grad_y, preact, static_cast<const void *>(grad_z)}) {
        if (reinterpret_cast<uintptr_t>(q) % esize) return fail(TS_ERR_INVALID_ARG, "a matrix is not aligned to its element size");
        vec &= reinterpret_cast<uintptr_t>(q) % 16 == 0;
    }
    if (reinterpret_cast<uintptr_t>(grad_bias) % 4) return fail(TS_ERR_INVALID_ARG, "grad_bias is not aligned to 4 bytes");
    if (M > 1) vec &= (ldy * esize) % 16 == 0 && (!preact || (ldp * esize) % 16 == 0) && (!grad_z || (ldg * esize) % 16 == 0);
    const RowsInMemory y{grad_y, M, N * esize, ldy * esize}, z{preact, M, N * esize, ldp * esize}, g{grad_z, M, N * esize, ldg * esize},
        bias{grad_bias, M > 0 ? 1 : 0, 4 * N, 4 * N};
    // each element of grad_z is written by the thread that has read the others at its place
    auto clash = [&](const RowsInMemory &q) { return rows_overlap(g, q) && !(q.ptr == g.ptr && (q.pitch == g.pitch || M <= 1)); };
    if (clash(y) || clash(z)) return fail(TS_ERR_INVALID_ARG, "grad_z overlaps an input, and is not that input");
    if (rows_overlap(bias, y) || rows_overlap(bias, z) || rows_overlap(bias, g))
        return fail(TS_ERR_INVALID_ARG, "grad_bias overlaps a matrix");
    ActParams p;
    std::memset(&p, 0, sizeof p);
    p.gy = grad_y;
    p.z = preact;
    p.gz = grad_z;
    p.gb = grad_bias;
    p.ldy = ldy;
    p.ldz = ldp;
    p.ldg = ldg;
    p.M = M;
    p.N = N;
    p.act = act;
    const int64_t sms = device_sms(current_device());
    if (sms <= 0) return fail(TS_ERR_CUDA, "cannot query the SM count");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto pick = [&](auto t, auto v) { return launch_act_grad<decltype(t), decltype(v)::value>(p, sms, st); };
    const cudaError_t e = dtype == TS_OUT_F32 ? (vec ? pick(float(), std::true_type()) : pick(float(), std::false_type()))
                                              : (vec ? pick(uint16_t(), std::true_type()) : pick(uint16_t(), std::false_type()));
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "activation gradient launch");
}
