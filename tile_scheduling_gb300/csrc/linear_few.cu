// A linear layer's product for few rows of x (a token, a batch of decoded tokens):
//
//   y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n],   M <= 8
//
// Bound by reading w once: 16 rows of w times 8 columns of tokens are one matrix instruction, and
// what counts is how many bytes of w are in flight.  A CTA takes 16 rows of w, its warps share K; a
// lane loads 16 bytes of two rows for each 32 of K straight into the registers that the instruction
// reads: the sum over k may take its terms in any order, so the eight values of a load serve as the
// operand's columns 2t, 2t + 1, 2t + 8 and 2t + 9 of two instructions.  x is loaded the same way.
// Where N gives too few CTAs, a cluster's CTAs share K as well.  The partial sums are added in a
// fixed order, so results do not depend on timing.
//
// While the CTAs all run at once they ask for the start of their part of w to be brought into L2 before
// they wait for the previous kernel in the stream: a prefetch changes nothing that a later write could
// not, and the data it fetches is read after the wait.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "act.cuh"
#include "common.h"
#include "linear_params.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 16;     // of w a CTA takes
constexpr int kFewBlock = 32;    // of K a warp takes at a time
constexpr int kFewCluster = 8;
// Bytes of a row that are asked for ahead: what the previous kernel's end covers.  More of them compete with the
// loads: one token, 4096 x 28672 39.6 us, 53.7 with whole rows, 40.0 with none; 4096 x 4096 7.4, 7.3 and 8.0.
constexpr int32_t kFewPrefetch = 4096;
constexpr int kFewDeep = 8, kFewShallow = 3;  // blocks in flight with two and with four CTAs on an SM

struct FewParams {
    const uint16_t *x, *w;
    int64_t ldx, ldw;
    int32_t M, N, K, blocks;  // blocks: of K
    int32_t split;            // CTAs of a cluster, which share K
    int32_t prefetch;
    int32_t act, out, bias_f32;
    const void *bias, *aux;
    int64_t ld_aux;
    void *pre, *y;
    int64_t ld_pre, ldy;
};

// bf16 16x16 times 16x8, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight values from k on, zeros from K on (what lies there is not read).
__device__ __forceinline__ uint4 load_k(const uint16_t *row, int32_t k, int32_t K) {
    if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i >> 1] |= uint32_t(__ldg(row + k + i)) << (16 * (i & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// UN: blocks of K a warp has in flight; CTAS: on an SM.
template <int UN, int CTAS>
__global__ void __launch_bounds__(kFewThreads, CTAS) linear_few_kernel(const __grid_constant__ FewParams p) {
    __shared__ __align__(16) float part[kFewWarps][kFewTokens][kFewRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int32_t n0 = static_cast<int32_t>(blockIdx.x) / p.split * kFewRows;
    const int32_t b0 = p.blocks / p.split * rank + min(rank, p.blocks % p.split);
    const int32_t b1 = b0 + p.blocks / p.split + (rank < p.blocks % p.split ? 1 : 0);
    const int32_t end = min(b1 * kFewBlock, p.K);
    if (p.prefetch && threadIdx.x < kFewRows && n0 + static_cast<int>(threadIdx.x) < p.N) {
        const int32_t bytes = min(kFewPrefetch / 2, end - b0 * kFewBlock) * 2 & ~15;
        if (bytes > 0) prefetch_l2(p.w + (n0 + static_cast<int>(threadIdx.x)) * p.ldw + b0 * kFewBlock, bytes);
    }
    grid_dep_wait();
    grid_dep_launch();
    // a row past the last reads the last: its sums are not stored
    const uint16_t *const w0 = p.w + min(n0 + g, p.N - 1) * p.ldw;
    const uint16_t *const w1 = p.w + min(n0 + g + 8, p.N - 1) * p.ldw;
    const uint16_t *const x = p.x + min(g, p.M - 1) * p.ldx;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int32_t b = b0 + warp; b < b1; b += UN * kFewWarps) {
        uint4 a0[UN], a1[UN], xx[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int32_t bu = b + u * kFewWarps;
            a0[u] = a1[u] = xx[u] = make_uint4(0u, 0u, 0u, 0u);
            if (bu < b1) {
                const int32_t k = bu * kFewBlock + 8 * t;
                a0[u] = load_k(w0, k, end);
                a1[u] = load_k(w1, k, end);
                xx[u] = load_k(x, k, end);
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            mma_16816(sum, a0[u].x, a1[u].x, a0[u].y, a1[u].y, xx[u].x, xx[u].y);
            mma_16816(sum, a0[u].z, a1[u].z, a0[u].w, a1[u].w, xx[u].z, xx[u].w);
        }
    }
    // sum: rows g and g + 8 of w, tokens 2 t and 2 t + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = sum[i];
    __syncthreads();
    constexpr int OUTS = kFewTokens * kFewRows;
    const int m = threadIdx.x / kFewRows, r = threadIdx.x % kFewRows;
    float z = 0.f;
    if (threadIdx.x < OUTS) {
#pragma unroll
        for (int q = 0; q < kFewWarps; ++q) z += part[q][m][r];
        part[0][m][r] = z;  // only this thread reads the output's sums
    }
    if (p.split > 1) {
        cluster_sync();
        if (rank == 0 && threadIdx.x < OUTS) {
            const uint32_t at = smem_u32(&part[0][m][r]);
            for (int c = 1; c < p.split; ++c) z += ld_cluster_f32(mapa(at, c));
        }
        cluster_sync();  // no CTA leaves while the first reads its sums
    }
    const int32_t n = n0 + r;
    if (rank != 0 || threadIdx.x >= OUTS || m >= p.M || n >= p.N) return;
    auto value = [&](const void *q, int64_t i, bool f32) {
        return f32 ? static_cast<const float *>(q)[i] : __uint_as_float(uint32_t(static_cast<const uint16_t *>(q)[i]) << 16);
    };
    auto store = [&](void *q, int64_t i, float f) {
        if (p.out == OUT_F32)
            static_cast<float *>(q)[i] = f;
        else
            static_cast<uint16_t *>(q)[i] = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(f), 0u));
    };
    if (p.bias) z += value(p.bias, n, p.bias_f32);
    if (p.pre) store(p.pre, m * p.ld_pre + n, z);
    float one[2] = {z, z};
    with_act(p.act, [&](auto act) { apply_act<decltype(act)::value>(one); });
    float f = one[0];
    if (p.aux) f += value(p.aux, m * p.ld_aux + n, p.out == OUT_F32);
    store(p.y, m * p.ldy + n, f);
}

template <int UN, int CTAS>
cudaError_t launch_few(const FewParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p.N, kFewRows) * p.split), 1, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.split > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<UN, CTAS>, p);
}

}  // namespace

bool linear_few_takes(const LinCall &c) {
    return c.M <= kFewTokens && c.batch == 1 && c.tile == TS_TILE_AUTO &&
           c.max_workers == 0;
}

ts_status linear_few(const LinCall &c) {
    const int64_t sms = device_sms(current_device());
    if (sms <= 0) return fail(TS_ERR_CUDA, "cannot query the SM count");
    FewParams p;
    std::memset(&p, 0, sizeof p);
    p.x = static_cast<const uint16_t *>(c.A);
    p.w = static_cast<const uint16_t *>(c.B);
    p.ldx = c.lda;
    p.ldw = c.ldb;
    p.M = static_cast<int32_t>(c.M);
    p.N = static_cast<int32_t>(c.N);
    p.K = static_cast<int32_t>(c.K);
    p.blocks = static_cast<int32_t>(cdiv(c.K, kFewBlock));
    p.act = c.act;
    p.out = c.out;
    p.bias = c.bias;
    p.bias_f32 = c.bias_f32;
    p.aux = c.aux;
    p.ld_aux = c.ld_aux;
    p.pre = c.pre;
    p.ld_pre = c.ld_pre;
    p.y = c.D;
    p.ldy = c.ldd;
    // Two CTAs on an SM with eight blocks of K in flight for each warp while they all run at once,
    // else four with three.  Measured, one token, 4096 x 4096 (256 CTAs): 7.6 us and 9.6; 8192 x 8192
    // (512 CTAs): 26.4 and 23.6.  A cluster shares K while its CTAs fit as well and a warp has more
    // blocks than it can have in flight.
    const int64_t tiles = cdiv(c.N, kFewRows);
    p.split = 1;
    while (p.split < kFewCluster && 2 * tiles * p.split <= 2 * sms && p.blocks > p.split * kFewDeep * kFewWarps) p.split *= 2;
    const bool deep = tiles * p.split <= 2 * sms;
    p.prefetch = deep;  // prefetches of CTAs that run later compete with the loads of those that run: 8192 x 8192 27.6 us
    const cudaError_t e = deep ? launch_few<kFewDeep, 2>(p, c.stream) : launch_few<kFewShallow, 4>(p, c.stream);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "few-token product launch");
}

}  // namespace ts
