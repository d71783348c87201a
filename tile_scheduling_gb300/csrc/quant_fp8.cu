// Quantisation to 8-bit floating point with one scale for each row and 128
// columns (or, transposed, each column and 128 rows) of a bf16 or fp32 matrix:
//
//   a = max |x| over the block (at least 2^-100),  s = a / top,  q = rne(x * (top / a))
//
// with top = 448 (e4m3) or 57344 (e5m2).  The row form may gather: output row r
// is input row rows[r] / rows_div, which lays tokens out by expert and quantises
// them in one pass.  A not-a-number stays one in q; an infinity gives s = inf and
// q = NaN at that place, so that both come out of a product as NaN.
#include <algorithm>

#include "common.h"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr int kBlk = 128;
constexpr int kQThreads = 256;
constexpr int kRowBlocks = 4;

struct QuantParams {
    const void *x;
    int64_t ldx;
    int64_t M, N;          // input rows and columns
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t s_row, s_blk;  // strides of s along q's rows and along the blocks of a row
    const int32_t *rows;   // gather index or nullptr
    int64_t R;             // output rows
    int32_t rows_div;
    int32_t vec;           // 16-byte loads and 8-byte stores are aligned
    unsigned long long *status;
};

__device__ __forceinline__ float top_of(bool e5m2) { return e5m2 ? 57344.f : 448.f; }

// Four fp32 values to four 8-bit ones, rounded to nearest even; past the largest
// value they saturate, a NaN stays one.
template <bool E5M2>
__device__ __forceinline__ uint32_t pack_f8x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if constexpr (E5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return uint32_t(lo) | (uint32_t(hi) << 16);
}

// The larger of two bf16 values in each half (the number, where one is not a number).  Half
// the instructions of fp32: 16384 x 4096 rows 35.4 -> 32.3 us, 8192 x 8192 transposed 37.9
// -> 34.1 (with eight CTAs on an SM for six).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight values as they lie in memory (a bf16's stay packed: half the registers).
template <class T>
struct Raw8 {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

// x[0 .. 8); n: how many of them exist (the rest read as 0).
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T *x, bool vec, int64_t n) {
    Raw8<T> r;
    if (vec && n >= 8) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x) + i);
            r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2 * static_cast<int>(sizeof(T)); ++i) r.w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    r.w[i] = __float_as_uint(x[i]);
                else
                    r.w[i >> 1] |= uint32_t(x[i]) << (16 * (i & 1));
            }
        }
    }
    return r;
}

// Row form.  Sixteen lanes take one block of one row, eight values each; a CTA
// takes 16 rows and BLOCKS blocks, so a warp reads whole 256-byte (bf16) runs.
// Bound by memory: 16384 x 4096 bf16 32.3 us (6.3 TB/s), fp32 49.7 (6.8).
template <class T, bool E5M2, int BLOCKS>
__global__ void __launch_bounds__(kQThreads) quant_rows_kernel(const __grid_constant__ QuantParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int part = threadIdx.x & 15;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int64_t kb0 = static_cast<int64_t>(blockIdx.y) * BLOCKS;
    const int64_t blocks = (p.N + kBlk - 1) / kBlk;
    int64_t src = r;
    bool there = r < p.R;
    if (there && p.rows) {
        const int32_t at = p.rows[r];
        src = at / p.rows_div;
        if (at < 0) {
            there = false;  // an empty slot: q and s are zero
            src = -1;
        } else if (src >= p.M) {
            if (part == 0 && blockIdx.y == 0) {
                if (atomicCAS(&p.status[0], 0ull, 5ull) == 0ull) atomicExch(&p.status[1], static_cast<unsigned long long>(r));
                atomicAdd(&p.status[2], 1ull);
            }
            there = false;
        }
    }
    const T *const x = static_cast<const T *>(p.x) + (there ? src : 0) * p.ldx;
    Raw8<T> v[BLOCKS];  // every load of this thread is in flight before the first is used
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const int64_t c = (kb0 + i) * kBlk + part * 8;
        v[i] = load8(x + c, p.vec, there ? p.N - c : 0);
    }
    // Every lane has its blocks' maxima; lane i of the sixteen divides for block i (a warp
    // that divides for each block spends half of its instructions on that: 42 us for
    // the 32 above).
    float a[BLOCKS], mine = 1.f;
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        if constexpr (sizeof(T) == 2) {
            uint32_t m = v[i].w[0] & 0x7fff7fffu;
#pragma unroll
            for (int j = 1; j < 4; ++j) m = max_bf16x2(m, v[i].w[j] & 0x7fff7fffu);
            a[i] = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        } else {
            a[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a[i] = fmaxf(a[i], fabsf(v[i][j]));
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], d));
        if (part == i) mine = fmaxf(a[i], 0x1p-100f);
    }
    const float factor = top_of(E5M2) / mine;
    if (r < p.R && part < BLOCKS && kb0 + part < blocks)
        p.s[r * p.s_row + (kb0 + part) * p.s_blk] = there ? mine / top_of(E5M2) : 0.f;
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const int64_t c = (kb0 + i) * kBlk + part * 8;
        const float f = __shfl_sync(0xffffffffu, factor, i, 16);
        const uint32_t lo = pack_f8x4<E5M2>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
        const uint32_t hi = pack_f8x4<E5M2>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f);
        if (r < p.R) {
            uint8_t *const dst = p.q + r * p.ldq + c;
            if (p.vec && c + 8 <= p.N) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < p.N) dst[j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
            }
        }
    }
}

// Transposed form: q[n][m] from x[m][n], blocks of 128 along m.  A CTA takes one
// block of 128 rows by 64 columns; each thread holds four consecutive rows of
// eight columns, so its four values of a column make one 32-bit word of q.  Bound by
// memory: 8192 x 8192 bf16 34.1 us (6.0 TB/s), fp32 55.2 (6.1).
template <class T, bool E5M2>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 8 : 4) quant_trans_kernel(const __grid_constant__ QuantParams p) {
    constexpr int PITCH = kBlk / 4 + 1;  // words of a column's 128 values, padded
    __shared__ float amax[8][64];
    __shared__ float factor[64];
    __shared__ uint32_t tile[64 * PITCH];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;  // column octet, row quad
    const int64_t mb = blockIdx.x;
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * 64;
    const int64_t m0 = mb * kBlk + rg * 4;
    const int64_t n = n0 + cg * 8;
    Raw8<T> v[4];
    float a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = load8(static_cast<const T *>(p.x) + (m0 + i < p.M ? m0 + i : 0) * p.ldx + n, p.vec,
                     m0 + i < p.M ? p.N - n : 0);
    if constexpr (sizeof(T) == 2) {
        // two columns at a time: the largest of bf16 values is one of them
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t m = max_bf16x2(max_bf16x2(v[0].w[j] & 0x7fff7fffu, v[1].w[j] & 0x7fff7fffu),
                                    max_bf16x2(v[2].w[j] & 0x7fff7fffu, v[3].w[j] & 0x7fff7fffu));
            m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 16));
            a[2 * j] = __uint_as_float(m << 16);
            a[2 * j + 1] = __uint_as_float(m & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])), fmaxf(fabsf(v[2][j]), fabsf(v[3][j])));
            a[j] = fmaxf(a[j], __shfl_xor_sync(0xffffffffu, a[j], 8));
            a[j] = fmaxf(a[j], __shfl_xor_sync(0xffffffffu, a[j], 16));
        }
    }
    if (lane < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax[warp][lane * 8 + j] = a[j];
    }
    __syncthreads();
    // one thread a column joins the warps' maxima and divides; every thread doing so for
    // its eight columns took half of the kernel's time
    if (threadIdx.x < 64) {
        float t = 0x1p-100f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t = fmaxf(t, amax[w][threadIdx.x]);
        factor[threadIdx.x] = top_of(E5M2) / t;
        if (n0 + threadIdx.x < p.N) p.s[(n0 + threadIdx.x) * p.s_row + mb * p.s_blk] = t / top_of(E5M2);
    }
    __syncthreads();
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = factor[cg * 8 + j];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        tile[(cg * 8 + j) * PITCH + rg] =
            pack_f8x4<E5M2>(v[0][j] * f[j], v[1][j] * f[j], v[2][j] * f[j], v[3][j] * f[j]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int col = warp + 8 * i;  // each warp stores a column's 128 bytes
        if (n0 + col >= p.N) break;
        const uint32_t w = tile[col * PITCH + lane];
        uint8_t *const dst = p.q + (n0 + col) * p.ldq + mb * kBlk + lane * 4;
        const int64_t left = p.M - (mb * kBlk + lane * 4);
        if (p.ldq % 4 == 0 && reinterpret_cast<uintptr_t>(p.q) % 4 == 0 && left >= 4) {
            *reinterpret_cast<uint32_t *>(dst) = w;
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b < left) dst[b] = static_cast<uint8_t>(w >> (8 * b));
        }
    }
}

template <class T>
cudaError_t quant_launch(const QuantParams &p, bool e5m2, bool transpose, cudaStream_t st) {
    if (transpose) {
        const dim3 grid(static_cast<unsigned>(cdiv(p.M, kBlk)), static_cast<unsigned>(cdiv(p.N, 64)));
        return e5m2 ? launch_pdl(quant_trans_kernel<T, true>, grid, dim3(kQThreads), 0, st, p)
                    : launch_pdl(quant_trans_kernel<T, false>, grid, dim3(kQThreads), 0, st, p);
    }
    // Two / four / eight blocks a CTA: 16384 x 4096 bf16 38.2 / 35.4 / 39.0 us, 256 x 4096
    // gathered 1.95 / 2.01 / 2.60.
    const dim3 grid(static_cast<unsigned>(cdiv(p.R, 16)), static_cast<unsigned>(cdiv(p.N, kRowBlocks * kBlk)));
    return e5m2 ? launch_pdl(quant_rows_kernel<T, true, kRowBlocks>, grid, dim3(kQThreads), 0, st, p)
                : launch_pdl(quant_rows_kernel<T, false, kRowBlocks>, grid, dim3(kQThreads), 0, st, p);
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_quant_fp8(const void *x, void *q, float *scales, int64_t M, int64_t N, int32_t x_type,
                                  int32_t q_type, const ts_quant_opts *opts, void *stream) {
    using namespace ts;
    const ts_quant_opts z = {};
    const ts_quant_opts *o = opts ? opts : &z;
    if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim || o->out_rows < 0 || o->out_rows > kMaxDim)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^31-1] (M=%lld N=%lld out_rows=%lld)",
                    static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(o->out_rows));
    if (x_type != TS_OUT_BF16 && x_type != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "x_type %d", x_type);
    if (q_type != TS_FP8_E4M3 && q_type != TS_FP8_E5M2) return fail(TS_ERR_INVALID_ARG, "q_type %d", q_type);
    if (o->transpose != 0 && o->transpose != 1)
        return fail(TS_ERR_INVALID_ARG, "transpose = %d (0 or 1)", o->transpose);
    if (o->transpose && o->rows) return fail(TS_ERR_UNSUPPORTED, "the transposed form does not gather rows");
    if (o->rows_div < 0) return fail(TS_ERR_INVALID_ARG, "rows_div = %d", o->rows_div);
    const int64_t R = o->rows ? o->out_rows : M;
    const int64_t q_rows = o->transpose ? N : R, q_cols = o->transpose ? M : N;
    QuantParams p = {};
    p.ldx = o->ldx ? o->ldx : N;
    p.ldq = o->ldq ? o->ldq : q_cols;
    if (p.ldx < N || p.ldq < q_cols)
        return fail(TS_ERR_INVALID_ARG, "leading dimensions must cover a row (ldx=%lld ldq=%lld)",
                    static_cast<long long>(p.ldx), static_cast<long long>(p.ldq));
    if (q_rows == 0 || q_cols == 0) return TS_OK;
    const int esize = x_type == TS_OUT_F32 ? 4 : 2;
    if ((!x && M > 0) || !q || !scales) return fail(TS_ERR_INVALID_ARG, "x, q or scales is NULL");
    if (reinterpret_cast<uintptr_t>(x) % esize || reinterpret_cast<uintptr_t>(scales) % 4 ||
        reinterpret_cast<uintptr_t>(o->rows) % 4)
        return fail(TS_ERR_INVALID_ARG, "x, scales or rows is not aligned to its element size");
    const int64_t xbytes = M > 0 ? ((M - 1) * p.ldx + N) * esize : 0;
    if (ranges_overlap(x, xbytes, q, (q_rows - 1) * p.ldq + q_cols))
        return fail(TS_ERR_INVALID_ARG, "q overlaps x");
    // the launch grid's second dimension, columns of x, has at most 65535 CTAs
    if (cdiv(N, o->transpose ? 64 : kRowBlocks * kBlk) > 65535)
        return fail(TS_ERR_UNSUPPORTED, "N = %lld columns are too many for one launch", static_cast<long long>(N));
    ts_status s;
    p.status = device_status_word(&s);
    if (!p.status) return s;
    p.x = x;
    p.M = M;
    p.N = N;
    p.q = static_cast<uint8_t *>(q);
    p.s = scales;
    p.s_row = o->s_row ? o->s_row : 1;
    p.s_blk = o->s_blk ? o->s_blk : q_rows;
    p.rows = o->rows;
    p.R = R;
    p.rows_div = o->rows_div ? o->rows_div : 1;
    const bool x_ok = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (p.ldx * esize) % 16 == 0;
    p.vec = x_ok && (o->transpose || (reinterpret_cast<uintptr_t>(q) % 8 == 0 && p.ldq % 8 == 0));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e5m2 = q_type == TS_FP8_E5M2;
    cudaError_t e = x_type == TS_OUT_F32 ? quant_launch<float>(p, e5m2, o->transpose, st)
                                         : quant_launch<uint16_t>(p, e5m2, o->transpose, st);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "quantisation launch");
}
