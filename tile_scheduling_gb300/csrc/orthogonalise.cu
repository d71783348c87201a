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
#include "orth.cuh"
#include "ptx.cuh"

namespace ts {
namespace {

constexpr int kOrthThreads = 256;
constexpr int64_t kOrthChunks = 1216;  // CTAs that share the matrices, about: eight for each SM
constexpr int64_t kOrthShare = 1024;   // vectors (or single values) of a CTA, while there are more of them

template <class T, bool VEC>
__global__ void __launch_bounds__(kOrthThreads) orth_norm_kernel(const __grid_constant__ OrthParams p) {
    grid_dep_wait();
    grid_dep_launch();
    orth_norm<T, VEC, kOrthThreads>(p, blockIdx.y, blockIdx.x);
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kOrthThreads) orth_scale_kernel(const __grid_constant__ OrthParams p) {
    grid_dep_wait();
    grid_dep_launch();
    orth_scale<T, VEC, kOrthThreads>(p, blockIdx.y, blockIdx.x);
}

// Where the iteration's matrices lie in the workspace, in bytes.
struct OrthPlan {
    int64_t ldx, ldn, n, x_bytes, n_bytes, partial_bytes, chunks;
    int64_t x(int i) const { return i * x_bytes; }
    int64_t a() const { return 2 * x_bytes; }
    int64_t b() const { return 2 * x_bytes + n_bytes; }
    int64_t partial() const { return 2 * x_bytes + 2 * n_bytes; }
    int64_t barrier() const { return partial() + partial_bytes; }
    int64_t total() const { return barrier() + 256; }
};

OrthPlan plan_orth(int64_t batch, int64_t R, int64_t C, int steps) {
    OrthPlan o;
    auto round = [](int64_t v) { return cdiv(v, 256) * 256; };
    o.n = std::min(R, C);
    // rows on 128-byte boundaries: a box of the products' loads then touches each line once (2300 x 1024
    // x 1001 8.0 us, with rows of 2016 bytes 8.8)
    o.ldx = cdiv(C, 64) * 64;
    o.ldn = cdiv(o.n, 64) * 64;
    o.x_bytes = steps > 0 ? round(batch * R * o.ldx * 2) : 0;
    o.n_bytes = steps > 0 ? round(batch * o.ldn * o.ldn * 2) : 0;
    // A share has fewer than 2^31 values, which the kernels count on: a batch has at most 2^40, so that with 1216
    // CTAs for one matrix a share has 2^40 / 1216, a whole matrix among more than 1216 fewer, and fewer CTAs
    // than that have a row of up to 2^20 each or a share of some 1024.
    o.chunks = std::max<int64_t>(1, std::min<int64_t>({cdiv(kOrthChunks, batch), R, cdiv(R * C, kOrthShare)}));
    o.partial_bytes = round(batch * o.chunks * 3 * 4);
    return o;
}

// Product `which` of step i, of matrices that are 4096 times their value.  What they leave in the
// workspace has a multiple of eight columns (and the symmetric ones as many rows), so that it is
// written in whole vectors; the columns beyond the matrix hold zeros or are never read.
LinCall orth_product(const OrthRun &r, int32_t i, int which) {
    const bool tall = r.R > r.C, last = i + 1 == r.steps;
    const int64_t x_matrix = r.R * r.ldx, n_matrix = r.ldn * r.ldn, n8 = cdiv(r.n, 8) * 8;
    const void *X = r.X[i & 1];
    LinCall c;
    std::memset(&c, 0, sizeof c);
    c.f16 = 1;
    c.out = OUT_F16;
    c.batch = r.batch;
    c.timeout_s = r.timeout_s;
    c.stream = r.stream;
    if (which < 2) {
        c.sym = 1;
        c.M = c.N = n8;
        c.a_rows = c.b_rows = r.n;
        c.ldd = r.ldn;
        c.d_matrix = n_matrix;
    }
    if (which == 0) {  // A = X X^T
        c.A = c.B = X;
        c.lda = c.ldb = r.ldx;
        c.a_matrix = c.b_matrix = x_matrix;
        c.a_mn = c.b_mn = tall;
        c.D = r.A;
        c.K = tall ? r.R : r.C;
        c.alpha = 1.f / kOrthScale;
    } else if (which == 1) {  // B = b A + c A^2
        c.A = c.B = c.aux = r.A;
        c.lda = c.ldb = c.ld_aux = r.ldn;
        c.a_matrix = c.b_matrix = c.aux_matrix = n_matrix;
        c.D = r.B;
        c.K = r.n;
        c.alpha = r.c / kOrthScale;
        c.beta = r.b;
    } else {  // X = a X + B X, or a X + X B
        c.A = tall ? X : r.B;
        c.lda = tall ? r.ldx : r.ldn;
        c.a_matrix = tall ? x_matrix : n_matrix;
        c.B = tall ? r.B : X;
        c.ldb = tall ? r.ldn : r.ldx;
        c.b_matrix = tall ? n_matrix : x_matrix;
        c.b_mn = !tall;
        c.aux = X;
        c.ld_aux = r.ldx;
        c.aux_matrix = x_matrix;
        c.D = last ? r.O : r.X[(i + 1) & 1];
        c.ldd = last ? r.ldo : r.ldx;
        c.d_matrix = last ? r.o_matrix : x_matrix;
        c.M = r.R;
        c.N = last ? r.C : cdiv(r.C, 8) * 8;
        c.b_rows = r.C;
        c.K = r.n;
        c.out = last ? OUT_BF16 : OUT_F16;
        c.alpha = last ? 1.f / (kOrthScale * kOrthScale) : 1.f / kOrthScale;
        c.beta = last ? r.a / kOrthScale : r.a;
    }
    return c;
}

// One launch where it takes fewer cycles than the chain, by the chain's estimates and this one of a step:
// a phase some 3 us (the barrier, the first loads, the stores), a K block of a tile 360 cycles with 64
// columns and 600 with 128.  Measured, a bf16 matrix in a graph, one launch / chain: 128 x 128 61 / 76 us,
// 512 x 768 85 / 90, 1024 x 1024 101 / 112, two of 700 x 700 100 / 118, 1280 x 1280 141 / 134, 2048 x 1024
// 143 / 121, 2304 x 1008 149 / 125.  (Outside a graph the chain's launches take the host some 80 us.)
bool one_is_quicker(const OrthRun &r) {
    const int64_t sms = device_sms(current_device());
    if (sms <= 0 || r.steps == 0) return false;
    int64_t chain = 0;
    for (int which = 0; which < 3; ++which) chain += linear_cycles(orth_product(r, 0, which));
    const OrthTiles t = orth_one_tiles(r, sms);
    const int64_t kn = cdiv(r.n, 64), km = cdiv(std::max(r.R, r.C), 64);
    const int64_t ws = cdiv(t.sym * r.batch, sms), wx = cdiv(t.x * r.batch, sms);
    return 18000 + (t.bn == 64 ? 360 : 600) * (ws * (km + kn) + wx * kn) < chain;
}

// The iteration as a chain of launches.
ts_status orth_chain(const OrthRun &r) {
    const dim3 grid(static_cast<unsigned>(r.prep.chunks), static_cast<unsigned>(r.batch)), block(kOrthThreads);
    cudaError_t e;
    auto prepare = [&](auto norm, auto scale) {
        e = launch_pdl(norm, grid, block, 0, r.stream, r.prep);
        if (e == cudaSuccess) e = launch_pdl(scale, grid, block, 0, r.stream, r.prep);
    };
    if (r.f32)
        r.vec ? prepare(orth_norm_kernel<float, true>, orth_scale_kernel<float, true>)
              : prepare(orth_norm_kernel<float, false>, orth_scale_kernel<float, false>);
    else
        r.vec ? prepare(orth_norm_kernel<uint16_t, true>, orth_scale_kernel<uint16_t, true>)
              : prepare(orth_norm_kernel<uint16_t, false>, orth_scale_kernel<uint16_t, false>);
    if (e != cudaSuccess) return cuda_fail(e, "normalisation launch");

    for (int32_t i = 0; i < r.steps; ++i)
        for (int which = 0; which < 3; ++which) {
            const ts_status s = linear_product(orth_product(r, i, which));
            if (s != TS_OK) return s;
        }
    return TS_OK;
}

constexpr int64_t kMaxSide = 1 << 20, kMaxBatch = 65535;

// Matrices of a batch lie behind one another, or side by side: a row of each before the next row.
bool behind(int64_t R, int64_t C, int64_t ld, int64_t matrix) { return matrix >= (R - 1) * ld + C; }
bool matrices_overlap(int64_t batch, int64_t R, int64_t C, int64_t ld, int64_t matrix) {
    return !behind(R, C, ld, matrix) && (matrix < C || ld < (batch - 1) * matrix + C);
}
// All rows of a batch as rows of one pitch, or what encloses them.
RowsInMemory rows_of_batch(const void *ptr, int64_t batch, int64_t R, int64_t C, int64_t ld, int64_t matrix, int64_t esize) {
    if (batch == 1) return {ptr, R, C * esize, ld * esize};
    if (!behind(R, C, ld, matrix)) return {ptr, R, ((batch - 1) * matrix + C) * esize, ld * esize};
    if (R == 1) return {ptr, batch, C * esize, matrix * esize};
    if (matrix % ld == 0) return {ptr, (batch - 1) * (matrix / ld) + R, C * esize, ld * esize};
    const int64_t all = ((batch - 1) * matrix + (R - 1) * ld + C) * esize;
    return {ptr, 1, all, all};
}

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
    if (batch > 1 && R > 0 && C > 0 && (matrices_overlap(batch, R, C, ldg, g_matrix) || matrices_overlap(batch, R, C, ldo, o_matrix) ||
                      g_matrix > (int64_t(1) << 37) || o_matrix > (int64_t(1) << 37)))
        return fail(TS_ERR_INVALID_ARG, "matrices overlap or are too far apart (g_matrix=%lld o_matrix=%lld)",
                    static_cast<long long>(g_matrix), static_cast<long long>(o_matrix));
    if (batch == 0 || R == 0 || C == 0) return TS_OK;
    if (!G || !O) return fail(TS_ERR_INVALID_ARG, "G or O is NULL");
    const int gsize = g_type == TS_OUT_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(G) % gsize || reinterpret_cast<uintptr_t>(O) % 2)
        return fail(TS_ERR_INVALID_ARG, "G or O is not aligned to its element size");
    const RowsInMemory g_rows = rows_of_batch(G, batch, R, C, ldg, g_matrix, gsize), o_rows = rows_of_batch(O, batch, R, C, ldo, o_matrix, 2);
    const OrthPlan plan = plan_orth(batch, R, C, steps);
    if (!workspace || workspace_bytes < plan.total())
        return fail(TS_ERR_INVALID_ARG, "the workspace must hold %lld bytes", static_cast<long long>(plan.total()));
    if (reinterpret_cast<uintptr_t>(workspace) % 256)
        return fail(TS_ERR_INVALID_ARG, "the workspace must start on a 256-byte boundary");
    if (rows_overlap(g_rows, o_rows)) return fail(TS_ERR_INVALID_ARG, "O overlaps G");
    const RowsInMemory scratch{workspace, 1, plan.total(), plan.total()};
    if (rows_overlap(scratch, g_rows) || rows_overlap(scratch, o_rows))
        return fail(TS_ERR_INVALID_ARG, "the workspace overlaps G or O");

    char *const ws = static_cast<char *>(workspace);
    OrthRun r;
    std::memset(&r, 0, sizeof r);
    r.f32 = gsize == 4;
    r.vec = reinterpret_cast<uintptr_t>(G) % 16 == 0 && (R <= 1 || (ldg * gsize) % 16 == 0) &&
            (batch <= 1 || (g_matrix * gsize) % 16 == 0);
    r.batch = batch;
    r.R = R;
    r.C = C;
    r.n = plan.n;
    r.steps = steps;
    r.a = a;
    r.b = b;
    r.c = cc;
    for (int i = 0; i < 2; ++i) r.X[i] = reinterpret_cast<uint16_t *>(ws + plan.x(i));
    r.A = reinterpret_cast<uint16_t *>(ws + plan.a());
    r.B = reinterpret_cast<uint16_t *>(ws + plan.b());
    r.ldx = plan.ldx;
    r.ldn = plan.ldn;
    r.O = O;
    r.ldo = ldo;
    r.o_matrix = o_matrix;
    r.barrier = reinterpret_cast<int32_t *>(ws + plan.barrier());
    r.timeout_s = o->timeout_s;
    r.stream = static_cast<cudaStream_t>(stream);
    OrthParams &p = r.prep;
    p.G = G;
    p.ldg = ldg;
    p.g_matrix = g_matrix;
    p.X = steps > 0 ? ws : static_cast<char *>(O);
    p.ldx = steps > 0 ? plan.ldx : ldo;
    p.x_matrix = steps > 0 ? R * plan.ldx : o_matrix;
    p.partial = reinterpret_cast<float *>(ws + plan.partial());
    p.R = R;
    p.C = C;
    p.vecs = cdiv(C, r.vec ? 16 / gsize : 1);
    p.div_vecs = fast_div_for(p.vecs);
    p.chunks = static_cast<int32_t>(std::min(plan.chunks, cdiv(R * p.vecs, kOrthShare)));
    p.to_bf16 = steps == 0;
    p.eps = o->eps > 0.f ? o->eps : 1e-7f;
    return one_is_quicker(r) ? orth_one(r) : orth_chain(r);
}

}  // extern "C"
