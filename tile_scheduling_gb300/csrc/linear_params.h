// Parameter block of the products with a fused epilogue (a linear layer's forward and
// backward products, the products of an orthogonalised update), shared by host and device code.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"
#include "gemm_params.h"

namespace ts {

enum : int32_t { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4, kActs = 5 };

// Element type of the outputs inside the library: the public ones and fp16.
enum : int32_t { OUT_F16 = 2 };

struct LinParams {
    int32_t M, N;                     // of D
    int32_t tiles_m, tiles_n, num_kb;
    int32_t num_units, tiles_per_matrix;  // all matrices of a batch; one matrix (its upper triangle with `sym`)
    int32_t bn, tx_bytes;             // columns of a tile; bytes of a stage's loads (both CTAs of a pair)
    int32_t bufs;                     // staging buffers of an epilogue warp
    int32_t raster_group;
    FastDiv div_group_tiles, div_group_rows, div_last_rows;  // sym: the first divides by tiles_n + 1
    FastDiv div_matrix;
    int32_t a_mn, b_mn;               // 1: the operand lies with its rows of D (its columns) contiguous, not K
    uint32_t idesc;                   // MMA instruction descriptor without the tile shape
    int32_t out;                      // OUT_BF16 / OUT_F32 / OUT_F16, also of pre (and of aux but in the iteration)
    int32_t act;                      // of the forward epilogue, or whose slope the backward one multiplies by
    int32_t slope;                    // 0: D = act(alpha * acc + bias) + beta * aux; 1: D = alpha * acc * act'(aux)
    int32_t stages;                   // of the operand ring
    int32_t split;                    // the split kernel: CTAs of a cluster that share K
    int32_t sym;                      // 1: D is symmetric: tiles above the diagonal are stored twice
    int32_t store_bytes;              // 16, 4 or 2: what the bases and rows of D, aux and pre are aligned to
    float alpha, beta;                // the iteration's products; 1 otherwise
    const void *bias;                 // N values added to every row, or NULL
    int32_t bias_f32, bias_vec;       // bias_vec (for the split kernel): it starts on a 16-byte boundary
    const void *aux;                  // residual or pre-activation [M][N], or NULL
    int64_t ld_aux, aux_matrix;
    void *pre;                        // alpha * acc + bias, or NULL
    int64_t ld_pre;
    void *D;
    int64_t ldd, d_matrix;            // elements
    uint64_t timeout_ns, drain_ns;
    unsigned long long *status;
};

struct LinLaunch {
    CUtensorMap a, b, d, aux, pre;
    LinParams p;
    int64_t grid;
    cudaStream_t stream;
};

// What a product's epilogue has beside the sum: aux at most; bias, activation and aux; pre as well; the slope.
enum : int { LIN_BARE, LIN_FULL, LIN_PRE, LIN_SLOPE };

struct LinVariant {
    int bn, cg, mode;
    cudaError_t (*launch[3])(const LinLaunch &);  // by the type of D, OUT_F16: the iteration's products
    int (*stages)(int bufs);
};

constexpr int kMaxSplit = 8;  // most CTAs that share a tile's K: the portable cluster size

struct SplitVariant {
    int bn, swap;
    cudaError_t (*launch)(const LinLaunch &);
    int (*clusters)(int size, int ctas);  // clusters of so many CTAs that run at once, with so many on an SM
    int (*stages)(int split, int ctas);   // operand stages of a CTA
};

// One product as its callers describe it: D[z] = epilogue(A[z] B[z]^T), z < batch.
struct LinCall {
    const void *A, *B;
    int64_t lda, ldb, a_matrix, b_matrix;  // elements
    int64_t a_rows, b_rows;                // rows that the operands have, 0: M and N (the rest of D comes of zeros)
    int a_mn, b_mn, f16;                   // f16: a product of the iteration, with fp16 operands and aux; else bf16, aux as D
    void *D;
    int64_t ldd, d_matrix;
    const void *aux;
    int64_t ld_aux, aux_matrix;
    void *pre;
    int64_t ld_pre;
    const void *bias;
    int bias_f32;
    int64_t M, N, K, batch;
    int out, act, slope, sym;
    float alpha, beta;
    int tile;                              // ts_tile
    int64_t max_workers;
    double timeout_s;
    cudaStream_t stream;
};
// Plans and launches a product whose arguments have been checked.
ts_status linear_product(const LinCall &c);
// An estimate of its cycles, from one launch to the next.
int64_t linear_cycles(const LinCall &c);

// The forward product of at most so many rows of x runs in a kernel of its own.
constexpr int kFewTokens = 8;
bool linear_few_takes(const LinCall &c);
ts_status linear_few(const LinCall &c);

}  // namespace ts
