// Parameter block of the block-scaled 8-bit products, shared by host and device code.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_params.h"

namespace ts {

constexpr int kScaleBlock = 128;   // elements of K (and, for block scales, rows of B) that share a scale
constexpr int kMaxCluster = 8;      // most CTAs that share a tile's K blocks: the portable cluster size
constexpr int kMaxExperts = 1024;  // most groups of a grouped product: their tile counts are scanned in shared memory

struct Fp8Params {
    int32_t M, N, K;
    int32_t tiles_m, tiles_n, num_kb;  // tiles_m and num_units: plain product only
    int32_t num_units;
    int32_t split;      // CTAs of a cluster that share a tile's K blocks (1: none; plain 128x128 tiles only)
    int32_t raster_group;
    FastDiv div_group_tiles, div_group_rows, div_last_rows;
    int32_t trans_b;    // 1: B is [K][N]
    int32_t out;        // OUT_BF16 / OUT_F32
    int32_t tma_store;  // 1: D's rows and base suit a TMA store
    int32_t store_bytes;  // 16, 4 or 2: what D's base and rows are aligned to
    uint32_t idesc;     // MMA instruction descriptor without the tile shape
    int32_t groups;     // grouped product: groups, and their row offsets on the device
    const int64_t *offsets;
    const float *sa;    // scale of A's row m, K block b: sa[m * sa_row + b * sa_blk]
    int64_t sa_row, sa_blk;
    int32_t sa_vec, sb_vec;  // four scales along M (row scales: along N) lie on a 16-byte boundary, from a multiple of four
    // scale of B: sb[g * sb_group + i * sb_n + b * sb_k] for K block b and column n of
    // D, i = n / 128 (block scales) or i = n (row scales)
    const float *sb;
    int64_t sb_n, sb_k, sb_group;
    void *D;
    int64_t ldd;
    uint64_t timeout_ns, drain_ns;
    unsigned long long *status;
};

struct Fp8Launch {
    CUtensorMap a, b, d;
    Fp8Params p;
    int64_t grid;
    int cluster;  // CTAs of a cluster
    cudaStream_t stream;
};

struct Fp8Variant {
    int bn, cg, rows, grouped, a_rows;
    cudaError_t (*launch)(const Fp8Launch &);
    int (*clusters)(int size);  // clusters of so many CTAs that run at once
};

}  // namespace ts
