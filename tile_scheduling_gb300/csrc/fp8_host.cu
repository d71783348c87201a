// Host side of the block-scaled 8-bit products: argument checks, planning, tensor maps, launch.
#include <algorithm>
#include <cstring>

#include "common.h"
#include "fp8_params.h"
#include "ptx.cuh"
#include "fp8_groups.cuh"

namespace ts {

extern const Fp8Variant fp8_128_1_block, fp8_128_1_row, fp8_128_1_grouped, fp8_256_1_block, fp8_256_1_row,
    fp8_256_1_grouped, fp8_256_2_block, fp8_256_2_row, fp8_256_2_grouped, fp8_32_block, fp8_32_grouped;

namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr double kDefaultTimeoutS = 2.0;
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
constexpr int kRasterGroup = 8;  // tile rows of a raster band, as the bf16 product's default

// K = 0: the rows of D (grouped: of group blockIdx.y) are empty sums.
template <class T>
__global__ void fp8_zero_kernel(T *D, int64_t N, int64_t ldd, const __grid_constant__ Fp8Params p) {
    grid_dep_wait();
    int64_t lo = 0, hi = p.M;
    if (p.groups > 0 && !group_rows(p, static_cast<int32_t>(blockIdx.y), lo, hi) && blockIdx.x == 0 && threadIdx.x == 0)
        report_group(p, static_cast<int32_t>(blockIdx.y));
    const int64_t total = (hi - lo) * N;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / N;
        D[(lo + r) * ldd + (i - r * N)] = T(0);
    }
}

const Fp8Variant *find_fp8(int bn, int cg, bool rows, bool grouped, int a_rows) {
    static const Fp8Variant *const all[] = {&fp8_128_1_block, &fp8_128_1_row, &fp8_128_1_grouped,
                                            &fp8_256_1_block, &fp8_256_1_row, &fp8_256_1_grouped,
                                            &fp8_256_2_block, &fp8_256_2_row, &fp8_256_2_grouped,
                                            &fp8_32_block,    &fp8_32_grouped};
    for (const Fp8Variant *v : all)
        if (v->bn == bn && v->cg == cg && v->rows == rows && v->grouped == grouped && v->a_rows == a_rows) return v;
    return nullptr;
}

// groups < 0: plain product.
ts_status fp8_product(const void *A, const float *SA, const void *B, const float *SB, void *D, const int64_t *offsets,
                      int64_t groups, int64_t M, int64_t N, int64_t K, int32_t out, const ts_fp8_opts *opts,
                      void *stream) {
    ts_fp8_opts z;
    std::memset(&z, 0, sizeof z);
    const ts_fp8_opts *o = opts ? opts : &z;
    const bool grouped = groups >= 0;
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^31-1] (M=%lld N=%lld K=%lld)",
                    static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K));
    if (grouped && groups > kMaxExperts)
        return fail(TS_ERR_UNSUPPORTED, "%lld groups exceed the %d-group limit", static_cast<long long>(groups),
                    kMaxExperts);
    // a group starts at any row, and the last row of its last tile must be a 32-bit coordinate
    if (grouped && M > kMaxDim - 255)
        return fail(TS_ERR_UNSUPPORTED, "M = %lld: a grouped product takes at most 2^31 - 256 rows",
                    static_cast<long long>(M));
    if (out != TS_OUT_BF16 && out != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "out_dtype %d", out);
    if (o->a_type != TS_FP8_E4M3 && o->a_type != TS_FP8_E5M2) return fail(TS_ERR_INVALID_ARG, "a_type %d", o->a_type);
    if (o->b_type != TS_FP8_E4M3 && o->b_type != TS_FP8_E5M2) return fail(TS_ERR_INVALID_ARG, "b_type %d", o->b_type);
    if (o->b_scale != TS_SCALE_BLOCK && o->b_scale != TS_SCALE_ROW)
        return fail(TS_ERR_INVALID_ARG, "b_scale %d", o->b_scale);
    if (o->trans_b != 0 && o->trans_b != 1) return fail(TS_ERR_INVALID_ARG, "trans_b = %d (0 or 1)", o->trans_b);
    if (o->tile < TS_TILE_AUTO || o->tile > TS_TILE_256x256_2CTA) return fail(TS_ERR_INVALID_ARG, "tile %d", o->tile);
    if (o->max_workers < 0 || o->timeout_s < 0 || o->lda < 0 || o->ldb < 0 || o->ldd < 0 || o->b_group < 0 ||
        o->sa_row < 0 || o->sa_blk < 0 || o->sb_row < 0 || o->sb_blk < 0 || o->sb_group < 0)
        return fail(TS_ERR_INVALID_ARG, "negative option");
    const bool rows = o->b_scale == TS_SCALE_ROW;
    if (rows && o->trans_b) return fail(TS_ERR_UNSUPPORTED, "row scales need B with K contiguous (trans_b = 0)");
    if (rows && grouped) return fail(TS_ERR_UNSUPPORTED, "grouped products take block scales");

    const int64_t b_rows = o->trans_b ? K : N, b_cols = o->trans_b ? N : K;
    const int64_t kblocks = cdiv(K, kScaleBlock), nblocks = cdiv(N, kScaleBlock);
    // a single row's pitch is never used, but for the default distance of B's groups: take one
    // that suits a tensor map
    const bool b_pitched = b_rows > 1 || (groups > 1 && !o->b_group);
    const int64_t b_pitch = b_pitched && o->ldb ? o->ldb : b_cols;
    const int64_t lda = M > 1 ? (o->lda ? o->lda : K) : cdiv(K, 16) * 16;
    const int64_t ldb = b_rows > 1 ? b_pitch : cdiv(b_cols, 16) * 16;
    const int64_t ldd = o->ldd ? o->ldd : N;
    if (lda < K || b_pitch < b_cols || ldd < N || lda > (int64_t(1) << 38) || b_pitch > (int64_t(1) << 38) ||
        ldd > (int64_t(1) << 37))
        return fail(TS_ERR_INVALID_ARG, "leading dimensions must cover a row (lda=%lld ldb=%lld ldd=%lld)",
                    static_cast<long long>(lda), static_cast<long long>(b_pitch), static_cast<long long>(ldd));
    if (M == 0 || N == 0 || groups == 0) return TS_OK;
    if (!D) return fail(TS_ERR_INVALID_ARG, "D is NULL");
    if (grouped && !offsets) return fail(TS_ERR_INVALID_ARG, "offsets is NULL");
    if (grouped && reinterpret_cast<uintptr_t>(offsets) % 8)
        return fail(TS_ERR_INVALID_ARG, "offsets is not aligned to 8 bytes");
    const int esize = out == TS_OUT_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(D) % esize) return fail(TS_ERR_INVALID_ARG, "D is not aligned to its element size");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t dbytes = ((M - 1) * ldd + N) * esize;
    if (K == 0) {
        ts_status zs;
        Fp8Params zp;
        std::memset(&zp, 0, sizeof zp);
        zp.status = device_status_word(&zs);
        if (!zp.status) return zs;
        zp.M = static_cast<int32_t>(M);
        zp.groups = grouped ? static_cast<int32_t>(groups) : 0;
        zp.offsets = offsets;
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>(cdiv(M * N, 256), grouped ? 64 : 4096)),
                        grouped ? static_cast<unsigned>(groups) : 1u);
        cudaError_t e = out == TS_OUT_F32
                            ? launch_pdl(fp8_zero_kernel<float>, grid, dim3(256), 0, st, static_cast<float *>(D), N,
                                         ldd, zp)
                            : launch_pdl(fp8_zero_kernel<uint16_t>, grid, dim3(256), 0, st,
                                         static_cast<uint16_t *>(D), N, ldd, zp);
        return e == cudaSuccess ? TS_OK : cuda_fail(e, "zero-fill launch");
    }
    if (!A || !B || !SA || !SB) return fail(TS_ERR_INVALID_ARG, "A, B or their scales are NULL");
    if (reinterpret_cast<uintptr_t>(A) % 16 || reinterpret_cast<uintptr_t>(B) % 16)
        return fail(TS_ERR_UNSUPPORTED, "A and B must start on a 16-byte boundary");
    if (reinterpret_cast<uintptr_t>(SA) % 4 || reinterpret_cast<uintptr_t>(SB) % 4)
        return fail(TS_ERR_INVALID_ARG, "scales are not aligned to 4 bytes");
    if (lda % 16 || ldb % 16)
        return fail(TS_ERR_UNSUPPORTED, "rows of A and B must start on 16-byte boundaries (lda, ldb multiples of 16)");
    const int64_t depth = grouped ? groups : 1;
    if (depth > 1 && (b_pitch > (int64_t(1) << 39) / b_rows || o->b_group > (int64_t(1) << 39)))
        return fail(TS_ERR_INVALID_ARG, "groups of B are too far apart (ldb=%lld b_group=%lld)",
                    static_cast<long long>(b_pitch), static_cast<long long>(o->b_group));
    const int64_t b_group = o->b_group ? o->b_group : b_rows * b_pitch;
    if (depth > 1 && b_group % 16)
        return fail(TS_ERR_UNSUPPORTED, "groups of B must start on 16-byte boundaries (b_group a multiple of 16)");
    if (depth > 1 && b_group < (b_rows - 1) * ldb + b_cols)
        return fail(TS_ERR_INVALID_ARG, "b_group %lld is shorter than a group of B", static_cast<long long>(b_group));
    const int64_t abytes = (M - 1) * lda + K, bbytes = (depth - 1) * b_group + (b_rows - 1) * ldb + b_cols;
    if (ranges_overlap(D, dbytes, A, abytes) || ranges_overlap(D, dbytes, B, bbytes))
        return fail(TS_ERR_INVALID_ARG, "D overlaps A or B");

    const int sms = device_sms(current_device());
    if (sms <= 0) return fail(TS_ERR_CUDA, "cannot query the SM count");
    const int64_t sms_ = sms;  // 64-bit for the products below
    // Few rows: tiles of 32 (of which the MMA makes 128).  A 128-row box that lies mostly past
    // A's end is slow to load, and the ring holds nine stages of weights instead of five: 1 x
    // 4096 x 8192 8.9 us for 13.8, 8 x 8192 x 8192 14.7 for 22.1; 40 rows over 32 groups of
    // 4096 x 2048 32.8 for 46.4.  With more rows there is no gain (256 over 64 groups of 2048 x
    // 2048 43.4 and 43.2, 1024 49.5 and 46.5).
    const bool few = !rows && (grouped ? M < 128 && M / groups <= 16 : M <= 32);
    // CTAs of a cluster that share the K blocks of each of `units` 128x128 tiles, and the
    // cycles that a tile then takes: 430 a K block (660 with row scales) and, from two CTAs
    // on, the exchange of their partial sums.  Measured, 128 x 4096 x 4096 (32 tiles) by 1 /
    // 2 / 4 CTAs 10.2 / 9.1 / 7.9 us, 128 x 512 x 8192 (4 tiles) by 1 / 2 / 4 / 8 16.9 / 12.2
    // / 8.9 / 7.7; but 128 x 2048 x 8192 by 4 / 8 9.2 / 15.4: its 16 clusters of eight do
    // not run at once.
    auto split_of = [&](int64_t units, int64_t &cycles) {
        int64_t best = 1;
        cycles = kblocks * (rows ? 660 : 430);
        const Fp8Variant *v1 = find_fp8(128, 1, rows, false, few ? 32 : 128);
        for (int64_t c = 2; c <= kMaxCluster && c <= kblocks && units * c <= sms_; ++c) {
            if (o->max_workers > 0 && units * c > o->max_workers) break;
            const int64_t t = cdiv(kblocks, c) * (rows ? 660 : 430) + 3000 + 16 * std::min<int64_t>(M, 128) + 150 * c;
            if (t >= cycles || (v1 && v1->clusters(static_cast<int>(c)) < units)) continue;
            best = c;
            cycles = t;
        }
        return best;
    };
    int tile = o->tile;
    if (tile == TS_TILE_AUTO && grouped) {
        // By the mean rows of a group, and the waves that its tiles make: tiles / workers and
        // half a wave, as their number is an estimate (a group ends in half a tile).  Measured,
        // 32 groups of 4096 x 2048, 128x128 / 128x256 / pair: 64 rows each 48 / 50 / 60 us, 128
        // 62 / 60 / 69, 256 89 / 82 / 85, 512 162 / 139 / 145; 8 groups of 2048 rows 142 / 119
        // / 120, of 128 rows 20.6 / 23.4 / 21.6; 20 groups of 300 rows, 1000 x 1500, 25.6 /
        // 21.3 / 25.7.
        const int64_t row_tiles = cdiv(M, 128) + groups / 2;
        const int64_t t1 = row_tiles * cdiv(N, 128), t2 = row_tiles * cdiv(N, 256);
        tile = M / groups >= 96 && (2 * t2 + sms_) * 740 < (2 * t1 + sms_) * 430 ? TS_TILE_128x256 : TS_TILE_128x128;
    } else if (tile == TS_TILE_AUTO) {
        // The tile with the fewest cycles: waves of workers times what a K block of a tile
        // takes (measured steady states; a pair's, with its smaller L2 traffic, is shorter
        // while a wave is the only one, but it starts later).  Measured, N = K = 4096,
        // 128x128 / 128x256 / pair: M = 512 10.9 / 15.0 / 15.6 us, 1024 19.2 / 17.7 / 16.6,
        // 1536 26.7 / 30.0 / 28.7, 2048 34.8 / 30.8 / 29.1; 2048^3 11.5 / 9.9 / 10.6; row
        // scales, M = 512 14.1 / 22.7 / 23.2, 1024 25.6 / 25.1 / 23.6, 2048 48.2 / 44.8 / 43.2.
        const int64_t u1 = cdiv(M, 128) * cdiv(N, 128), u2 = cdiv(M, 128) * cdiv(N, 256),
                      u3 = cdiv(M, 256) * cdiv(N, 256);
        int64_t c1;
        split_of(u1, c1);
        c1 *= cdiv(u1, sms_);
        const int64_t c2 = cdiv(u2, sms_) * kblocks * (rows ? 1230 : 740);
        const int64_t w3 = cdiv(u3, sms_ / 2);
        const int64_t c3 = w3 > 1 ? w3 * kblocks * (rows ? 1195 : 720) : kblocks * (rows ? 1120 : 640) + 2000;
        tile = c1 <= c2 && c1 <= c3 ? TS_TILE_128x128 : c2 <= c3 ? TS_TILE_128x256 : TS_TILE_256x256_2CTA;
    }
    const int bn = tile == TS_TILE_128x128 ? 128 : 256, cg = tile == TS_TILE_256x256_2CTA ? 2 : 1;
    const int a_rows = few && tile == TS_TILE_128x128 ? 32 : 128;
    const Fp8Variant *v = find_fp8(bn, cg, rows, grouped, a_rows);
    if (!v) return fail(TS_ERR_UNSUPPORTED, "no compiled variant");

    Fp8Launch L;
    std::memset(&L, 0, sizeof L);
    Fp8Params &p = L.p;
    const int64_t tile_m = a_rows < 128 ? a_rows : 128 * cg;
    const int64_t tiles_m = cdiv(M, tile_m), tiles_n = cdiv(N, bn);
    // grouped: every group may end in a partial tile
    const int64_t units = grouped ? (tiles_m + groups) * tiles_n : tiles_m * tiles_n;
    if (units * cg > kMaxDim) return fail(TS_ERR_UNSUPPORTED, "too many output tiles");
    ts_status s;
    {
        const int64_t dims[2] = {K, M}, strides[1] = {lda};
        const int box[2] = {kScaleBlock, a_rows};
        if ((s = encode_map(&L.a, A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dims, strides, box)) != TS_OK) return s;
    }
    {
        const int64_t dims[3] = {b_cols, b_rows, depth}, strides[2] = {ldb, depth > 1 ? b_group : cdiv(b_group, 16) * 16};
        const int box[3] = {128, o->trans_b ? 128 : bn / cg, 1};
        if ((s = encode_map(&L.b, B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box)) != TS_OK) return s;
    }
    p.store_bytes = 2;
    for (int b : {16, 4})
        if (reinterpret_cast<uintptr_t>(D) % b == 0 && (ldd * esize) % b == 0) {
            p.store_bytes = b;
            break;
        }
    p.tma_store = p.store_bytes == 16;
    if (p.tma_store) {
        const int64_t dims[3] = {N, M, 1}, strides[2] = {ldd * esize, M * ldd * esize};
        const int box[3] = {128 / esize, 32, 1};  // a warp's staging buffer
        if ((s = encode_map(&L.d, D, out == TS_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            3, dims, strides, box)) != TS_OK)
            return s;
    }
    unsigned long long *status = device_status_word(&s);
    if (!status) return s;

    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.tiles_m = static_cast<int32_t>(tiles_m);
    p.tiles_n = static_cast<int32_t>(tiles_n);
    p.num_kb = static_cast<int32_t>(kblocks);
    p.num_units = static_cast<int32_t>(units);
    int64_t tile_cycles;
    p.split = !grouped && tile == TS_TILE_128x128 ? static_cast<int32_t>(split_of(units, tile_cycles)) : 1;
    p.raster_group = kRasterGroup;
    p.div_group_tiles = fast_div_for(kRasterGroup * tiles_n);
    p.div_group_rows = fast_div_for(kRasterGroup);
    p.div_last_rows = fast_div_for(tiles_m - (cdiv(tiles_m, kRasterGroup) - 1) * kRasterGroup);
    p.trans_b = o->trans_b;
    p.out = out;
    // Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A format at bits
    // 7-9 and B format at 10-12 (0 e4m3, 1 e5m2), A K-major (bit 15 = 0), B K-major or
    // N-major (bit 16); the kernel adds N and M of its tile.
    p.idesc = (1u << 4) | (uint32_t(o->a_type) << 7) | (uint32_t(o->b_type) << 10) | (uint32_t(o->trans_b) << 16);
    p.groups = grouped ? static_cast<int32_t>(groups) : 0;
    p.offsets = offsets;
    p.sa = SA;
    const bool sa_given = o->sa_row || o->sa_blk, sb_given = o->sb_row || o->sb_blk;
    p.sa_row = sa_given ? o->sa_row : 1;
    p.sa_blk = sa_given ? o->sa_blk : M;
    p.sb = SB;
    // strides of SB as it lies ([rows of B / 128][columns of B / 128], or [N][K / 128] for
    // row scales), then along N and along K
    const int64_t sb_row = sb_given ? o->sb_row : (rows ? kblocks : cdiv(b_cols, kScaleBlock));
    const int64_t sb_blk = sb_given ? o->sb_blk : 1;
    p.sb_n = o->trans_b ? sb_blk : sb_row;
    p.sb_k = o->trans_b ? sb_row : sb_blk;
    p.sb_group = o->sb_group ? o->sb_group : kblocks * nblocks;
    p.sa_vec = p.sa_row == 1 && p.sa_blk % 4 == 0 && reinterpret_cast<uintptr_t>(SA) % 16 == 0;
    p.sb_vec = rows && p.sb_n == 1 && p.sb_k % 4 == 0 && reinterpret_cast<uintptr_t>(SB) % 16 == 0;
    p.D = D;
    p.ldd = ldd;
    const double tmo = o->timeout_s > 0 ? o->timeout_s : kDefaultTimeoutS;
    p.timeout_ns = std::max<uint64_t>(1, static_cast<uint64_t>(std::min(tmo, 60.0) * 1e9));
    p.drain_ns = kDrainNs;
    p.status = status;
    int64_t workers = std::min<int64_t>(units, sms / cg);
    if (o->max_workers > 0) workers = std::min<int64_t>(workers, o->max_workers);
    L.grid = p.split > 1 ? units * p.split : workers * cg;
    L.cluster = p.split > 1 ? p.split : cg;
    L.stream = st;
    cudaError_t e = v->launch(L);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "8-bit product launch");
}

}  // namespace
}  // namespace ts

extern "C" {

ts_status ts_gemm_fp8(const void *A, const float *SA, const void *B, const float *SB, void *D, int64_t M, int64_t N,
                      int64_t K, int32_t out_dtype, const ts_fp8_opts *opts, void *stream) {
    return ts::fp8_product(A, SA, B, SB, D, nullptr, -1, M, N, K, out_dtype, opts, stream);
}

ts_status ts_gemm_fp8_grouped(const void *A, const float *SA, const void *B, const float *SB, void *D,
                              const int64_t *offsets, int64_t groups, int64_t M, int64_t N, int64_t K,
                              int32_t out_dtype, const ts_fp8_opts *opts, void *stream) {
    if (groups < 0) return ts::fail(TS_ERR_INVALID_ARG, "groups = %lld", static_cast<long long>(groups));
    return ts::fp8_product(A, SA, B, SB, D, offsets, groups, M, N, K, out_dtype, opts, stream);
}

}  // extern "C"
