// Host side of the fused-epilogue products: argument checks, planning, tensor maps, launch.
#include <algorithm>
#include <cstring>

#include "common.h"
#include "linear_params.h"

namespace ts {

extern const SplitVariant split_128[3], split_swap_64[3], split_swap_32[3];  // by the type of D
#define TS_LINEAR_MODES(TILE) linear_##TILE##_bare, linear_##TILE##_full, linear_##TILE##_pre, linear_##TILE##_slope
extern const LinVariant TS_LINEAR_MODES(128_1), TS_LINEAR_MODES(256_1), TS_LINEAR_MODES(256_2);

namespace {

constexpr int64_t kMaxSize = 0x7fffffffLL - 511;  // the last tile's coordinates stay in 32 bits
constexpr int64_t kMaxPitch = int64_t(1) << 37;
// The epilogue of a tile waits for the whole of its K loop, some 0.2 us for 64 of K: what a wait may take by itself,
// and for each K block.
constexpr double kDefaultTimeoutS = 2.0, kDefaultBlockS = 1e-6;
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
constexpr int kRasterGroup = 8;
// What a tile takes beside its columns, as columns: the loads and barriers of a K block.
constexpr int64_t kWidthOverhead = 16;

const LinVariant &find_linear(int bn, int cg, int mode) {
#define TS_LINEAR_TILE(TILE) {&linear_##TILE##_bare, &linear_##TILE##_full, &linear_##TILE##_pre, &linear_##TILE##_slope}
    static const LinVariant *const all[3][4] = {TS_LINEAR_TILE(128_1), TS_LINEAR_TILE(256_1), TS_LINEAR_TILE(256_2)};
    return *all[cg == 2 ? 2 : bn > 128 ? 1 : 0][mode];
}

int64_t aligned_pitch(int64_t ld, int64_t rows, int64_t cols, int unit) {
    return rows > 1 ? ld : cdiv(cols, unit) * unit;  // a single row's pitch is never used
}

// Tensor map of an operand of `rows` rows of D by K, in boxes of 64 of K by box_rows, or (mn) of 64 rows by 64 of K.
ts_status operand_map(CUtensorMap *m, const void *ptr, int mn, int64_t rows, int64_t K, int64_t batch, int64_t ld,
                      int64_t matrix, int box_rows) {
    const int64_t outer = mn ? K : rows, inner = mn ? rows : K;
    const int64_t pitch = aligned_pitch(ld, outer, inner, 8);
    // Rows that end in the first half of a 32-byte sector make the boxes that pass their end slow (both
    // gradients' operands 1000 wide, 4096 deep: 16.5 us, 1024 wide 12.1).  Where the last row starts on a sector
    // the map takes them to its end: the sector is there, and what it holds meets only rows of D that do not exist.
    const uintptr_t last = reinterpret_cast<uintptr_t>(ptr) + ((batch - 1) * matrix + (outer - 1) * pitch) * 2;
    const int64_t dims[3] = {mn && last % 32 == 0 ? cdiv(inner, 16) * 16 : inner, outer, batch};
    const int64_t strides[2] = {pitch * 2, (batch > 1 ? matrix : outer * pitch) * 2};
    const int box[3] = {64, mn ? 64 : box_rows, 1};
    return encode_map(m, ptr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box);
}

ts_status output_map(CUtensorMap *m, const void *ptr, int esize, int64_t M, int64_t N, int64_t batch, int64_t ld,
                     int64_t matrix) {
    const int64_t pitch = aligned_pitch(ld, M, N, 16 / esize);
    const int64_t dims[3] = {N, M, batch}, strides[2] = {pitch * esize, (batch > 1 ? matrix : M * pitch) * esize};
    const int box[3] = {128 / esize, 32, 1};  // a warp's staging buffer
    return encode_map(m, ptr, esize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims,
                      strides, box);
}

}  // namespace

namespace {

int64_t triangle(int64_t n) { return n * (n + 1) / 2; }

// How a product runs: a tile of a persistent CTA or pair with `bn` columns, or (sv) a tile whose K is
// shared by a cluster of `split` CTAs, `ctas` of them on an SM.
struct LinPlan {
    int bn, cg;
    const SplitVariant *sv;
    int split, ctas;
    int64_t cycles;  // an estimate, from one launch to the next
};

// Cycles that the loads of 16 rows of an operand take for a K block (or of 16 of its rows of K, 64 wide):
// a row is 128 bytes, one line of memory where rows start on lines, else two, and five sectors where rows
// start off sectors.  Measured on K blocks of 256 and 384 rows: on lines no more than the rest of a K
// block, on sectors 1.9 cycles a row (480 to 510 and 720), off them 2.8 (700 to 720 and 1040).
int64_t row_cycles(const void *ptr, int64_t rows, int64_t ld, int64_t batch, int64_t matrix) {
    const uint64_t at = reinterpret_cast<uintptr_t>(ptr) | (rows > 1 ? ld * 2 : 0) | (batch > 1 ? matrix * 2 : 0);
    return at % 128 == 0 ? 16 : at % 32 == 0 ? 30 : 44;
}

LinPlan plan_product(const LinCall &c, int64_t sms) {
    const int64_t nkb = cdiv(c.K, 64);
    const int kind = c.f16 ? OUT_F16 : c.out;
    const int64_t load_a = row_cycles(c.A, c.a_mn ? c.K : c.M, c.lda, c.batch, c.a_matrix);
    const int64_t load_b = row_cycles(c.B, c.b_mn ? c.K : c.N, c.ldb, c.batch, c.b_matrix);
    // cycles of a K block: what they are with rows on lines, or the loads of so many rows of A and B
    auto block = [&](int64_t cycles, int64_t rows_a, int64_t rows_b, int64_t b_least = 0) {
        return std::max(cycles, (rows_a * load_a + rows_b * std::max(load_b, b_least)) / 16);
    };
    const int64_t m1 = cdiv(c.M, 128), m2 = cdiv(c.M, 256), n1 = cdiv(c.N, 128), n2 = cdiv(c.N, 256);
    const int64_t u1 = c.batch * (c.sym ? triangle(n1) : m1 * n1), u3 = c.batch * (c.sym ? triangle(n2) : m2 * n2);
    LinPlan pl{128, 1, nullptr, 1, 1, INT64_MAX};
    // Few tiles: K shared by a cluster, the fewest cycles of a cluster size whose clusters all run at once.
    if (c.tile == TS_TILE_AUTO && nkb > 0 && c.max_workers == 0) {
        // Cycles fitted to measurements: K blocks of a CTA, its launch, and the rest.  Of 128-column tiles with a
        // bf16 output, K 512, by 2 / 4 / 8 CTAs a tile and by a persistent CTA: 9 tiles 5.7 / 5.2 / 5.9 and
        // 5.4 us, 36 tiles 5.9 / 6.4 and 5.5; a silu adds 0.4 to the first and 0.9 to the last, a residual
        // 0.7 and 0.4.  Of tiles for 32 tokens, K 1024, by 1 / 2 / 4 / 8 CTAs: 16 tiles 5.2 / 4.4 / 3.8 / 8.0
        // (which do not all run at once), 64 tiles 5.4 / 5.1; for 64 tokens 6.2 / 5.1 / 4.4 and 6.2 / 5.7.
        // For up to 32 tokens also more tiles than run at once, two on an SM: 9 and 16 tokens, 65536 x 2048, 45 us,
        // by persistent CTAs 64 and 63; 128000 x 4096 159, 192 and 161.  (For 64 tokens 50 and 47.)
        struct Fit {
            int64_t block[4], cta, rest[4];  // by 1, 2, 4 and 8 CTAs a tile
        };
        auto consider = [&](const SplitVariant &v, int64_t units, const Fit &f) {
            for (int k = v.swap ? 1 : 2, i = v.swap ? 0 : 1; k <= kMaxSplit && k <= nkb; k *= 2, ++i) {
                const int ctas = v.swap && units * k > sms ? 2 : 1;
                const bool queue = v.bn == 32 && k == 1 && ctas == 2;
                if ((units * k > ctas * sms && !queue) || (k > 1 && v.clusters(k, ctas) < units)) break;
                const int64_t loop = cdiv(nkb, k) * block(f.block[i], v.swap ? v.bn : 128, 128);
                const int64_t t = (queue ? loop * units / sms : loop * ctas) + f.cta * units * k + f.rest[i] +
                                  (c.act ? 900 : 0) + (c.aux ? 1300 : 0);
                if (t < pl.cycles) pl.cycles = t, pl.sv = &v, pl.split = k, pl.ctas = ctas;
            }
        };
        consider(split_128[kind], u1, {{0, 390, 500, 500}, 18, {0, 9200, 8900, 10100}});
        // an operand with its rows contiguous comes in boxes of 64
        if (!c.sym && c.batch == 1 && c.M <= 64) {
            if (c.M <= 32 && !c.a_mn)
                consider(split_swap_32[kind], n1, {{290, 290, 380, 470}, 10, {5600, 6500, 6100, 6300}});
            else
                consider(split_swap_64[kind], n1, {{290, 290, 380, 470}, 10, {7200, 7500, 7000, 7700}});
        }
    }
    // Columns of a 256-column tile: the width whose waves of workers take the fewest cycles in all.  With
    // B's rows contiguous a CTA's columns start on sectors, and on lines where they are whole boxes of 64:
    // 4096 x 4096 x 4096 on pairs 81 us with 224 columns (four waves either way), 87 with 256;
    // 4096 x 2048 x 2048 24.6 with 256, 30.1 with 240, whose halves start off sectors.
    auto cost = [&](int64_t pair, int64_t bn) {  // of a K block on a 256-column tile
        return block((pair == 2 ? 520 : 590) * (bn + kWidthOverhead) / (256 + kWidthOverhead), 128, bn / pair,
                     c.b_mn && bn % (64 * pair) != 0 ? 30 : 0);
    };
    // A wave behind another takes its K loop or, if that is shorter, an epilogue: cycles of one, from 8192 x 4096 x 64 on 128- and 256-column tiles
    // (bf16 18.5 and 15.4 us, with silu 28.2 and 27.1, with a residual 29.5 and 27.9; fp32 22.4 and 23.6).
    const int64_t column = 1250 + (c.act ? 1450 : 0) + (c.aux ? 1650 : 0) + (c.out == OUT_F32 ? 600 : 0);
    auto wave_cycles = [&](int64_t waves, int64_t k_block, int64_t bn) {
        return (waves - 1) * std::max(nkb * k_block, 900 + bn * column / 128) + nkb * k_block;
    };
    auto width = [&](int64_t rows, int64_t workers, int64_t pair, int64_t &waves) {
        int64_t bn = 256;
        waves = cdiv(rows * n2 * c.batch, workers);
        for (int64_t b = 240; !c.sym && b > 128; b -= 16) {
            if (c.b_mn && b % (16 * pair) != 0) continue;
            const int64_t w = cdiv(rows * cdiv(c.N, b) * c.batch, workers);
            if (wave_cycles(w, cost(pair, b), b) < wave_cycles(waves, cost(pair, bn), bn)) bn = b, waves = w;
        }
        return bn;
    };
    int64_t w2, w3;
    const int64_t bn2 = width(m1, sms, 1, w2), bn3 = width(m2, sms / 2, 2, w3);
    // The tile with the fewest cycles: waves of workers times what a K block of a tile takes, and the rest,
    // in which the last epilogue shows.
    // (Plain, 9 and 144 tiles: 128 columns 7700 cycles, 256 9200 and 11100, pairs 9400 and 12400.)
    const int64_t slow = (c.act ? 2100 : 0) + (c.aux ? 700 : 0) + (c.sym ? 5000 : 0);
    const int64_t slow2 = (c.act ? 3000 : 0) + (c.aux ? 1300 : 0) + (c.sym ? 5000 : 0);
    const int64_t c1 = wave_cycles(cdiv(u1, sms), block(385, 128, 128), 128) + 7700 + slow;
    const int64_t c2 = wave_cycles(w2, cost(1, bn2), bn2) + 9200 + 13 * std::min(m1 * n2 * c.batch, sms) + slow2;
    const int64_t c3 = wave_cycles(c.sym ? cdiv(u3, sms / 2) : w3, cost(2, bn3), bn3) + 9400 + 40 * std::min(u3, sms / 2) + slow2;
    int tile = c.tile;
    if (tile == TS_TILE_AUTO) {
        const int64_t least = std::min(c1, std::min(c.sym ? c1 : c2, c3));
        if (pl.cycles < least) return pl;
        tile = least == c1 ? TS_TILE_128x128 : least == c3 ? TS_TILE_256x256_2CTA : TS_TILE_128x256;
    }
    pl.sv = nullptr;
    pl.bn = static_cast<int>(tile == TS_TILE_128x128 ? 128 : tile == TS_TILE_256x256_2CTA ? bn3 : bn2);
    pl.cg = tile == TS_TILE_256x256_2CTA ? 2 : 1;
    pl.cycles = tile == TS_TILE_128x128 ? c1 : tile == TS_TILE_256x256_2CTA ? c3 : c2;
    return pl;
}

}  // namespace

int64_t linear_cycles(const LinCall &c) { return plan_product(c, std::max(1, device_sms(current_device()))).cycles; }

ts_status linear_product(const LinCall &c) {
    const int64_t sms = device_sms(current_device()), nkb = cdiv(c.K, 64);
    if (sms <= 0) return fail(TS_ERR_CUDA, "cannot query the SM count");
    const LinPlan pl = plan_product(c, sms);
    const SplitVariant *const sv = pl.sv;
    const int bn = pl.bn, cg = pl.cg;
    const LinVariant &v = find_linear(bn, cg, c.pre ? LIN_PRE : c.slope && c.act ? LIN_SLOPE : c.bias || c.act ? LIN_FULL : LIN_BARE);

    LinLaunch L;
    std::memset(&L, 0, sizeof L);
    LinParams &p = L.p;
    const bool swap = sv && sv->swap;
    const int64_t tiles_m = swap ? 1 : cdiv(c.M, sv ? 128 : 128 * cg), tiles_n = cdiv(c.N, sv ? 128 : bn);
    const int64_t per = c.sym ? triangle(tiles_n) : tiles_m * tiles_n, units = per * c.batch;
    if (units * cg > 0x7fffffffLL) return fail(TS_ERR_UNSUPPORTED, "too many output tiles");
    const int esize = c.out == OUT_F32 ? 4 : 2;
    p.store_bytes = 2;
    for (int b : {16, 4}) {
        auto fits = [&](const void *ptr, int64_t ld, int64_t matrix) {
            return !ptr || (reinterpret_cast<uintptr_t>(ptr) % b == 0 && (c.M <= 1 || (ld * esize) % b == 0) &&
                            (c.batch <= 1 || (matrix * esize) % b == 0));
        };
        if (fits(c.D, c.ldd, c.d_matrix) && fits(c.aux, c.ld_aux, c.aux_matrix) && fits(c.pre, c.ld_pre, 0)) {
            p.store_bytes = b;
            break;
        }
    }
    ts_status s = TS_OK;
    if (c.K > 0) {
        // swapped, the rows of D are the instruction's columns
        CUtensorMap &a = swap ? L.b : L.a, &b = swap ? L.a : L.b;
        const int a_box = swap ? sv->bn : 128, b_box = sv ? 128 : bn / cg;
        if ((s = operand_map(&a, c.A, c.a_mn, c.a_rows ? c.a_rows : c.M, c.K, c.batch, c.lda, c.a_matrix, a_box)) != TS_OK) return s;
        if ((s = operand_map(&b, c.B, c.b_mn, c.b_rows ? c.b_rows : c.N, c.K, c.batch, c.ldb, c.b_matrix, b_box)) != TS_OK) return s;
    }
    if (p.store_bytes == 16 && !sv) {
        if ((s = output_map(&L.d, c.D, esize, c.M, c.N, c.batch, c.ldd, c.d_matrix)) != TS_OK) return s;
        if (c.aux && (s = output_map(&L.aux, c.aux, esize, c.M, c.N, c.batch, c.ld_aux, c.aux_matrix)) != TS_OK) return s;
        if (c.pre && (s = output_map(&L.pre, c.pre, esize, c.M, c.N, 1, c.ld_pre, 0)) != TS_OK) return s;
    }
    unsigned long long *status = device_status_word(&s);
    if (!status) return s;

    p.M = static_cast<int32_t>(c.M);
    p.N = static_cast<int32_t>(c.N);
    p.tiles_m = static_cast<int32_t>(tiles_m);
    p.tiles_n = static_cast<int32_t>(tiles_n);
    p.num_kb = static_cast<int32_t>(nkb);
    p.num_units = static_cast<int32_t>(units);
    p.tiles_per_matrix = static_cast<int32_t>(per);
    p.raster_group = kRasterGroup;
    p.div_group_tiles = fast_div_for(c.sym ? tiles_n + 1 : kRasterGroup * tiles_n);
    p.div_group_rows = fast_div_for(kRasterGroup);
    p.div_last_rows = fast_div_for(tiles_m - (cdiv(tiles_m, kRasterGroup) - 1) * kRasterGroup);
    p.div_matrix = fast_div_for(per);
    p.a_mn = swap ? c.b_mn : c.a_mn;
    p.b_mn = swap ? c.a_mn : c.b_mn;
    // Instruction descriptor, kind::f16: D fp32 (bits 4-5 = 1), A and B bf16 (bits 7-9 and 10-12 = 1)
    // or fp16 (0), A and B K-major (bits 15 and 16 = 0) or not; the kernel adds N and M of its tile.
    const uint32_t type = c.f16 ? 0u : 1u;
    p.idesc = (1u << 4) | (type << 7) | (type << 10) | (uint32_t(p.a_mn) << 15) | (uint32_t(p.b_mn) << 16);
    p.out = c.out;
    p.act = c.act;
    p.slope = c.slope;
    p.sym = c.sym;
    p.alpha = c.alpha;
    p.beta = c.beta;
    p.bias = c.bias;
    p.bias_f32 = c.bias_f32;
    p.bias_vec = reinterpret_cast<uintptr_t>(c.bias) % 16 == 0;
    p.aux = c.aux;
    p.ld_aux = c.ld_aux;
    p.aux_matrix = c.aux_matrix;
    p.pre = c.pre;
    p.ld_pre = c.ld_pre;
    p.D = c.D;
    p.ldd = c.ldd;
    p.d_matrix = c.d_matrix;
    const double tmo = c.timeout_s > 0 ? c.timeout_s : kDefaultTimeoutS + kDefaultBlockS * static_cast<double>(nkb);
    p.timeout_ns = std::max<uint64_t>(1, static_cast<uint64_t>(std::min(tmo, 60.0) * 1e9));
    p.drain_ns = kDrainNs;
    p.status = status;
    L.stream = c.stream;
    if (sv) {
        p.split = pl.split;
        p.stages = sv->stages(pl.split, pl.ctas);
        L.grid = units * pl.split;
        const cudaError_t e = sv->launch(L);
        return e == cudaSuccess ? TS_OK : cuda_fail(e, "split product launch");
    }
    p.bn = bn;
    // boxes of 64 rows where an operand's rows are contiguous, which may pass the tile's columns
    p.tx_bytes = cg * (128 * 128 + (c.b_mn ? cdiv(bn / cg, 64) * 64 : bn / cg) * 128);
    // Short K loops leave the epilogue as the bound, which two buffers keep moving: 4096 x 4096 x 256 with a
    // residual 15.5 us, 16.9 with one; x 1024 with gelu_tanh and preact 27.8 and 28.6 (alone 22.8 and 22.7).
    // Long ones need the ring: x 2048 48.4 and 45.9.
    p.bufs = nkb <= (c.act || c.aux || c.pre ? 16 : 8) ? 2 : 1;
    p.stages = v.stages(p.bufs);
    int64_t workers = std::min<int64_t>(units, sms / cg);
    if (c.max_workers > 0) workers = std::min<int64_t>(workers, c.max_workers);
    L.grid = workers * cg;
    const cudaError_t e = v.launch[c.f16 ? OUT_F16 : c.out](L);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "linear product launch");
}

namespace {

struct Matrix {
    const void *ptr;
    int64_t rows, cols, ld;
    int esize;
    RowsInMemory in_memory() const { return {ptr, rows, cols * esize, ld * esize}; }
};

bool overlap(const Matrix &a, const Matrix &b) { return rows_overlap(a.in_memory(), b.in_memory()); }

ts_status check_sizes(int64_t M, int64_t N, int64_t K, int32_t out, int32_t act, int32_t tile, int32_t max_workers,
                      double timeout_s) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return fail(TS_ERR_INVALID_ARG, "sizes must be in [0, 2^31 - 512] (M=%lld N=%lld K=%lld)",
                    static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K));
    if (out != TS_OUT_BF16 && out != TS_OUT_F32) return fail(TS_ERR_INVALID_ARG, "out_dtype %d", out);
    if (act < 0 || act >= kActs) return fail(TS_ERR_INVALID_ARG, "act %d", act);
    if (tile < TS_TILE_AUTO || tile > TS_TILE_256x256_2CTA) return fail(TS_ERR_INVALID_ARG, "tile %d", tile);
    if (max_workers < 0 || !(timeout_s >= 0)) return fail(TS_ERR_INVALID_ARG, "negative option");
    return TS_OK;
}

ts_status check_pitch(const char *name, int64_t ld, int64_t cols) {
    if (ld < cols || ld > kMaxPitch)
        return fail(TS_ERR_INVALID_ARG, "the row stride of %s (%lld) must cover a row of %lld elements", name,
                    static_cast<long long>(ld), static_cast<long long>(cols));
    return TS_OK;
}

ts_status check_operand(const char *name, const Matrix &m) {
    if (!m.ptr) return fail(TS_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(m.ptr) % 16)
        return fail(TS_ERR_UNSUPPORTED, "%s must start on a 16-byte boundary", name);
    if (m.rows > 1 && m.ld % 8)
        return fail(TS_ERR_UNSUPPORTED, "rows of %s must start on 16-byte boundaries (a stride that is a multiple of 8)",
                    name);
    return TS_OK;
}

ts_status check_output(const char *name, const Matrix &m) {
    if (reinterpret_cast<uintptr_t>(m.ptr) % m.esize)
        return fail(TS_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return TS_OK;
}

// `aux` may be D itself, element for element, and overlaps it in no other way.
ts_status check_aliases(const Matrix &A, const Matrix &B, const Matrix &D, const Matrix &aux, const Matrix &pre) {
    if (overlap(D, A) || overlap(D, B)) return fail(TS_ERR_INVALID_ARG, "the output overlaps an operand");
    if (overlap(D, aux) && !(D.ptr == aux.ptr && (D.ld == aux.ld || D.rows <= 1)))
        return fail(TS_ERR_INVALID_ARG, "the output overlaps the matrix its epilogue reads, and is not that matrix");
    if (overlap(pre, A) || overlap(pre, B) || overlap(pre, D) || overlap(pre, aux))
        return fail(TS_ERR_INVALID_ARG, "preact overlaps another matrix");
    return TS_OK;
}

#define TS_TRY(call)                       \
    do {                                   \
        const ts_status s_ = (call);       \
        if (s_ != TS_OK) return s_;        \
    } while (0)

// The two gradient products: D (rows x cols) from A and B, contracted over K.
ts_status grad_product(const char *b_name, const char *d_name, const Matrix &A, const Matrix &B, const Matrix &D,
                       const Matrix &aux, bool a_mn, bool slope, int64_t K, int32_t out, const ts_linear_grad_opts *o,
                       void *stream) {
    TS_TRY(check_pitch("grad_z", A.ld, A.cols));
    TS_TRY(check_pitch(b_name, B.ld, B.cols));
    TS_TRY(check_pitch(d_name, D.ld, D.cols));
    if (aux.ptr) TS_TRY(check_pitch(slope ? "preact" : "base", aux.ld, aux.cols));
    if (D.rows == 0 || D.cols == 0) return TS_OK;
    if (!D.ptr) return fail(TS_ERR_INVALID_ARG, "%s is NULL", d_name);
    TS_TRY(check_output(d_name, D));
    TS_TRY(check_output(slope ? "preact" : "base", aux));
    if (K > 0) {
        TS_TRY(check_operand("grad_z", A));
        TS_TRY(check_operand(b_name, B));
    }
    TS_TRY(check_aliases(A, B, D, aux, Matrix{nullptr, 0, 0, 0, 1}));
    LinCall c;
    std::memset(&c, 0, sizeof c);
    c.A = A.ptr;
    c.lda = A.ld;
    c.a_mn = a_mn;
    c.B = B.ptr;
    c.ldb = B.ld;
    c.b_mn = 1;
    c.D = const_cast<void *>(D.ptr);
    c.ldd = D.ld;
    c.aux = aux.ptr;
    c.ld_aux = aux.ld;
    c.M = D.rows;
    c.N = D.cols;
    c.K = K;
    c.batch = 1;
    c.out = out;
    c.act = slope ? o->act : ACT_NONE;
    c.slope = slope;
    c.alpha = c.beta = 1.f;
    c.tile = o->tile;
    c.max_workers = o->max_workers;
    c.timeout_s = o->timeout_s;
    c.stream = static_cast<cudaStream_t>(stream);
    return linear_product(c);
}

}  // namespace
}  // namespace ts

extern "C" {

ts_status ts_linear(const void *x, const void *w, void *y, int64_t M, int64_t N, int64_t K, int32_t out_dtype,
                    const ts_linear_opts *opts, void *stream) {
    using namespace ts;
    ts_linear_opts z;
    std::memset(&z, 0, sizeof z);
    const ts_linear_opts *o = opts ? opts : &z;
    TS_TRY(check_sizes(M, N, K, out_dtype, o->act, o->tile, o->max_workers, o->timeout_s));
    if (o->bias && o->bias_type != TS_OUT_BF16 && o->bias_type != TS_OUT_F32)
        return fail(TS_ERR_INVALID_ARG, "bias_type %d", o->bias_type);
    const int esize = out_dtype == TS_OUT_F32 ? 4 : 2, bsize = o->bias_type == TS_OUT_F32 ? 4 : 2;
    const Matrix A{x, M, K, o->ldx ? o->ldx : K, 2}, B{w, N, K, o->ldw ? o->ldw : K, 2};
    const Matrix D{y, M, N, o->ldy ? o->ldy : N, esize};
    const Matrix R{o->residual, M, N, o->ld_residual ? o->ld_residual : N, esize};
    const Matrix Z{o->preact, M, N, o->ld_preact ? o->ld_preact : N, esize};
    TS_TRY(check_pitch("x", A.ld, K));
    TS_TRY(check_pitch("w", B.ld, K));
    TS_TRY(check_pitch("y", D.ld, N));
    if (R.ptr) TS_TRY(check_pitch("residual", R.ld, N));
    if (Z.ptr) TS_TRY(check_pitch("preact", Z.ld, N));
    if (M == 0 || N == 0) return TS_OK;
    if (!y) return fail(TS_ERR_INVALID_ARG, "y is NULL");
    TS_TRY(check_output("y", D));
    TS_TRY(check_output("residual", R));
    TS_TRY(check_output("preact", Z));
    if (K > 0) {
        TS_TRY(check_operand("x", A));
        TS_TRY(check_operand("w", B));
    }
    TS_TRY(check_aliases(A, B, D, R, Z));
    const Matrix bias{o->bias, 1, N, N, bsize};
    if (reinterpret_cast<uintptr_t>(o->bias) % bsize)
        return fail(TS_ERR_INVALID_ARG, "bias is not aligned to its element size");
    if (overlap(bias, D) || overlap(bias, Z)) return fail(TS_ERR_INVALID_ARG, "an output overlaps the bias");
    LinCall c;
    std::memset(&c, 0, sizeof c);
    c.A = x;
    c.lda = A.ld;
    c.B = w;
    c.ldb = B.ld;
    c.D = y;
    c.ldd = D.ld;
    c.aux = R.ptr;
    c.ld_aux = R.ld;
    c.pre = o->preact;
    c.ld_pre = Z.ld;
    c.bias = o->bias;
    c.bias_f32 = o->bias_type == TS_OUT_F32;
    c.M = M;
    c.N = N;
    c.K = K;
    c.batch = 1;
    c.out = out_dtype;
    c.act = o->act;
    c.alpha = c.beta = 1.f;
    c.tile = o->tile;
    c.max_workers = o->max_workers;
    c.timeout_s = o->timeout_s;
    c.stream = static_cast<cudaStream_t>(stream);
    return linear_few_takes(c) ? linear_few(c) : linear_product(c);
}

ts_status ts_linear_grad_input(const void *grad_z, const void *w, void *grad_x, int64_t M, int64_t N, int64_t K,
                               int32_t out_dtype, const ts_linear_grad_opts *opts, void *stream) {
    using namespace ts;
    ts_linear_grad_opts z;
    std::memset(&z, 0, sizeof z);
    const ts_linear_grad_opts *o = opts ? opts : &z;
    TS_TRY(check_sizes(M, N, K, out_dtype, o->act, o->tile, o->max_workers, o->timeout_s));
    if ((o->act != TS_ACT_NONE) != (o->aux != nullptr))
        return fail(TS_ERR_INVALID_ARG, "an activation and its pre-activations are given together");
    const int esize = out_dtype == TS_OUT_F32 ? 4 : 2;
    return grad_product("w", "grad_x", Matrix{grad_z, M, N, o->ldg ? o->ldg : N, 2},
                        Matrix{w, N, K, o->ldb ? o->ldb : K, 2}, Matrix{grad_x, M, K, o->ldd ? o->ldd : K, esize},
                        Matrix{o->aux, M, K, o->ld_aux ? o->ld_aux : K, esize}, false, true, N, out_dtype, o, stream);
}

ts_status ts_linear_grad_weight(const void *grad_z, const void *x, void *grad_w, int64_t M, int64_t N, int64_t K,
                                int32_t out_dtype, const ts_linear_grad_opts *opts, void *stream) {
    using namespace ts;
    ts_linear_grad_opts z;
    std::memset(&z, 0, sizeof z);
    const ts_linear_grad_opts *o = opts ? opts : &z;
    TS_TRY(check_sizes(M, N, K, out_dtype, o->act, o->tile, o->max_workers, o->timeout_s));
    if (o->act != TS_ACT_NONE) return fail(TS_ERR_INVALID_ARG, "a weight gradient passes no activation");
    const int esize = out_dtype == TS_OUT_F32 ? 4 : 2;
    return grad_product("x", "grad_w", Matrix{grad_z, M, N, o->ldg ? o->ldg : N, 2},
                        Matrix{x, M, K, o->ldb ? o->ldb : K, 2}, Matrix{grad_w, N, K, o->ldd ? o->ldd : K, esize},
                        Matrix{o->aux, N, K, o->ld_aux ? o->ld_aux : K, esize}, true, false, M, out_dtype, o, stream);
}

}  // extern "C"
