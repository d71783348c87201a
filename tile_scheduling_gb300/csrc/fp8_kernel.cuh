// Block-scaled 8-bit product for sm_103a, plain and grouped by rows:
//
//   D[m][n] = sum over K blocks b of  SA[m][b] * SB[n][b] * sum_{k in b} A[m][k] * B[n][k]
//
// with 8-bit operands (e4m3 or e5m2) and one fp32 scale for each row of A and
// 128 elements of K, and for each 128 x 128 block (or each row) of B.
//
// The scales change every 128 elements of K, so the tensor core cannot carry one
// accumulator through the K loop.  Each K block of a tile is a chain of four MMAs (K = 32
// each) into a TMEM slot; promotion warps read the slot back, scale it, and add it to fp32
// registers that hold the tile's running sum, while the MMAs fill the other slots.
//
// What bounds it.  A K block of 128 x 256 outputs takes the tensor core 512 cycles; the
// promotion reads 128 KB of TMEM and issues 512 two-wide multiply-adds (1024 with row
// scales) beside it.  The steady state is 720 to 760 cycles a K block, 1200 with row scales.
// On a pair it is the promotion warps that share the MMA warp's scheduler (in the CTA that
// issues, they run 1.8 times slower than in the other); on 128x256 tiles the operands'
// traffic through shared memory, 96 KB a K block written and read, is close to its
// bandwidth as well.  From the commit of a slot to its hand-back some 1000 cycles pass,
// most of them latencies: 128-column slots (four of them) hide it on a pair (8192^3 603 us
// with two of 256 columns); two 256-column slots are enough where both halves of the
// promotion warps read every slot (128x256).
//
// Measured, launches back to back: 8192^3, e4m3, bf16 out, 361 us at the full clock and 400
// once the power cap lowers it, after some 40 ms (3050 and 2750 TFLOP/s; a pair); 4096 x
// 4096 x 8191 with row scales 158 to 161 us (1740; 128x128); 2047 x 4096 x 6144 41 us (2530;
// a pair); 16384 rows over 32 groups of 4096 x 2048, ragged, 131 us and 147 under the cap
// (2100 and 1870; 128x256); 1 x 4096 x 8192 7.7 to 8.9 us (4 TB/s; split over four CTAs a
// tile).
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer of the operand ring
//   warp 1       TMEM allocator and MMA issuer
//   warp 2       scales: copies them to shared memory, a chunk of four K blocks at a time
//   warp 3       initialises the barriers
//   warps 4..11  promotion and epilogue: warp 4 + j holds rows 32 * (j % 4) of the
//                tile, one row per lane; j / 4 picks the columns (see Fp8Cfg)
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fp8_groups.cuh"
#include "fp8_params.h"
#include "gemm_kernel.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace ts {

template <int BN_, int CG_, bool ROWS_, bool GROUPED_, int SC_, int AR_>
struct Fp8Cfg {
    static constexpr int BN = BN_, CG = CG_;
    static constexpr bool ROWS = ROWS_, GROUPED = GROUPED_;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (kRoleWarps + EPI_WARPS);
    // The MMA always takes BM = 128 rows of A.  Tiles of few rows (AR = 32: a batch of
    // decoded tokens, or experts with a few rows each) load only those; what the MMA reads
    // past them is whatever lies there, and the rows it makes of it are never read.
    static constexpr int BM = 128, AR = AR_, TILE_M = AR == BM ? BM * CG : AR;
    static constexpr int BK = kScaleBlock;  // one scale block: a 128-byte swizzle row
    static constexpr int UMMA_K = 32;
    static constexpr int B_ROWS = BN / CG;
    static constexpr int A_BYTES = AR * BK;
    static constexpr int B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int TX_BYTES = STAGE_BYTES * CG;
    // TMEM slots of SC columns; a K block fills H of them.  H = 1: all eight promotion
    // warps read every slot, warp j the half j / 4 of its columns.  H = 2: the warps with
    // j / 4 = h read slot h of the K block whole; on a CTA pair its MMA takes 64 rows of B
    // from each CTA's tile, so its two 64-column segments lie 128 columns apart.
    static constexpr int SC = SC_;
    static constexpr bool SPLIT = BN == 128 && CG == 1 && !GROUPED;  // K may be split over a cluster
    static constexpr int SLOTS = 512 / SC;
    static constexpr int H = BN / SC;
    static constexpr int COLS = BN / 2;  // columns of one promotion warp
    // Columns of one TMEM load; PIPE: the next load is issued before a load's columns are
    // added.  Row scales, 4096 x 4096 x 8191 on 128x128 / 128x256 / pair: 157 / 170 / 162 us,
    // without 176 / 177 / 168.  Block scales, 8192 x 8192 x 2048: 128x128 134 us, without
    // 138; but 155 and 117 on the wider tiles against 120 and 112, and 256
    // rows over 64 experts of 2048 x 2048 (32-row tiles) 44.0 against 43.6.
    static constexpr bool PIPE = ROWS || (BN == 128 && AR == BM);
    static constexpr int LD = PIPE ? 32 : 64;
    static constexpr int TEMPTY_ARRIVALS = EPI_WARPS / H * CG;
    static constexpr int TMEM_COLS = 512;
    // First column, within the tile, of a promotion warp's 64-column segment seg.
    static __device__ __forceinline__ int32_t seg_col(int h, int seg) {
        if constexpr (H == 2 && CG == 2) return 64 * h + 128 * seg;
        return COLS * h + 64 * seg;
    }
    // A 256-column tile's running sums take 128 registers of a promotion thread, with the
    // loads in flight more than an even split of the register file gives it: the role
    // warps hand theirs over.  128 * ROLE_REGS + 256 * EPI_REGS = 384 * LAUNCH_REGS.
    static constexpr bool SHIFT_REGS = BN == 256;
    static constexpr int LAUNCH_REGS = 168, ROLE_REGS = 56, EPI_REGS = 224;
    static_assert(128 * ROLE_REGS + 256 * EPI_REGS == 384 * LAUNCH_REGS, "register split");
    // Store staging of one warp: buffers of 32 rows x 128 bytes, enough for its part of a
    // bf16 tile, so that the part is written, fenced and stored at once (subtile after
    // subtile through fewer buffers, the epilogue took 3000 cycles of a pair).
    static constexpr int EPI_ROW = 128, EPI_BUF = 32 * EPI_ROW, EPI_BUFS = COLS / 64;
    static constexpr int EPI_BYTES = EPI_WARPS * EPI_BUFS * EPI_BUF;
    // Scales travel in chunks of four K blocks, four chunks deep: per K block those of the
    // tile's rows, then those of its one or two 128-column blocks (ROWS: its columns).
    static constexpr int CHUNK = 4, CHUNKS = 4;
    static constexpr int KB_SCALES = 128 + (ROWS ? BN : 4);
    static constexpr int CHUNK_BYTES = CHUNK * KB_SCALES * 4;
    static constexpr int SCALE_BYTES = CHUNKS * CHUNK_BYTES;
    static constexpr int PREFIX_BYTES = GROUPED ? (kMaxExperts + 8) * 4 : 0;
    static constexpr int BAR_BYTES = 512;
    static constexpr int FIXED_BYTES = 1024 + EPI_BYTES + SCALE_BYTES + PREFIX_BYTES + BAR_BYTES;
    static constexpr int STAGES = (kSmemLimit - FIXED_BYTES) / STAGE_BYTES;
    static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * STAGE_BYTES;
    static_assert(STAGES >= 2, "ring too shallow");
    static_assert(AR == BM || (AR == 32 && CG == 1), "tile rows");
    // the MMA's reads past a short A stage, and the split's partial sums, stay in the ring
    static_assert((STAGES - 1) * A_BYTES + BM * BK <= STAGES * STAGE_BYTES, "A overrun");
    static_assert(!SPLIT || STAGES * STAGE_BYTES >= BM * BN * 4, "partial sums");
    static_assert((2 * STAGES + 2 * SLOTS + 2 * CHUNKS + 1) * 8 + 16 <= BAR_BYTES, "barrier region");
};

// Shared-memory descriptor of a B tile whose rows run along N (B is [K][N]): rows of
// 128 bytes (128 values of n) for consecutive k, 8-row atoms 1024 bytes apart along
// K (stride byte offset), the next 128 values of n in the next 16 KB box (leading
// byte offset).
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t smem_addr) {
    return uint64_t((smem_addr & 0x3FFFFu) >> 4) | (uint64_t(16384 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Where four columns (group g of BN / 4 = 32) of row r lie among a CTA's partial sums: a
// row is 512 bytes, so that the reading warps (a lane a group) fetch whole lines of another
// CTA's shared memory, its 16-byte units permuted within 128, so that the writing warps (a
// lane a row) meet no bank conflicts.  128 x 4096 x 4096 by four CTAs a tile 7.9 us; with
// the 16 bytes of a column group's rows next to each other instead, 11.9.
__device__ __forceinline__ uint32_t partial_at(int32_t g, int32_t r) {
    return static_cast<uint32_t>(r * 32 + (g ^ (r & 7))) * 16u;
}

// A warp stores `rows` rows of 128 bytes from swizzled staging to D, from row0 and col
// on, the columns below N: `bytes` (16, 4 or 2) is what D's rows are aligned to and a
// lane stores at once.
template <int ESIZE>
__device__ __forceinline__ void store_rows(char *D, int32_t row0, int32_t rows, int32_t col, int32_t N, int64_t ldd,
                                           int32_t bytes, uint32_t stage, int lane) {
    // byte b of a staged row r
    auto at = [&](int r, int b) { return stage + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15); };
    const int32_t left = min(N - col, 128) * ESIZE;  // bytes of a row below N, where they end within the subtile
    char *const dst = D + (static_cast<int64_t>(row0) * ldd + col) * ESIZE;
    const int64_t pitch = ldd * ESIZE;
    if (bytes == 16 && left >= 128) {
        const int b = (lane & 7) * 16;
#pragma unroll 4
        for (int r = lane >> 3; r < rows; r += 4)
            *reinterpret_cast<uint4 *>(dst + r * pitch + b) = ld_shared_v4(at(r, b));
    } else if (bytes >= 4) {
        const int b = lane * 4;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint32_t v = ld_shared_u32(at(r, b));
            if (b + 4 <= left)
                *reinterpret_cast<uint32_t *>(dst + r * pitch + b) = v;
            else if (ESIZE == 2 && b + 2 <= left)
                *reinterpret_cast<uint16_t *>(dst + r * pitch + b) = static_cast<uint16_t>(v);
        }
    } else {
        const int b = lane * 2;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint16_t v0 = ld_shared_u16(at(r, b)), v1 = ld_shared_u16(at(r, b + 64));
            if (b + 2 <= left) *reinterpret_cast<uint16_t *>(dst + r * pitch + b) = v0;
            if (b + 66 <= left) *reinterpret_cast<uint16_t *>(dst + r * pitch + b + 64) = v1;
        }
    }
}

// One work unit: an output tile.
struct Fp8Unit {
    int32_t row0, row_end;  // rows [row0, row_end) of D may be written (row_end: past the group's, D's or a short tile's last)
    int32_t col0;
    int32_t group;
};

template <class C>
__device__ __forceinline__ Fp8Unit fp8_unit(int32_t u, const Fp8Params &p, const int32_t *prefix) {
    Fp8Unit w;
    if constexpr (C::GROUPED) {
        // prefix[g]: units of the groups before g.  Units of a group walk its row
        // tiles first, so the CTAs that share a panel of its weights run together.
        int32_t lo = 0, hi = p.groups;  // prefix[lo] <= u < prefix[hi]
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (prefix[mid] <= u) lo = mid; else hi = mid;
        }
        int64_t r0, r1;
        group_rows(p, lo, r0, r1);
        const int32_t tm = static_cast<int32_t>((r1 - r0 + C::TILE_M - 1) / C::TILE_M);
        const int32_t local = u - prefix[lo];
        const int32_t nb = local / tm;
        w.group = lo;
        w.row0 = static_cast<int32_t>(r0) + (local - nb * tm) * C::TILE_M;
        w.row_end = C::TILE_M < C::BM ? min(static_cast<int32_t>(r1), w.row0 + C::TILE_M) : static_cast<int32_t>(r1);
        w.col0 = nb * C::BN;
    } else {
        int32_t mb, nb;
        raster(u, p, mb, nb);
        w.group = 0;
        w.row0 = mb * C::TILE_M;
        w.row_end = C::TILE_M < C::BM ? min(p.M, w.row0 + C::TILE_M) : p.M;
        w.col0 = nb * C::BN;
    }
    return w;
}

template <int BN, int CG, bool ROWS, bool GROUPED, int SC, int AR>
__global__ void __launch_bounds__(Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>::THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const __grid_constant__ Fp8Params p) {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t s_a = base;
    const uint32_t s_b = s_a + C::STAGES * C::A_BYTES;
    const uint32_t s_epi = s_b + C::STAGES * C::B_BYTES;
    const uint32_t s_scale = s_epi + C::EPI_BYTES;
    const uint32_t s_prefix = s_scale + C::SCALE_BYTES;
    const uint32_t s_bar = s_prefix + C::PREFIX_BYTES;
    int32_t *const prefix = reinterpret_cast<int32_t *>(gbase + (s_prefix - base));
    auto full = [&](uint32_t s) { return s_bar + 8u * s; };
    auto empty = [&](uint32_t s) { return s_bar + 8u * (C::STAGES + s); };
    auto tfull = [&](uint32_t a) { return s_bar + 8u * (2 * C::STAGES + a); };
    auto tempty = [&](uint32_t a) { return s_bar + 8u * (2 * C::STAGES + C::SLOTS + a); };
    auto sfull = [&](uint32_t c) { return s_bar + 8u * (2 * C::STAGES + 2 * C::SLOTS + c); };
    auto sempty = [&](uint32_t c) { return s_bar + 8u * (2 * C::STAGES + 2 * C::SLOTS + C::CHUNKS + c); };
    const uint32_t mma_done = s_bar + 8u * (2 * C::STAGES + 2 * C::SLOTS + 2 * C::CHUNKS);
    const uint32_t tail = s_bar + 8u * (2 * C::STAGES + 2 * C::SLOTS + 2 * C::CHUNKS + 1);
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(gbase + (tail - base));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(gbase + (tail - base) + 4);

    // uniform across the warp, and known to be: the role loops then run on uniform registers
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (p.tma_store) prefetch_tmap(&tmD);
    }
    if (warp == 3 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < C::SLOTS; ++a) {
            mbar_init(tfull(a), 1);
            mbar_init(tempty(a), C::TEMPTY_ARRIVALS);
        }
        for (int c = 0; c < C::CHUNKS; ++c) {
            mbar_init(sfull(c), 32);  // every lane of the scale warp, when its copies have landed
            mbar_init(sempty(c), C::EPI_WARPS);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(tail, C::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    grid_dep_wait();
    grid_dep_launch();
    int32_t num_units = p.num_units;
    if constexpr (GROUPED) {
        // Units per group, then their running sum (warp 2, 32 groups at a time).  Ordered offsets
        // make at most p.num_units in all; disordered ones may leave groups whose ranges overlap
        // and whose sum passes 32 bits: it is formed in 64 and cut there.
        for (int32_t g = threadIdx.x; g < p.groups; g += C::THREADS) {
            int64_t lo, hi;
            if (!group_rows(p, g, lo, hi) && blockIdx.x == 0) report_group(p, g);
            prefix[g + 1] = static_cast<int32_t>((hi - lo + C::TILE_M - 1) / C::TILE_M) * p.tiles_n;
        }
        if (threadIdx.x == 0) prefix[0] = 0;
        __syncthreads();
        if (warp == 2) {
            int64_t run = 0;
            for (int32_t g0 = 0; g0 < p.groups; g0 += 32) {
                const int32_t g = g0 + lane;
                int64_t v = g < p.groups ? prefix[g + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += o;
                }
                if (g < p.groups) prefix[g + 1] = static_cast<int32_t>(min(run + v, static_cast<int64_t>(p.num_units)));
                run += __shfl_sync(0xffffffffu, v, 31);
            }
        }
    }
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if constexpr (GROUPED) num_units = prefix[p.groups];
    int32_t first = static_cast<int32_t>(blockIdx.x) / CG;
    const int32_t step = static_cast<int32_t>(gridDim.x) / CG;
    // K blocks [kb0, kb0 + num_kb) of every unit; split over a cluster, this CTA's share of
    // its one unit (step is then at least the number of units)
    int32_t kb0 = 0, num_kb = p.num_kb, part = 0;
    if constexpr (C::SPLIT) {
        if (p.split > 1) {
            part = static_cast<int32_t>(cluster_ctarank());
            first = static_cast<int32_t>(blockIdx.x) / p.split;
            kb0 = static_cast<int32_t>(static_cast<int64_t>(part) * p.num_kb / p.split);
            num_kb = static_cast<int32_t>(static_cast<int64_t>(part + 1) * p.num_kb / p.split) - kb0;
        }
    }

    if (warp < kRoleWarps) {
    if constexpr (C::SHIFT_REGS) regs_dec<C::ROLE_REGS>();
    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        {
            const bool leader = elect_one();
            uint32_t stage = 0, phase = 0, issued = 0;
            bool alive = true;
            for (int32_t u = first; u < num_units && alive; u += step) {
                const Fp8Unit w = fp8_unit<C>(u, p, prefix);
                const int32_t a_row = w.row0 + static_cast<int32_t>(rank) * C::BM;
                const int32_t b_row = w.col0 + static_cast<int32_t>(rank) * C::B_ROWS;
                for (int32_t kb = 0; kb < num_kb; ++kb) {
                    if (!wait_phase(empty(stage), phase ^ 1u, abort_flag, p, WAIT_PRODUCER_EMPTY)) {
                        alive = false;
                        break;
                    }
                    if (rank == 0 && leader) mbar_arrive_expect_tx(full(stage), C::TX_BYTES);
                    const uint32_t da = s_a + stage * C::A_BYTES;
                    const uint32_t db = s_b + stage * C::B_BYTES;
                    const uint32_t fb = CG == 2 ? mapa(full(stage), 0) : full(stage);
                    const int32_t k = (kb0 + kb) * C::BK;
                    auto load_b = [&](uint32_t dst, int32_t x, int32_t y) {
                        if constexpr (CG == 1)
                            tma_load_3d(dst, &tmB, fb, x, y, w.group);
                        else
                            tma_load_3d_pair(dst, &tmB, fb, x, y, w.group);
                    };
                    if (leader) {
                        if constexpr (CG == 1)
                            tma_load_2d(da, &tmA, fb, k, a_row);
                        else
                            tma_load_2d_pair(da, &tmA, fb, k, a_row);
                        if (p.trans_b) {
#pragma unroll
                            for (int c = 0; c < C::B_ROWS / 128; ++c) load_b(db + c * 16384, b_row + 128 * c, k);
                        } else {
                            load_b(db, k, b_row);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every load has landed (seen on the even CTA's barriers) and every stage is released
            if (rank == 0) {
                const uint32_t n = issued < C::STAGES ? issued : C::STAGES;
                for (uint32_t i = 1; i <= n; ++i) {
                    const uint32_t b = issued - i;
                    wait_drain(full(b % C::STAGES), (b / C::STAGES) & 1u, abort_flag, p);
                }
            }
            for (int i = 0; i < C::STAGES; ++i) {
                if (!wait_drain(empty(stage), phase ^ 1u, abort_flag, p)) break;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        // The whole warp runs the loop, one elected lane issues: with the loop inside one
        // lane's branch every descriptor went through per-thread registers, and a K block
        // took some 630 cycles to issue (8192^3, no promotion: 362 us against 286).
        if (rank == 0) {
            const bool leader = elect_one();
            const uint32_t idesc = p.idesc | (uint32_t(SC >> 3) << 17) | (uint32_t((C::BM * CG) >> 4) << 24);
            // steps of B's start address in 16-byte units: one K = 32 MMA (32 bytes along a
            // K-major row, or 32 rows of 128 bytes) and one slot (its rows, or, along a row of
            // n, half of it or the next box)
            const uint32_t k_step = p.trans_b ? (32 * 128) >> 4 : 32 >> 4;
            const uint32_t h_step = p.trans_b ? (CG == 2 ? 64 : 16384) >> 4 : (C::B_BYTES / C::H) >> 4;
            uint32_t stage = 0, phase = 0, slot = 0, slot_phase = 0;
            bool alive = true;
            for (int32_t u = first; u < num_units && alive; u += step) {
                for (int32_t kb = 0; kb < num_kb && alive; ++kb) {
                    if (!wait_phase(full(stage), phase, abort_flag, p, WAIT_MMA_FULL)) {
                        alive = false;
                        break;
                    }
                    const uint64_t da = sw128_kmajor_desc(s_a + stage * C::A_BYTES);
                    const uint32_t b_at = s_b + stage * C::B_BYTES;
                    const uint64_t db = p.trans_b ? sw128_nmajor_desc(b_at) : sw128_kmajor_desc(b_at);
#pragma unroll 1
                    for (int h = 0; h < C::H; ++h) {
                        if (!wait_phase(tempty(slot), slot_phase ^ 1u, abort_flag, p, WAIT_MMA_TMEM_EMPTY)) {
                            alive = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < C::BK / C::UMMA_K; ++kk)
                                mma_f8<CG>(tmem_base + slot * SC, da + 2u * kk, db + h_step * h + k_step * kk, idesc,
                                           kk != 0);
                            if constexpr (CG == 1)
                                mma_commit(tfull(slot));
                            else
                                mma_commit_pair(tfull(slot), 0x3);
                        }
                        __syncwarp();
                        if (++slot == C::SLOTS) {
                            slot = 0;
                            slot_phase ^= 1u;
                        }
                    }
                    if (!alive) break;
                    if (leader) {
                        if constexpr (CG == 1)
                            mma_commit(empty(stage));
                        else
                            mma_commit_pair(empty(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every MMA has completed before TMEM is freed
            if (leader) {
                if constexpr (CG == 1)
                    mma_commit(mma_done);
                else
                    mma_commit_pair(mma_done, 0x1);
            }
            __syncwarp();
            wait_drain(mma_done, 0, abort_flag, p);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales
        // Asynchronous copies, completing on the chunk's barrier: nothing here waits for
        // global memory, and the promotion warps' K loop holds no global load (in it, a
        // load's latency of some 1000 cycles showed through a distance of two K blocks).
        // The loop is kept small: a warp that shares its scheduler with two promotion warps
        // slows them by what it pushes out of the instruction cache.
        uint32_t chunk = 0;
        bool alive = true;
        for (int32_t u = first; u < num_units && alive; u += step) {
            const Fp8Unit w = fp8_unit<C>(u, p, prefix);
            // four scales a copy where they lie next to each other on a 16-byte boundary
            const int32_t row0 = w.row0 + static_cast<int32_t>(rank) * C::BM;
            const bool vec_a = p.sa_vec && (row0 & 3) == 0, vec_b = ROWS && p.sb_vec;
            const int32_t row = row0 + (vec_a ? 4 : 1) * lane;  // this lane's first row
            // bytes of rows and columns that exist, from those left in the tile (times four they stay in 32 bits)
            const int32_t row_left = min(w.row_end - row0, C::BM), col_left = min(p.N - w.col0, BN);
            const int32_t a_bytes = max(0, min(16, 4 * (row_left - 4 * lane)));
            const float *pa = p.sa + (row < w.row_end ? static_cast<int64_t>(row) * p.sa_row : 0) + kb0 * p.sa_blk;
            // this lane's first column (ROWS) or block of columns
            const int32_t n = w.col0 + (ROWS ? (vec_b ? 4 : 1) : kScaleBlock) * lane;
            const bool has_b = ROWS || lane < BN / 128;
            const float *pb = p.sb + w.group * p.sb_group + static_cast<int64_t>(ROWS ? n : n / kScaleBlock) * p.sb_n + kb0 * p.sb_k;
            for (int32_t kb = 0; kb < num_kb; ++kb) {
                const uint32_t buf = chunk % C::CHUNKS;
                if (kb % C::CHUNK == 0) {
                    const bool ok = wait_phase(sempty(buf), ((chunk / C::CHUNKS) & 1u) ^ 1u, abort_flag, p, WAIT_SCALES);
                    if (!__all_sync(0xffffffffu, ok)) {
                        alive = false;
                        break;
                    }
                }
                const uint32_t at = s_scale + buf * C::CHUNK_BYTES + (kb % C::CHUNK) * (C::KB_SCALES * 4);
                if (vec_a) {
                    copy_async_16(at + 16 * lane, pa, a_bytes);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        copy_async_f32(at + 4 * lane + 128 * i, row + 32 * i < w.row_end ? pa + 32 * i * p.sa_row : p.sa,
                                       row + 32 * i < w.row_end);
                }
                pa += p.sa_blk;
                if constexpr (ROWS) {
                    if (vec_b) {
#pragma unroll
                        for (int i = 0; i < BN / 128; ++i)
                            copy_async_16(at + 512 + 512 * i + 16 * lane, n + 128 * i < p.N ? pb + 128 * i : p.sb,
                                          max(0, min(16, 4 * (col_left - 4 * lane - 128 * i))));
                    } else {
#pragma unroll
                        for (int i = 0; i < BN / 32; ++i)
                            copy_async_f32(at + 512 + 4 * lane + 128 * i, n + 32 * i < p.N ? pb + 32 * i * p.sb_n : p.sb,
                                           n + 32 * i < p.N);
                    }
                } else if (has_b) {
                    copy_async_f32(at + 512 + 4 * lane, n < p.N ? pb : p.sb, n < p.N);
                }
                pb += p.sb_k;
                if (kb % C::CHUNK == C::CHUNK - 1 || kb + 1 == num_kb) {
                    copy_async_arrive(sfull(buf));
                    ++chunk;
                }
            }
        }
        copy_async_wait();
        __syncwarp();
    }
    } else {
        // ------------------------------------------- promotion and epilogue
        if constexpr (C::SHIFT_REGS) regs_inc<C::EPI_REGS>();
        const int j = warp - kRoleWarps;
        const int q = j & 3, h = j >> 2;
        const uint32_t stg = s_epi + static_cast<uint32_t>(j) * (C::EPI_BUFS * C::EPI_BUF);
        const uint64_t store_policy = policy_evict_first();
        // slots of this warp: count s of its K blocks since the start gives slot and phase
        uint32_t count = C::H == 2 ? h : 0, chunk = 0;
        bool alive = true;
        for (int32_t u = first; u < num_units && alive; u += step) {
            const Fp8Unit w = fp8_unit<C>(u, p, prefix);
            const int32_t row0 = w.row0 + static_cast<int32_t>(rank) * C::BM + 32 * q;
            const int32_t col0 = w.col0 + C::seg_col(h, 0);
            const bool work = row0 < w.row_end && col0 < p.N;  // otherwise only the barriers are served
            // on a pair a slot's two segments lie in two scale blocks, else in one
            constexpr int NB = !ROWS && C::H == 2 && CG == 2 ? 2 : 1;
            uint64_t sum[C::COLS / 2];
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) sum[i] = 0ull;
            for (int32_t kb = 0; kb < num_kb; ++kb) {
                if (kb % C::CHUNK == 0) {
                    const bool ok = wait_lean(sfull(chunk % C::CHUNKS), (chunk / C::CHUNKS) & 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) {
                        alive = false;
                        break;
                    }
                }
                const uint32_t sc_at = s_scale + (chunk % C::CHUNKS) * C::CHUNK_BYTES + (kb % C::CHUNK) * (C::KB_SCALES * 4);
                const float row_scale = ld_shared_f32(sc_at + (32 * q + lane) * 4);
                uint64_t s2[2];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int blk = NB == 2 ? i : (BN == 256 ? h : 0);
                    const float f = ROWS ? row_scale : row_scale * ld_shared_f32(sc_at + 512 + 4 * blk);
                    s2[i] = pair_f32(f, f);
                }
                // the chunk is read: back to the scale warp
                auto chunk_done = [&] {
                    if (kb % C::CHUNK == C::CHUNK - 1 || kb + 1 == num_kb) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sempty(chunk % C::CHUNKS));
                        ++chunk;
                    }
                };
                if (!ROWS || !work) chunk_done();
                const uint32_t slot = count % C::SLOTS;
                const bool ok = wait_lean(tfull(slot), (count / C::SLOTS) & 1u, abort_flag);
                count += C::H;
                if (!__all_sync(0xffffffffu, ok)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                // the slot is read: back to the MMA issuer
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 1)
                            mbar_arrive(tempty(slot));
                        else
                            mbar_arrive_cluster(mapa(tempty(slot), 0));
                    }
                };
                if (!work) {
                    release();
                    continue;
                }
                const uint32_t taddr =
                    tmem_base + (static_cast<uint32_t>(32 * q) << 16) + slot * SC + (C::H == 1 ? C::COLS * h : 0);
                // ROWS: the scales of sixteen columns, read sixteen columns ahead
                uint64_t cs[2][8];
                auto load_cols = [&](int g) {
                    if constexpr (ROWS) {
                        if (g < C::COLS / 16) {
                            const uint32_t at = sc_at + 512 + (C::seg_col(h, g / 4) + 16 * (g % 4)) * 4;
#pragma unroll
                            for (int i = 0; i < 4; ++i) ld_shared_v2u64(at + 16 * i, cs[g & 1][2 * i], cs[g & 1][2 * i + 1]);
                        }
                    }
                };
                load_cols(0);
                constexpr int NC = C::COLS / C::LD;
                uint32_t v[C::PIPE ? 2 : 1][C::LD];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (!C::PIPE || c == 0) tmem_ld(taddr + C::LD * c, v[0]);
                    tmem_ld_wait();
                    if (c + 1 == NC)
                        release();  // the slot's last columns are in registers
                    else if constexpr (C::PIPE)
                        tmem_ld(taddr + C::LD * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                    for (int g = 0; g < C::LD / 16; ++g) {
                        const int gg = C::LD / 16 * c + g;
                        load_cols(gg + 1);
                        if constexpr (ROWS) {
                            // the products first: each multiply-add waits for none of them
#pragma unroll
                            for (int i = 0; i < 8; ++i) cs[gg & 1][i] = mul2(cs[gg & 1][i], s2[0]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t *const at = v[C::PIPE ? c & 1 : 0] + 16 * g + 2 * i;
                            const uint64_t x = pair_u32(at[0], at[1]);
                            if constexpr (ROWS)
                                fma2(sum[8 * gg + i], x, cs[gg & 1][i]);
                            else
                                fma2(sum[8 * gg + i], x, s2[NB == 2 ? gg / 4 : 0]);
                        }
                    }
                }
                if (ROWS) chunk_done();
            }
            if (!alive || !work) continue;
            if constexpr (C::SPLIT) {
                if (p.split > 1) {
                    // the partial sums go to shared memory (the ring has been read), for the
                    // cluster's reduction below: four columns of a row per 16 bytes
#pragma unroll
                    for (int i = 0; i < C::COLS / 4; ++i) {
                        const int g = C::COLS / 4 * h + i, r = 32 * q + lane;
                        uint32_t x0, x1, x2, x3;
                        unpair(sum[2 * i], x0, x1);
                        unpair(sum[2 * i + 1], x2, x3);
                        st_shared_v4(s_a + partial_at(g, r), x0, x1, x2, x3);
                    }
                    continue;
                }
            }
            // Store the tile part through swizzled staging, in 128-byte wide subtiles: by TMA
            // where D's rows suit it, the subtile lies inside N (a store past a row's end writes
            // whole 16-byte units) and (grouped) the 32 rows are the group's own; else by the
            // warp, along the rows: 12639 x 3695 x 401 in 18 groups, bf16, 55 us.  (Each lane
            // storing its own row, a store touches the sectors of 32 rows: 453 us.)
            const bool tma = p.tma_store && (!GROUPED || row0 + 32 <= w.row_end);
            auto emit = [&](auto out_tag) {
                constexpr int OUT = decltype(out_tag)::value;
                constexpr int ESIZE = OUT == OUT_F32 ? 4 : 2, SUB = C::EPI_ROW / ESIZE;  // columns
                auto col_of = [&](int s) { return w.col0 + C::seg_col(h, s * SUB / 64) + s * SUB % 64; };
#pragma unroll
                for (int s0 = 0; s0 < C::COLS / SUB; s0 += C::EPI_BUFS) {
                    if (lane == 0) bulk_wait_read<0>();  // the stores that used the buffers have read them
                    __syncwarp();
#pragma unroll
                    for (int s = s0; s < s0 + C::EPI_BUFS; ++s) {
                        if (col_of(s) >= p.N) continue;
                        const uint64_t *const part = sum + s * SUB / 2;
                        uint32_t o[32];
#pragma unroll
                        for (int i = 0; i < SUB / 2; ++i) {
                            uint32_t lo, hi;
                            unpair(part[i], lo, hi);
                            if constexpr (OUT == OUT_F32) {
                                o[2 * i] = lo;
                                o[2 * i + 1] = hi;
                            } else {
                                o[i] = pack_bf16x2(lo, hi);
                            }
                        }
                        const uint32_t at = stg + (s - s0) * C::EPI_BUF + static_cast<uint32_t>(lane) * C::EPI_ROW;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            st_shared_v4(at + ((static_cast<uint32_t>(i) ^ (lane & 7u)) << 4), o[4 * i], o[4 * i + 1],
                                         o[4 * i + 2], o[4 * i + 3]);
                    }
                    if (tma) fence_proxy_async_smem();
                    __syncwarp();
                    if (tma && lane == 0) {
#pragma unroll
                        for (int s = s0; s < s0 + C::EPI_BUFS; ++s)
                            if (col_of(s) + SUB <= p.N)
                                tma_store_3d(&tmD, stg + (s - s0) * C::EPI_BUF, col_of(s), row0, 0, store_policy);
                        bulk_commit();
                    }
#pragma unroll
                    for (int s = s0; s < s0 + C::EPI_BUFS; ++s)
                        if (!tma || col_of(s) + SUB > p.N)
                            store_rows<ESIZE>(static_cast<char *>(p.D), row0, min(32, w.row_end - row0), col_of(s), p.N,
                                              p.ldd, p.store_bytes, stg + (s - s0) * C::EPI_BUF, lane);
                }
            };
            if (p.out == OUT_F32)
                emit(std::integral_constant<int, OUT_F32>{});
            else
                emit(std::integral_constant<int, OUT_BF16>{});
        }
        if (!alive && lane == 0 && !*abort_flag) {  // no other role gave up: the polls ran out
            report_timeout(p, WAIT_PROMOTION);
            *abort_flag = 1;
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    }

    if constexpr (C::SPLIT) {
        if (p.split > 1) {
            // Every CTA sums a share of the tile over the cluster's partial sums, in the
            // order of their K blocks, so results do not depend on timing.
            __syncwarp();
            cluster_sync();
            const Fp8Unit w = fp8_unit<C>(first, p, prefix);
            const int32_t rows = min(w.row_end - w.row0, C::BM);
            for (int32_t i = part * C::THREADS + static_cast<int32_t>(threadIdx.x); i < rows * (BN / 4);
                 i += p.split * C::THREADS) {
                const int32_t r = i / (BN / 4), g = i % (BN / 4);
                const int32_t col = w.col0 + 4 * g;
                if (col >= p.N) continue;
                float4 x[kMaxCluster];
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < p.split) x[c] = ld_cluster_f32x4(mapa(s_a + partial_at(g, r), c));
                float4 t = x[0];
#pragma unroll
                for (int c = 1; c < kMaxCluster; ++c)
                    if (c < p.split) {
                        t.x += x[c].x;
                        t.y += x[c].y;
                        t.z += x[c].z;
                        t.w += x[c].w;
                    }
                const int64_t at = static_cast<int64_t>(w.row0 + r) * p.ldd + col;
                const bool whole = p.store_bytes == 16 && col + 4 <= p.N;
                const float f[4] = {t.x, t.y, t.z, t.w};
                if (p.out == OUT_F32) {
                    float *dst = static_cast<float *>(p.D) + at;
                    if (whole) {
                        *reinterpret_cast<float4 *>(dst) = t;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (col + k < p.N) dst[k] = f[k];
                    }
                } else {
                    uint16_t *dst = static_cast<uint16_t *>(p.D) + at;
                    const uint2 o = make_uint2(pack_bf16x2(__float_as_uint(t.x), __float_as_uint(t.y)),
                                               pack_bf16x2(__float_as_uint(t.z), __float_as_uint(t.w)));
                    if (whole) {
                        *reinterpret_cast<uint2 *>(dst) = o;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (col + k < p.N) dst[k] = static_cast<uint16_t>((k < 2 ? o.x : o.y) >> (16 * (k & 1)));
                    }
                }
            }
            __syncwarp();
            cluster_sync();  // no CTA leaves while another reads its partial sums
        }
    }
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
}

}  // namespace ts
