// Products with a fused epilogue for sm_103a: a linear layer's forward and backward products and
// the products of an orthogonalised update.
//
//   D[z] = act(alpha * A[z] B[z]^T + bias) + beta * aux[z]        (forward; optionally the sum before act too)
//   D[z] = alpha * A[z] B[z]^T * act'(aux[z])                     (backward through the activation before)
//
// with 16-bit operands (bf16, or fp16 inside the library), fp32 accumulation in Tensor Memory and
// an epilogue in fp32.  Either operand may lie with K contiguous or with its rows of D contiguous:
// a layer's input gradient reads the weights, its weight gradient both operands, the other way
// around, in place.  With `sym` D is symmetric: the tiles on and above the diagonal are computed
// and those above it stored twice.
//
// The tensor core's additions cut towards zero instead of rounding: a sum that one CTA forms is off by some
// 1e-9 for each term (an fp32 gradient over 4096 rows by 4.4e-6 of its norm, over 1024 or by four CTAs
// 1.0e-6; rounded additions 2.5e-7 to 6e-7).  Bf16 results do not show it.  Sums moved to registers every few K
// blocks would round, for as many more reads of the accumulator.
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer of the operand ring
//   warp 1       TMEM allocator and MMA issuer
//   warp 3       initialises the barriers
//   warps 4..11  epilogue: warp 4 + j holds rows 32 * (j % 4) of the tile, one row per lane, and
//                half j / 4 of its columns, in subtiles of 128 bytes of D
//
// A 256-column tile may be used with fewer columns (LinParams::bn, a multiple of 16 above 128): the
// host picks the width whose tiles fill their waves of workers best.
//
// Two accumulators in TMEM: the epilogue of a tile overlaps the mainloop of the next.  The epilogue
// fetches aux by TMA into the staging buffer that the result leaves from: with two buffers a subtile
// ahead, over the end of a tile too, with one before it waits for the accumulator.  Bias comes a tile
// ahead, a column a lane.
//
// What bounds it: large products the tensor cores and, when they last, the card's power (8192 x 4096 x
// 8192 with bias and residual 290 us in a graph, 1.90 PFLOP/s; in a long series 340); K loops of up to
// some 1000 the epilogue, two of whose warps share a scheduler and wait for its instructions' latencies:
// 8192 x 4096 x 64 in bf16 15 us (the memory would take 10), with silu 26, in fp32 with a residual 46 (40).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "gemm_kernel.cuh"
#include "linear_params.h"
#include "ptx.cuh"
#include "waits.cuh"

namespace ts {

// A poll ordered over the cluster costs some 100 cycles more, in loops of 250 to 500.
template <>
constexpr bool kCtaScope<LinParams> = true;

template <int BN_, int CG_, int PRE_>
struct LinCfg {
    static constexpr int BN = BN_, CG = CG_, PRE = PRE_;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (kRoleWarps + EPI_WARPS);
    static constexpr int BM = 128, TILE_M = BM * CG;
    static constexpr int BK = 64, UMMA_K = 16;
    static constexpr int B_ROWS = BN / CG;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = B_ROWS * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES, TX_BYTES = STAGE_BYTES * CG;
    static constexpr int BOX_BYTES = 64 * BK * 2;  // operand with its rows contiguous: 64 of them by BK
    static constexpr int COLS = BN / 2;            // columns of an epilogue warp
    // Staging of a warp: one or two buffers of 32 rows x 128 bytes for D (and aux before it), and one
    // for the sum before the activation.  A buffer for all warps costs the ring a stage: two pay off
    // with short K loops alone, where the epilogue shows (see the host).  And 32 columns of bias.
    static constexpr int EPI_BUF = 32 * 128, MAX_BUFS = 2;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int BAR_BYTES = 512, BIAS_BYTES = EPI_WARPS * 128;
    static constexpr int MAX_STAGES = 8;
    static constexpr int smem_bytes(int stages, int bufs) {
        return 1024 + stages * STAGE_BYTES + EPI_WARPS * (bufs + PRE) * EPI_BUF + BIAS_BYTES + BAR_BYTES;
    }
    static constexpr int stages(int bufs) {
        const int n = (kSmemLimit - smem_bytes(0, bufs)) / STAGE_BYTES;
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
    static_assert((2 * MAX_STAGES + 5 + EPI_WARPS * MAX_BUFS) * 8 + 8 <= BAR_BYTES, "barrier region");
};

// Shared-memory descriptor of an operand tile with its rows (columns of D for B) contiguous: boxes
// of 64 of them by 64 of K, rows of 128 bytes along the first for consecutive k, 8-row atoms 1024
// bytes apart along K (stride byte offset), the next 64 rows in the next 8 KB box (leading byte
// offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t smem_addr) {
    return uint64_t((smem_addr & 0x3FFFFu) >> 4) | (uint64_t(8192 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ float f16_to_f32(uint16_t h) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
    return f;
}

// Byte b of staged row r: 16-byte units permuted within the row as the TMA's 128-byte swizzle does.
__device__ __forceinline__ uint32_t staged(uint32_t stage, int r, int b) {
    return stage + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15);
}

// A warp moves `rows` rows of `left` <= 128 bytes between global memory (pitch in bytes) and swizzled
// staging, lanes along the rows, in units of `unit` = 16, 4 or 2 bytes (the alignment of the rows; 16
// where `left` is a multiple too).  Where TMA cannot: a subtile that is cut off by N or by the tile's
// width, rows that start off 16-byte boundaries.
__device__ __forceinline__ void stage_rows_in(const char *src, int64_t pitch, int rows, int left, int unit,
                                              uint32_t stage, int lane) {
    if (unit == 16 && left % 16 == 0) {
        const int per = left / 16;
        for (int i = lane; i < rows * per; i += 32) {
            const int r = i / per, b = (i - r * per) * 16;
            const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(src + r * pitch + b));
            st_shared_v4(staged(stage, r, b), v.x, v.y, v.z, v.w);
        }
    } else if (unit >= 4) {
        const int b = lane * 4;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            uint32_t v = 0;
            if (b + 4 <= left)
                v = __ldcg(reinterpret_cast<const uint32_t *>(src + r * pitch + b));
            else if (b + 2 <= left)
                v = __ldcg(reinterpret_cast<const uint16_t *>(src + r * pitch + b));
            st_shared_u32(staged(stage, r, b), v);
        }
    } else {
        const int b = lane * 2;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint16_t v0 = b + 2 <= left ? __ldcg(reinterpret_cast<const uint16_t *>(src + r * pitch + b)) : 0;
            const uint16_t v1 = b + 66 <= left ? __ldcg(reinterpret_cast<const uint16_t *>(src + r * pitch + b + 64)) : 0;
            st_shared_u16(staged(stage, r, b), v0);
            st_shared_u16(staged(stage, r, b + 64), v1);
        }
    }
}
__device__ __forceinline__ void stage_rows_out(char *dst, int64_t pitch, int rows, int left, int unit, uint32_t stage,
                                               int lane) {
    if (unit == 16 && left % 16 == 0) {
        const int per = left / 16;
        for (int i = lane; i < rows * per; i += 32) {
            const int r = i / per, b = (i - r * per) * 16;
            *reinterpret_cast<uint4 *>(dst + r * pitch + b) = ld_shared_v4(staged(stage, r, b));
        }
    } else if (unit >= 4) {
        const int b = lane * 4;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint32_t v = ld_shared_u32(staged(stage, r, b));
            if (b + 4 <= left)
                *reinterpret_cast<uint32_t *>(dst + r * pitch + b) = v;
            else if (b + 2 <= left)
                *reinterpret_cast<uint16_t *>(dst + r * pitch + b) = static_cast<uint16_t>(v);
        }
    } else {
        const int b = lane * 2;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            const uint16_t v0 = ld_shared_u16(staged(stage, r, b)), v1 = ld_shared_u16(staged(stage, r, b + 64));
            if (b + 2 <= left) *reinterpret_cast<uint16_t *>(dst + r * pitch + b) = v0;
            if (b + 66 <= left) *reinterpret_cast<uint16_t *>(dst + r * pitch + b + 64) = v1;
        }
    }
}

struct LinUnit {
    int32_t mb, nb, z;  // tile and matrix
};

template <class C>
__device__ __forceinline__ LinUnit lin_unit(int32_t u, const LinParams &p) {
    LinUnit w;
    w.z = fast_div(u, p.div_matrix);
    const int32_t t = u - w.z * p.tiles_per_matrix;
    if (p.sym) {
        // rows i and n - 1 - i of the triangle together hold n + 1 tiles (the middle row alone, half)
        const int32_t n = p.tiles_n, i = fast_div(t, p.div_group_tiles), r = t - i * (n + 1);
        w.mb = r < n - i ? i : n - 1 - i;
        w.nb = r < n - i ? i + r : w.mb + (r - (n - i));
    } else {
        raster(t, p, w.mb, w.nb);
    }
    return w;
}

// OUT: type of D.  OUT_BF16 and OUT_F32 are a layer's products (alpha = beta = 1, aux and pre of D's type, not
// symmetric); OUT_F16 the iteration's: D fp16 or bf16 (p.out), aux fp16, without bias, activation and pre.
// One kernel for all of them is slower: what the epilogue's loop executes then comes from places far apart,
// and it waits for its instructions (8192 x 4096 x 64 in bf16 21.6 us, on its own 16.2).
template <int BN, int CG, int MODE, int OUT>
__global__ void __launch_bounds__(LinCfg<BN, CG, MODE == LIN_PRE>::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmAux,
                  const __grid_constant__ CUtensorMap tmPre, const __grid_constant__ LinParams p) {
    constexpr bool PRE = MODE == LIN_PRE;
    using C = LinCfg<BN, CG, PRE>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t stages = static_cast<uint32_t>(p.stages), bufs = static_cast<uint32_t>(p.bufs);
    const uint32_t s_a = base;
    const uint32_t s_b = s_a + stages * C::A_BYTES;
    const uint32_t s_epi = s_b + stages * C::B_BYTES;
    const uint32_t s_bias = s_epi + C::EPI_WARPS * (bufs + PRE) * C::EPI_BUF, s_bar = s_bias + C::BIAS_BYTES;
    auto full = [&](uint32_t s) { return s_bar + 8u * s; };
    auto empty = [&](uint32_t s) { return s_bar + 8u * (stages + s); };
    auto tfull = [&](uint32_t a) { return s_bar + 8u * (2 * stages + a); };
    auto tempty = [&](uint32_t a) { return s_bar + 8u * (2 * stages + 2 + a); };
    const uint32_t mma_done = s_bar + 8u * (2 * stages + 4);
    auto aux_full = [&](uint32_t j, uint32_t b) { return s_bar + 8u * (2 * stages + 5 + j * C::MAX_BUFS + b); };
    const uint32_t tail = s_bar + 8u * (2 * stages + 5 + C::EPI_WARPS * C::MAX_BUFS);
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(gbase + (tail - base));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(gbase + (tail - base) + 4);

    // uniform across the warp, and known to be: the role loops then run on uniform registers
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool tma_d = p.store_bytes == 16;

    if (warp == 0 && lane == 0 && p.num_kb > 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 3 && lane == 0) {
        for (uint32_t s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull(a), 1);
            mbar_init(tempty(a), C::EPI_WARPS * CG);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < C::EPI_WARPS * C::MAX_BUFS; ++i) mbar_init(aux_full(0, i), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(tail, C::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_wait();
    grid_dep_launch();
    const int32_t first = static_cast<int32_t>(blockIdx.x) / CG;
    const int32_t step = static_cast<int32_t>(gridDim.x) / CG;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const bool leader = elect_one();
        uint32_t stage = 0, phase = 0, issued = 0;
        bool alive = true;
        for (int32_t u = first; u < p.num_units && alive; u += step) {
            const LinUnit w = lin_unit<C>(u, p);
            const int32_t a_row = w.mb * C::TILE_M + static_cast<int32_t>(rank) * C::BM;
            const int32_t b_row = w.nb * p.bn + static_cast<int32_t>(rank) * (p.bn / CG);
            for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                if (!wait_phase(empty(stage), phase ^ 1u, abort_flag, p, WAIT_PRODUCER_EMPTY)) {
                    alive = false;
                    break;
                }
                if (rank == 0 && leader) mbar_arrive_expect_tx(full(stage), p.tx_bytes);
                const uint32_t fb = CG == 2 ? mapa(full(stage), 0) : full(stage);
                auto load = [&](uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y) {
                    if constexpr (CG == 1)
                        tma_load_3d(dst, m, fb, x, y, w.z);
                    else
                        tma_load_3d_pair(dst, m, fb, x, y, w.z);
                };
                if (leader) {
                    const uint32_t da = s_a + stage * C::A_BYTES, db = s_b + stage * C::B_BYTES;
                    const int32_t k = kb * C::BK;
                    if (p.a_mn) {
#pragma unroll
                        for (int c = 0; c < C::BM / 64; ++c) load(da + c * C::BOX_BYTES, &tmA, a_row + 64 * c, k);
                    } else {
                        load(da, &tmA, k, a_row);
                    }
                    if (p.b_mn) {
#pragma unroll
                        for (int c = 0; c < C::B_ROWS / 64; ++c)
                            if (64 * c * CG < p.bn) load(db + c * C::BOX_BYTES, &tmB, b_row + 64 * c, k);
                    } else {
                        load(db, &tmB, k, b_row);
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every load has landed (seen on the even CTA's barriers) and every stage is released
        if (rank == 0) {
            const uint32_t n = issued < stages ? issued : stages;
            for (uint32_t i = 1; i <= n; ++i) {
                const uint32_t b = issued - i;
                wait_drain(full(b % stages), (b / stages) & 1u, abort_flag, p);
            }
        }
        for (uint32_t i = 0; i < stages; ++i) {
            if (!wait_drain(empty(stage), phase ^ 1u, abort_flag, p)) break;
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        // The whole warp runs the loop, one elected lane issues.
        if (rank == 0) {
            const bool leader = elect_one();
            const uint32_t idesc = p.idesc | (uint32_t(p.bn >> 3) << 17) | (uint32_t((C::BM * CG) >> 4) << 24);
            // steps of a start address for K = 16, in 16-byte units: 32 bytes along a K-major row, or
            // 16 rows of 128 bytes
            const uint32_t a_step = p.a_mn ? (16 * 128) >> 4 : 32 >> 4, b_step = p.b_mn ? (16 * 128) >> 4 : 32 >> 4;
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool alive = true;
            for (int32_t u = first; u < p.num_units && alive; u += step) {
                if (!wait_phase(tempty(acc), acc_phase ^ 1u, abort_flag, p, WAIT_MMA_TMEM_EMPTY)) break;
                tc_fence_after();
                for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_phase(full(stage), phase, abort_flag, p, WAIT_MMA_FULL)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
                    if (leader) {
                        const uint32_t at_a = s_a + stage * C::A_BYTES, at_b = s_b + stage * C::B_BYTES;
                        const uint64_t da = p.a_mn ? sw128_mn_desc(at_a) : sw128_kmajor_desc(at_a);
                        const uint64_t db = p.b_mn ? sw128_mn_desc(at_b) : sw128_kmajor_desc(at_b);
#pragma unroll
                        for (int kk = 0; kk < C::BK / C::UMMA_K; ++kk)
                            mma_bf16<CG>(tmem_base + acc * BN, da + a_step * kk, db + b_step * kk, idesc,
                                         kb != 0 || kk != 0);
                        if constexpr (CG == 1)
                            mma_commit(empty(stage));
                        else
                            mma_commit_pair(empty(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!alive) break;
                if (leader) {
                    if constexpr (CG == 1)
                        mma_commit(tfull(acc));
                    else
                        mma_commit_pair(tfull(acc), 0x3);
                }
                __syncwarp();
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
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
    } else if (warp >= kRoleWarps) {
        // --------------------------------------------------------- epilogue
        const int j = warp - kRoleWarps;
        const int q = j & 3, h = j >> 2;
        const uint32_t stg = s_epi + static_cast<uint32_t>(j) * (bufs + PRE) * C::EPI_BUF;
        const uint32_t stg_pre = stg + bufs * C::EPI_BUF;
        constexpr bool f32 = OUT == OUT_F32, iteration = OUT == OUT_F16, full = MODE == LIN_FULL || PRE;
        constexpr int sub = f32 ? 32 : 64, esize = f32 ? 4 : 2;
        const int cols = h ? p.bn - C::COLS : C::COLS;  // of this warp (of the kernel's tile the host may use fewer)
        const bool aux_tma = p.aux != nullptr && tma_d;
        // until the store that last used the next buffer has read it
        auto wait_store = [&] {
            if (bufs == 1)
                bulk_wait_read<0>();
            else
                bulk_wait_read<1>();
        };
        uint32_t acc = 0, acc_phase = 0, aux_phase = 0;  // aux_phase: bit b, parity of buffer b's next load
        uint32_t aux_pending = 0;                        // bit b: a load into buffer b has not been waited for
        bool alive = true;
        // The bias of a tile's columns, one of every 32 for a lane, fetched a tile ahead: a tile's columns are
        // seldom those of the tile before, and the fetch comes from L2.
        constexpr int CHUNKS = C::COLS / 32;
        float bias[CHUNKS];
        const uint32_t bias_at = s_bias + 128 * j;
        auto fetch_bias = [&](int32_t u) {
            const int32_t c0 = u < p.num_units ? lin_unit<C>(u, p).nb * p.bn + C::COLS * h + lane : p.N;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i)
                bias[i] = c0 + 32 * i >= p.N ? 0.f
                          : p.bias_f32       ? __ldg(static_cast<const float *>(p.bias) + c0 + 32 * i)
                                             : __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t *>(p.bias) + c0 + 32 * i)) << 16);
        };
        if (full && p.bias) fetch_bias(first);
        // Where this warp's subtiles lie.
        struct Place {
            int32_t row0, col0, col_end, z;
            bool work;
        };
        auto place = [&](int32_t u) {
            const LinUnit w = lin_unit<C>(u, p);
            Place t;
            t.row0 = w.mb * C::TILE_M + static_cast<int32_t>(rank) * C::BM + 32 * q;
            t.col0 = w.nb * p.bn + C::COLS * h;
            t.col_end = min(t.col0 + cols, p.N);
            t.z = w.z;
            t.work = t.row0 < p.M && t.col0 < t.col_end;
            return t;
        };
        // aux by TMA: one subtile's load into a free buffer
        auto load_aux = [&](uint32_t b, int32_t col, int32_t row, int32_t z) {
            if (lane == 0) {
                mbar_arrive_expect_tx(aux_full(j, b), C::EPI_BUF);
                tma_load_3d(stg + b * C::EPI_BUF, &tmAux, aux_full(j, b), col, row, z);
            }
            aux_pending |= 1u << b;
        };
        // With two buffers aux is loaded a subtile ahead, over the end of a tile too.
        const bool ahead = aux_tma && bufs == 2;
        int32_t next_u = first, next_col = 0;
        Place next;
        auto next_tile = [&] {
            for (; next_u < p.num_units; next_u += step) {
                next = place(next_u);
                next_col = next.col0;
                if (next.work) break;
            }
        };
        auto load_next = [&](uint32_t b) {
            if (next_u >= p.num_units) return;
            load_aux(b, next_col, next.row0, next.z);
            if ((next_col += sub) >= next.col_end) {
                next_u += step;
                next_tile();
            }
        };
        if (ahead) {
            next_tile();
            load_next(0);
        }
        uint32_t buf = 0;  // of the subtile
        auto tiles = [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            for (int32_t u = first; u < p.num_units && alive; u += step) {
                const LinUnit w = lin_unit<C>(u, p);
                const Place t = place(u);
                const int32_t row0 = t.row0, col0 = t.col0, col_end = t.col_end;
                const bool work = t.work;
                if (work && aux_tma && !ahead) {
                    __syncwarp();  // all lanes have stored what the last tile left in the buffer
                    if (lane == 0) {
                        bulk_wait_read<0>();  // the store that used the buffer has read it
                        fence_proxy_async_smem();
                    }
                    load_aux(0, col0, row0, w.z);
                    __syncwarp();
                }
                int ok = 1;
                if (lane == 0) ok = wait_long(tfull(acc), acc_phase, abort_flag, p, WAIT_EPI_TMEM_FULL);
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * BN + C::COLS * h;
                // the accumulator is read: back to the MMA issuer
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 1)
                            mbar_arrive(tempty(acc));
                        else
                            mbar_arrive_cluster(mapa(tempty(acc), 0));
                    }
                };
                if (!work) release();
                const int rows = min(32, p.M - row0);
                float bias_now[CHUNKS];
                if (full && p.bias) {
#pragma unroll
                    for (int i = 0; i < CHUNKS; ++i) bias_now[i] = bias[i];
                    fetch_bias(u + step);
                }
                // a subtile at a time
#pragma unroll 1
                for (int32_t col = col0; work && col < col_end; col += sub, buf ^= bufs - 1) {
                    const uint32_t at = stg + buf * C::EPI_BUF;
                    const int left = min(col_end - col, sub) * esize;
                    const bool tma = tma_d && left == 128;
                    // its buffer: free, or holding aux
                    if (aux_tma) {
                        if (!ahead && col > col0) {
                            __syncwarp();
                            if (lane == 0) {
                                bulk_wait_read<0>();
                                fence_proxy_async_smem();
                            }
                            load_aux(buf, col, row0, w.z);
                        }
                        const bool got = wait_phase(aux_full(j, buf), (aux_phase >> buf) & 1u, abort_flag, p, WAIT_AUX);
                        if (!__all_sync(0xffffffffu, got)) {
                            alive = false;
                            break;
                        }
                        aux_phase ^= 1u << buf;
                        aux_pending &= ~(1u << buf);
                    } else {
                        if (lane == 0) wait_store();
                        __syncwarp();
                        if (p.aux) {
                            stage_rows_in(static_cast<const char *>(p.aux) +
                                              (w.z * p.aux_matrix + static_cast<int64_t>(row0) * p.ld_aux + col) * esize,
                                          p.ld_aux * esize, rows, left, p.store_bytes, at, lane);
                            __syncwarp();
                        }
                    }
                    if (PRE && aux_tma) {
                        if (lane == 0) wait_store();  // the last store of pre has read its buffer
                        __syncwarp();
                    }
                    // 32 columns at a time: a subtile of fp32, half of a 16-bit one
#pragma unroll 1
                    for (int32_t c0 = col, piece = 0; c0 < min(col + sub, col_end); c0 += 32, piece += 4) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(taddr + (c0 - col0), v);
                        if (full && p.bias) {
                            float b = bias_now[0];
#pragma unroll
                            for (int i = 1; i < CHUNKS; ++i) b = c0 - col0 == 32 * i ? bias_now[i] : b;
                            __syncwarp();  // the last chunk's have been read
                            st_shared_f32(bias_at + 4 * lane, b);
                            __syncwarp();
                        }
                        tmem_ld_wait();
                        if (c0 + 32 >= col_end) release();
                        float x[32];
                        if (p.num_kb > 0) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                x[i] = __uint_as_float(v[i]), x[i + 1] = __uint_as_float(v[i + 1]);
                                if constexpr (iteration) split(two(p.alpha) * two(x[i], x[i + 1]), x[i], x[i + 1]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = 0.f;
                        }
                        if (full && p.bias) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {  // the same address in all lanes
                                const uint4 b = ld_shared_v4(bias_at + 16 * i);
                                split(two(x[4 * i], x[4 * i + 1]) + two(__uint_as_float(b.x), __uint_as_float(b.y)), x[4 * i], x[4 * i + 1]);
                                split(two(x[4 * i + 2], x[4 * i + 3]) + two(__uint_as_float(b.z), __uint_as_float(b.w)), x[4 * i + 2], x[4 * i + 3]);
                            }
                        }
                        // x into this lane's row of a staging buffer
                        auto put = [&](uint32_t buffer) {
                            const uint32_t row_at = buffer + lane * 128;
                            if constexpr (f32) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    st_shared_v4(row_at + ((i ^ (lane & 7)) << 4), __float_as_uint(x[4 * i]),
                                                 __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                                                 __float_as_uint(x[4 * i + 3]));
                            } else {
                                uint32_t o[16];
                                if (iteration && p.out == OUT_F16) {
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        o[i] = pack_f16x2(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]));
                                } else {
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        o[i] = pack_bf16x2(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]));
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    st_shared_v4(row_at + (((piece + i) ^ (lane & 7)) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2],
                                                 o[4 * i + 3]);
                                if (iteration && p.sym && w.nb > w.mb) {
                                    // The entry's mirror image: a column of this warp's is 32 consecutive values
                                    // there.  Lanes 2i and 2i + 1 exchange halves, so that an even lane holds two rows
                                    // of an even column, an odd one of the column behind it, and stores them at once.
                                    const int32_t r = row0 + (lane & ~1), cm = c0 + (lane & 1);
                                    uint16_t *m = static_cast<uint16_t *>(p.D) + w.z * p.d_matrix + cm * p.ldd + r;
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const uint32_t got = __shfl_xor_sync(0xffffffffu, o[i], 1);
                                        const uint32_t both = lane & 1 ? __byte_perm(got, o[i], 0x7632) : __byte_perm(o[i], got, 0x5410);
                                        // rows of the mirror image: D, of a multiple of eight rows and columns, is square
                                        if (cm + 2 * i < p.N && r < p.M) *reinterpret_cast<uint32_t *>(m) = both;
                                        m += 2 * p.ldd;
                                    }
                                }
                            }
                        };
                        if constexpr (PRE) put(stg_pre);
                        float a[32];
                        if (p.aux) {
                            const uint32_t row_at = at + lane * 128;
                            if constexpr (f32) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint4 t = ld_shared_v4(row_at + ((i ^ (lane & 7)) << 4));
                                    a[4 * i] = __uint_as_float(t.x);
                                    a[4 * i + 1] = __uint_as_float(t.y);
                                    a[4 * i + 2] = __uint_as_float(t.z);
                                    a[4 * i + 3] = __uint_as_float(t.w);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint4 t = ld_shared_v4(row_at + (((piece + i) ^ (lane & 7)) << 4));
                                    const uint32_t w4[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        a[8 * i + 2 * e] = iteration ? f16_to_f32(static_cast<uint16_t>(w4[e])) : __uint_as_float(w4[e] << 16);
                                        a[8 * i + 2 * e + 1] = iteration ? f16_to_f32(static_cast<uint16_t>(w4[e] >> 16))
                                                                         : __uint_as_float(w4[e] & 0xffff0000u);
                                    }
                                }
                            }
                            if (ahead && c0 == col) {
                                // the other buffer: all lanes, or the store before this one, have read it
                                __syncwarp();
                                if (lane == 0) {
                                    bulk_wait_read<0>();
                                    fence_proxy_async_smem();
                                }
                                load_next(buf ^ 1u);
                            }
                        }
                        if constexpr (MODE == LIN_SLOPE) {
                            apply_slope<ACT>(x, a);
                        } else {
                            apply_act<ACT>(x);
                            if (p.aux) {
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    if constexpr (iteration)
                                        split(fma(two(p.beta), two(a[i], a[i + 1]), two(x[i], x[i + 1])), x[i], x[i + 1]);
                                    else
                                        split(two(a[i], a[i + 1]) + two(x[i], x[i + 1]), x[i], x[i + 1]);
                                }
                            }
                        }
                        put(at);
                    }
                    // the staged subtiles leave
                    auto leave = [&](uint32_t buffer, const CUtensorMap *map, void *dst, int64_t matrix, int64_t ld) {
                        if (tma) {
                            tma_store_3d(map, buffer, col, row0, w.z, policy_evict_first());
                        } else {
                            stage_rows_out(static_cast<char *>(dst) +
                                               (w.z * matrix + static_cast<int64_t>(row0) * ld + col) * esize,
                                           ld * esize, rows, left, p.store_bytes, buffer, lane);
                        }
                    };
                    if (tma) fence_proxy_async_smem();
                    __syncwarp();
                    if constexpr (PRE) {
                        if (!tma || lane == 0) leave(stg_pre, &tmPre, p.pre, 0, p.ld_pre);
                        if (lane == 0) bulk_commit();
                    }
                    if (!tma || lane == 0) leave(at, &tmD, p.D, p.d_matrix, p.ldd);
                    if (lane == 0) bulk_commit();
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        };
        // a loop for each activation, so that a tile's instructions lie together
        if constexpr (MODE == LIN_BARE)
            tiles(ActTag<ACT_NONE>{});
        else
            with_act(p.act, tiles);
        // loads of aux that a given-up wait left in flight
        for (uint32_t b = 0; b < bufs; ++b)
            if ((aux_pending >> b) & 1u) wait_drain(aux_full(j, b), (aux_phase >> b) & 1u, abort_flag, p);
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
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
