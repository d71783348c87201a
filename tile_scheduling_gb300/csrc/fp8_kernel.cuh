// Block-scaled 8-bit product for sm_103a, plain and grouped by rows:
//
//   D[m][n] = sum over K blocks b of  SA[m][b] * SB[n][b] * sum_{k in b} A[m][k] * B[n][k]
//
// with 8-bit operands (e4m3 or e5m2) and one fp32 scale for each row of A and
// 128 elements of K, and for each 128 x 128 block (or each row) of B.
//
// The scales change every 128 elements of K, so the tensor core cannot carry one
// accumulator through the K loop.  Each K block is a chain of four MMAs (K = 32
// each) into one of two TMEM accumulators; promotion warps read it back, scale
// it, and add it to fp32 registers that hold the tile's running sum, while the
// MMAs of the next K block fill the other accumulator.
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer of the operand ring
//   warp 1       TMEM allocator and MMA issuer
//   warp 3       barrier initialisation
//   warps 4..11  promotion and epilogue: warp 4 + j holds rows 32 * (j % 4) and the
//                column half j / 4 of the tile, one row per lane
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

template <int BN_, int CG_, bool ROWS_, bool GROUPED_>
struct Fp8Cfg {
    static constexpr int BN = BN_, CG = CG_;
    static constexpr bool ROWS = ROWS_, GROUPED = GROUPED_;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (kRoleWarps + EPI_WARPS);
    static constexpr int BM = 128, TILE_M = BM * CG;
    static constexpr int BK = kScaleBlock;  // one scale block: a 128-byte swizzle row
    static constexpr int UMMA_K = 32;
    static constexpr int B_ROWS = BN / CG;
    static constexpr int A_BYTES = BM * BK;
    static constexpr int B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int TX_BYTES = STAGE_BYTES * CG;
    static constexpr int COLS = BN / 2;  // columns of one promotion warp
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int EPI_BUF = 32 * 128;  // store staging of one warp: 32 rows x 128 bytes
    static constexpr int EPI_BYTES = EPI_WARPS * EPI_BUF;
    static constexpr int SCALE_BYTES = ROWS ? EPI_WARPS * 2 * COLS * 4 : 0;  // a warp's column scales, two K blocks
    static constexpr int PREFIX_BYTES = GROUPED ? (kMaxExperts + 8) * 4 : 0;
    static constexpr int BAR_BYTES = 256;
    static constexpr int FIXED_BYTES = 1024 + EPI_BYTES + SCALE_BYTES + PREFIX_BYTES + BAR_BYTES;
    static constexpr int STAGES = (kSmemLimit - FIXED_BYTES) / STAGE_BYTES;
    static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * STAGE_BYTES;
    static_assert(STAGES >= 2, "ring too shallow");
    static_assert((2 * STAGES + 5) * 8 + 16 <= BAR_BYTES, "barrier region");
};

// Shared-memory descriptor of a B tile whose rows run along N (B is [K][N]): rows of
// 128 bytes (128 values of n) for consecutive k, 8-row atoms 1024 bytes apart along
// K (stride byte offset), the next 128 values of n in the next 16 KB box (leading
// byte offset).
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t smem_addr) {
    return uint64_t((smem_addr & 0x3FFFFu) >> 4) | (uint64_t(16384 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// One work unit: an output tile.
struct Fp8Unit {
    int32_t row0, row_end;  // rows [row0, row_end) of D may be written (row_end: the group's or D's last + 1)
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
        w.row_end = static_cast<int32_t>(r1);
        w.col0 = nb * C::BN;
    } else {
        int32_t mb, nb;
        raster(u, p, mb, nb);
        w.group = 0;
        w.row0 = mb * C::TILE_M;
        w.row_end = p.M;
        w.col0 = nb * C::BN;
    }
    return w;
}

template <int BN, int CG, bool ROWS, bool GROUPED>
__global__ void __launch_bounds__(384, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const __grid_constant__ Fp8Params p) {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED>;
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
    auto tempty = [&](uint32_t a) { return s_bar + 8u * (2 * C::STAGES + 2 + a); };
    const uint32_t mma_done = s_bar + 8u * (2 * C::STAGES + 4);
    const uint32_t tail = s_bar + 8u * (2 * C::STAGES + 5);
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(gbase + (tail - base));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(gbase + (tail - base) + 4);

    const int warp = threadIdx.x >> 5;
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
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull(a), 1);
            mbar_init(tempty(a), C::EPI_WARPS * CG);
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
        // Units per group, then their running sum (warp 2, 32 groups at a time).
        for (int32_t g = threadIdx.x; g < p.groups; g += C::THREADS) {
            int64_t lo, hi;
            if (!group_rows(p, g, lo, hi) && blockIdx.x == 0) report_group(p, g);
            prefix[g + 1] = static_cast<int32_t>((hi - lo + C::TILE_M - 1) / C::TILE_M) * p.tiles_n;
        }
        if (threadIdx.x == 0) prefix[0] = 0;
        __syncthreads();
        if (warp == 2) {
            int32_t run = 0;
            for (int32_t g0 = 0; g0 < p.groups; g0 += 32) {
                const int32_t g = g0 + lane;
                int32_t v = g < p.groups ? prefix[g + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += o;
                }
                if (g < p.groups) prefix[g + 1] = run + v;
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
    const int32_t first = static_cast<int32_t>(blockIdx.x) / CG;
    const int32_t step = static_cast<int32_t>(gridDim.x) / CG;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            bool alive = true;
            for (int32_t u = first; u < num_units && alive; u += step) {
                const Fp8Unit w = fp8_unit<C>(u, p, prefix);
                const int32_t a_row = w.row0 + static_cast<int32_t>(rank) * C::BM;
                const int32_t b_row = w.col0 + static_cast<int32_t>(rank) * C::B_ROWS;
                for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_phase(empty(stage), phase ^ 1u, abort_flag, p, WAIT_PRODUCER_EMPTY)) {
                        alive = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(full(stage), C::TX_BYTES);
                    const uint32_t da = s_a + stage * C::A_BYTES;
                    const uint32_t db = s_b + stage * C::B_BYTES;
                    const uint32_t fb = CG == 2 ? mapa(full(stage), 0) : full(stage);
                    const int32_t k = kb * C::BK;
                    auto load_b = [&](uint32_t dst, int32_t x, int32_t y) {
                        if constexpr (CG == 1)
                            tma_load_3d(dst, &tmB, fb, x, y, w.group);
                        else
                            tma_load_3d_pair(dst, &tmB, fb, x, y, w.group);
                    };
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
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = p.idesc | (uint32_t(BN >> 3) << 17) | (uint32_t(C::TILE_M >> 4) << 24);
            // start-address step (in 16-byte units) of one K = 32 MMA: 32 bytes along a
            // K-major row, or 32 rows of 128 bytes
            const uint32_t b_step = p.trans_b ? (32 * 128) >> 4 : 32 >> 4;
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool alive = true;
            for (int32_t u = first; u < num_units && alive; u += step) {
                for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_phase(tempty(acc), acc_phase ^ 1u, abort_flag, p, WAIT_MMA_TMEM_EMPTY) ||
                        !wait_phase(full(stage), phase, abort_flag, p, WAIT_MMA_FULL)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = sw128_kmajor_desc(s_a + stage * C::A_BYTES);
                    const uint32_t b_at = s_b + stage * C::B_BYTES;
                    const uint64_t db = p.trans_b ? sw128_nmajor_desc(b_at) : sw128_kmajor_desc(b_at);
#pragma unroll
                    for (int kk = 0; kk < C::BK / C::UMMA_K; ++kk)
                        mma_f8<CG>(tmem_base + acc * BN, da + 2u * kk, db + b_step * kk, idesc, kk != 0);
                    if constexpr (CG == 1) {
                        mma_commit(empty(stage));
                        mma_commit(tfull(acc));
                    } else {
                        mma_commit_pair(empty(stage), 0x3);
                        mma_commit_pair(tfull(acc), 0x3);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            }
            // every MMA has completed before TMEM is freed
            if constexpr (CG == 1)
                mma_commit(mma_done);
            else
                mma_commit_pair(mma_done, 0x1);
            wait_drain(mma_done, 0, abort_flag, p);
        }
        __syncwarp();
    } else if (warp >= kRoleWarps) {
        // ------------------------------------------- promotion and epilogue
        const int j = warp - kRoleWarps;
        const int q = j & 3, h = j >> 2;
        const uint32_t stg = s_epi + static_cast<uint32_t>(j) * C::EPI_BUF;
        const uint32_t wsc = s_scale + static_cast<uint32_t>(j) * (2 * C::COLS * 4);
        const uint64_t store_policy = policy_evict_first();
        uint32_t acc_i = 0, acc_phase = 0;
        bool alive = true;
        for (int32_t u = first; u < num_units && alive; u += step) {
            const Fp8Unit w = fp8_unit<C>(u, p, prefix);
            const int32_t row0 = w.row0 + static_cast<int32_t>(rank) * C::BM + 32 * q;
            const int32_t row = row0 + lane;
            const int32_t col0 = w.col0 + h * C::COLS;
            const bool work = row0 < w.row_end && col0 < p.N;  // otherwise only the barriers are served
            const bool mine = work && row < w.row_end;
            const float *const sa = p.sa + static_cast<int64_t>(row) * p.sa_row;
            const float *const sb = p.sb + w.group * p.sb_group + (ROWS ? 0 : (col0 / kScaleBlock) * p.sb_n);
            // Scales are read two K blocks ahead: their latency (an L2 hit) is about that long.
            auto load_a = [&](int32_t kb) { return mine && kb < p.num_kb ? __ldg(sa + kb * p.sa_blk) : 0.f; };
            auto load_b = [&](int32_t kb) {
                return !ROWS && mine && kb < p.num_kb ? __ldg(sb + kb * p.sb_k) : 1.f;
            };
            float col_scale[C::COLS / 32];
            auto load_cols = [&](int32_t kb) {
                if constexpr (ROWS) {
#pragma unroll
                    for (int i = 0; i < C::COLS / 32; ++i) {
                        const int32_t n = col0 + lane + 32 * i;
                        col_scale[i] = n < p.N && kb < p.num_kb ? __ldg(sb + n * p.sb_n + kb * p.sb_k) : 0.f;
                    }
                }
            };
            float a0 = load_a(0), b0 = load_b(0), a1 = load_a(1), b1 = load_b(1);
            load_cols(0);
            uint64_t sum[C::COLS / 2];
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) sum[i] = 0ull;
            for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                const float sc = a0 * b0;
                a0 = a1;
                b0 = b1;
                a1 = load_a(kb + 2);
                b1 = load_b(kb + 2);
                const uint32_t sbuf = wsc + (kb & 1) * (C::COLS * 4);
                if constexpr (ROWS) {
                    if (work) {
#pragma unroll
                        for (int i = 0; i < C::COLS / 32; ++i)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sbuf + (lane + 32 * i) * 4), "f"(col_scale[i])
                                         : "memory");
                        __syncwarp();
                        load_cols(kb + 1);
                    }
                }
                const bool ok = wait_phase(tfull(acc_i), acc_phase, abort_flag, p, WAIT_EPI_TMEM_FULL);
                if (!__all_sync(0xffffffffu, ok)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                const uint64_t s2 = pair_f32(sc, sc);
                if (work) {
                    const uint32_t taddr =
                        tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc_i * BN + h * C::COLS;
                    uint32_t v[2][32];
                    tmem_ld_32x32b_x32(taddr, v[0]);
                    tmem_ld_wait(v[0]);
#pragma unroll
                    for (int c = 0; c < C::COLS / 32; ++c) {
                        if (c + 1 < C::COLS / 32) tmem_ld_32x32b_x32(taddr + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint64_t x = pair_u32(v[c & 1][2 * i], v[c & 1][2 * i + 1]);
                            if constexpr (ROWS) {
                                uint64_t cs;
                                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(cs) : "r"(sbuf + (32 * c + 2 * i) * 4));
                                fma2(sum[16 * c + i], mul2(x, s2), cs);
                            } else {
                                fma2(sum[16 * c + i], x, s2);
                            }
                        }
                        if (c + 1 < C::COLS / 32) tmem_ld_wait(v[(c + 1) & 1]);
                    }
                }
                // this warp's part of the accumulator is read: back to the MMA issuer
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1)
                        mbar_arrive(tempty(acc_i));
                    else
                        mbar_arrive_cluster(mapa(tempty(acc_i), 0));
                }
                if (++acc_i == 2) {
                    acc_i = 0;
                    acc_phase ^= 1u;
                }
            }
            if (!alive || !work) continue;
            // Store the tile part: 128-byte wide subtiles through swizzled staging and a
            // TMA store where the subtile lies inside D (and, grouped, inside the
            // group), else each lane its own row.
            auto emit = [&](auto out_tag, int s, const uint64_t *part) {
                constexpr int OUT = decltype(out_tag)::value;
                constexpr int SUB = OUT == OUT_F32 ? 32 : 64;
                uint32_t o[32];
                if constexpr (OUT == OUT_F32) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) unpair(part[i], o[2 * i], o[2 * i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        uint32_t lo, hi;
                        unpair(part[i], lo, hi);
                        o[i] = pack_bf16x2(lo, hi);
                    }
                }
                const int32_t col = col0 + s * SUB;
                if (col >= p.N) return;
                const bool whole = col + SUB <= p.N;
                if (p.tma_store && whole && (!GROUPED || row0 + 32 <= w.row_end)) {
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    const uint32_t at = stg + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(at + ((static_cast<uint32_t>(i) ^ (lane & 7u)) << 4), o[4 * i], o[4 * i + 1],
                                     o[4 * i + 2], o[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tmD, stg, col, row0, 0, store_policy);
                        bulk_commit();
                    }
                } else if (mine) {
                    const int64_t at = static_cast<int64_t>(row) * p.ldd + col;
                    if (p.vec_store && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(p.D) + at * (OUT == OUT_F32 ? 4 : 2));
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    } else if constexpr (OUT == OUT_F32) {
                        float *dst = static_cast<float *>(p.D) + at;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col + i < p.N) dst[i] = __uint_as_float(o[i]);
                    } else {
                        uint16_t *dst = static_cast<uint16_t *>(p.D) + at;
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (col + i < p.N) dst[i] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
                    }
                }
            };
            if (p.out == OUT_F32) {
#pragma unroll
                for (int s = 0; s < C::COLS / 32; ++s) emit(std::integral_constant<int, OUT_F32>{}, s, sum + 16 * s);
            } else {
#pragma unroll
                for (int s = 0; s < C::COLS / 64; ++s) emit(std::integral_constant<int, OUT_BF16>{}, s, sum + 32 * s);
            }
        }
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
