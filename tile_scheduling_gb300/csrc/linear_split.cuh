// The fused-epilogue product where there are few output tiles: a cluster's CTAs share K.
//
// One tile of 128 x BN per cluster.  Each CTA multiplies its share of K into Tensor Memory and sends
// its fp32 partial sums to the CTAs that own them, each a share of the accumulator's rows: a slot for
// every sender, written through the cluster's shared memory.  After one cluster barrier an owner adds
// its slots up in the order of the K shares (so results do not depend on timing), applies the
// epilogue and stores.  Sent rather than fetched: a fetch waits for a second round trip after the
// barrier, and needs a second barrier before a CTA may leave.
//
// What bounds it is latency: one TMA round trip (some 0.8 us), the exchange, and the launch; a
// persistent CTA that walks the K loop alone has 192 KB in flight and needs several.  In a graph, 768 x
// 768 x 768 by four CTAs a tile 6.4 us, 24 x 2048 x 8192 with a residual 10.2 (5 of them w's bytes).
//
// SWAP: the rows of D (few tokens) are the instruction's columns and the columns of D (the rows of
// w) its 128 rows, so that a tile reads 128 rows of w for BN = 32 or 64 tokens.
#pragma once
#include "linear_kernel.cuh"

namespace ts {

template <int BN_, bool SWAP_>
struct SplitCfg {
    static constexpr int BN = BN_;
    static constexpr bool SWAP = SWAP_;
    static constexpr int THREADS = 256;
    static constexpr int BM = 128, BK = 64, UMMA_K = 16;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BOX_BYTES = 64 * BK * 2;
    static constexpr int TILE_ROWS = SWAP ? BN : BM, TILE_COLS = SWAP ? BM : BN;  // of D
    // Partial sums: GROUPS of four columns of D and rows of D in a slot, a row of groups (without
    // SWAP: a group's rows) PITCH apart.  Senders write a lane a row of the accumulator, owners read
    // a lane a group; one unit of padding keeps the second conflict-free without SWAP.
    static constexpr int BAR_BYTES = 256;
    static constexpr int MAX_STAGES = 12;
    static constexpr int slot_bytes(int split) { return SWAP ? BM * BN * 4 : (BM / split + 1) * (BN / 4) * 16 * split; }
    static constexpr int smem_bytes(int stages, int split) { return 1024 + stages * STAGE_BYTES + slot_bytes(split) + BAR_BYTES; }
    // with so many CTAs on an SM
    static constexpr int stages(int split, int ctas) {
        const int n = (kSmemLimit / ctas - (ctas > 1 ? 1024 : 0) - smem_bytes(0, split)) / STAGE_BYTES;
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
    static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
    static_assert((2 * MAX_STAGES + 1) * 8 + 8 <= BAR_BYTES, "barrier region");
};

// `count` <= 8 values of a matrix from element `i` on; eight of them (whole) lie on a 16-byte boundary.
__device__ __forceinline__ void load8(const void *q, int64_t i, int type, bool whole, int count, float (&f)[8]) {
    if (type == OUT_F32) {
        const float *const s = static_cast<const float *>(q) + i;
        if (whole) {
            const float4 t = __ldcg(reinterpret_cast<const float4 *>(s)), u = __ldcg(reinterpret_cast<const float4 *>(s) + 1);
            f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w, f[4] = u.x, f[5] = u.y, f[6] = u.z, f[7] = u.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = k < count ? __ldcg(s + k) : 0.f;
        }
        return;
    }
    const uint16_t *const s = static_cast<const uint16_t *>(q) + i;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (whole) {
        const uint4 t = __ldcg(reinterpret_cast<const uint4 *>(s));
        w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) w[k >> 1] |= uint32_t(__ldcg(s + k)) << (16 * (k & 1));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = type == OUT_BF16 ? __uint_as_float(w[k] << 16) : f16_to_f32(static_cast<uint16_t>(w[k]));
        f[2 * k + 1] = type == OUT_BF16 ? __uint_as_float(w[k] & 0xffff0000u) : f16_to_f32(static_cast<uint16_t>(w[k] >> 16));
    }
}
__device__ __forceinline__ void pack8(int type, const float (&f)[8], uint32_t (&o)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = type == OUT_BF16 ? pack_bf16x2(__float_as_uint(f[2 * k]), __float_as_uint(f[2 * k + 1]))
                                : pack_f16x2(__float_as_uint(f[2 * k]), __float_as_uint(f[2 * k + 1]));
}
__device__ __forceinline__ void store8(void *q, int64_t i, int type, bool whole, int count, const float (&f)[8]) {
    if (type == OUT_F32) {
        float *const d = static_cast<float *>(q) + i;
        if (whole) {
            reinterpret_cast<float4 *>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) d[k] = f[k];
        }
        return;
    }
    uint16_t *const d = static_cast<uint16_t *>(q) + i;
    uint32_t o[4];
    pack8(type, f, o);
    if (whole) {
        *reinterpret_cast<uint4 *>(d) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) d[k] = static_cast<uint16_t>(o[k >> 1] >> (16 * (k & 1)));
    }
}

// OUT as in the persistent kernel.
template <int BN, bool SWAP, int OUT>
__global__ void __launch_bounds__(SplitCfg<BN, SWAP>::THREADS, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ LinParams p) {
    using C = SplitCfg<BN, SWAP>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t stages = static_cast<uint32_t>(p.stages);
    const uint32_t s_a = base, s_b = s_a + stages * C::A_BYTES, s_slot = s_b + stages * C::B_BYTES;
    const uint32_t s_bar = s_slot + C::slot_bytes(p.split);
    auto full = [&](uint32_t s) { return s_bar + 8u * s; };
    auto empty = [&](uint32_t s) { return s_bar + 8u * (stages + s); };
    const uint32_t mma_done = s_bar + 8u * (2 * stages);
    const uint32_t tail = s_bar + 8u * (2 * stages + 1);
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(gbase + (tail - base));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(gbase + (tail - base) + 4);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int32_t part = p.split > 1 ? static_cast<int32_t>(cluster_ctarank()) : 0;

    if (warp == 0 && lane == 0) {
        for (uint32_t s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc<1>(tail, C::TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (p.split > 1) cluster_arrive();  // this CTA runs: waited for before anything is sent
    const int32_t u = static_cast<int32_t>(blockIdx.x) / p.split;
    const LinUnit w = lin_unit<C>(u, p);
    const int32_t row0 = w.mb * C::TILE_ROWS, col0 = w.nb * C::TILE_COLS;
    const int32_t a_row = SWAP ? col0 : row0, b_row = SWAP ? row0 : col0;  // of the instruction's operands
    const int32_t kb0 = static_cast<int32_t>(static_cast<int64_t>(part) * p.num_kb / p.split);
    const int32_t kb1 = static_cast<int32_t>(static_cast<int64_t>(part + 1) * p.num_kb / p.split);
    grid_dep_wait();
    grid_dep_launch();

    uint32_t stage = 0, phase = 0;
    auto advance = [&] {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    };
    if (warp == 0) {
        const bool leader = elect_one();
        bool alive = true;
        int32_t issued = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            alive = wait_phase(empty(stage), phase ^ 1u, abort_flag, p, WAIT_PRODUCER_EMPTY);
            if (!alive) break;
            if (leader) {
                mbar_arrive_expect_tx(full(stage), C::STAGE_BYTES);
                const uint32_t da = s_a + stage * C::A_BYTES, db = s_b + stage * C::B_BYTES;
                if (p.a_mn) {
#pragma unroll
                    for (int c = 0; c < C::BM / 64; ++c)
                        tma_load_3d(da + c * C::BOX_BYTES, &tmA, full(stage), a_row + 64 * c, kb * C::BK, w.z);
                } else {
                    tma_load_3d(da, &tmA, full(stage), kb * C::BK, a_row, w.z);
                }
                if (p.b_mn) {
#pragma unroll
                    for (int c = 0; c < (BN + 63) / 64; ++c)
                        tma_load_3d(db + c * C::BOX_BYTES, &tmB, full(stage), b_row + 64 * c, kb * C::BK, w.z);
                } else {
                    tma_load_3d(db, &tmB, full(stage), kb * C::BK, b_row, w.z);
                }
            }
            __syncwarp();
            ++issued;
            advance();
        }
        // every load has landed, whether or not the MMA warp came to wait for it
        for (int32_t i = 0; i < static_cast<int32_t>(stages) && i < issued; ++i) {
            if (stage == 0) {
                stage = stages;
                phase ^= 1u;
            }
            --stage;
            wait_drain(full(stage), phase, abort_flag, p);
        }
    } else if (warp == 1) {
        const bool leader = elect_one();
        const uint32_t idesc = p.idesc | (uint32_t(BN >> 3) << 17) | (uint32_t(C::BM >> 4) << 24);
        const uint32_t a_step = p.a_mn ? (16 * 128) >> 4 : 32 >> 4, b_step = p.b_mn ? (16 * 128) >> 4 : 32 >> 4;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            if (!wait_phase(full(stage), phase, abort_flag, p, WAIT_MMA_FULL)) break;
            tc_fence_after();
            if (leader) {
                const uint32_t at_a = s_a + stage * C::A_BYTES, at_b = s_b + stage * C::B_BYTES;
                const uint64_t da = p.a_mn ? sw128_mn_desc(at_a) : sw128_kmajor_desc(at_a);
                const uint64_t db = p.b_mn ? sw128_mn_desc(at_b) : sw128_kmajor_desc(at_b);
#pragma unroll
                for (int kk = 0; kk < C::BK / C::UMMA_K; ++kk)
                    mma_bf16<1>(tmem_base, da + a_step * kk, db + b_step * kk, idesc, kb != kb0 || kk != 0);
                mma_commit(empty(stage));
            }
            __syncwarp();
            advance();
        }
        if (leader) mma_commit(mma_done);
    }
    __syncwarp();
    // given up or not, the instructions in flight have completed before TMEM is read and freed
    if (!wait_phase(mma_done, 0, abort_flag, p, WAIT_EPI_TMEM_FULL)) wait_drain(mma_done, 0, abort_flag, p);
    __syncwarp();
    tc_fence_after();
    if (p.split > 1) cluster_wait();
    // Partial sums to their owners: warps w and w + 4 read lane quarter w % 4, half of the columns each.
    const int32_t share = C::BM / p.split;  // rows of the accumulator that a CTA owns
    {
        constexpr int HALF = BN / 2;  // 16 or more
        constexpr int STEP = HALF < 32 ? HALF : 32;
        const int q = warp & 3, c0 = (warp >> 2) * HALF;
        const int l = 32 * q + lane;  // the accumulator's row
        const int32_t owner = l / share, local = l - owner * share;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + c0;
        const uint32_t slot = p.split > 1 ? mapa(s_slot, owner) : s_slot;
#pragma unroll
        for (int c = 0; c < HALF; c += STEP) {
            uint32_t v[STEP];
            if constexpr (STEP == 32)
                tmem_ld_32x32b_x32(taddr + c, v);
            else
                tmem_ld_32x32b_x16(taddr + c, v);
            tmem_ld_wait();
            if constexpr (SWAP) {
                const uint32_t at = slot + (part * BN * share + local) * 4;
#pragma unroll
                for (int i = 0; i < STEP; ++i) st_cluster_u32(at + (c0 + c + i) * share * 4, v[i]);
            } else {
                const uint32_t at = slot + (part * (BN / 4) * (share + 1) + local) * 16;
#pragma unroll
                for (int i = 0; i < STEP / 4; ++i)
                    st_cluster_v4(at + ((c0 + c) / 4 + i) * (share + 1) * 16, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        }
    }
    tc_fence_before();
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(tmem_base, C::TMEM_COLS);
    if (*abort_flag) return;
    // The owned part of the tile: R rows by G groups of eight columns, a group at a time.  The loop's
    // code is kept small: it runs a few times at most, and fetching it is part of the latency (four
    // groups at once, unrolled, took 1.8 us a turn).
    const int32_t R = min(p.M - row0 - (SWAP ? 0 : part * share), SWAP ? BN : share);
    const int32_t log_g = SWAP ? 28 - __clz(share) : 31 - __clz(BN / 8);  // G = share / 8 or BN / 8, a power of two
    const int32_t row_at = row0 + (SWAP ? 0 : part * share), col_at = col0 + (SWAP ? part * share : 0);
    // A lane a group, or (symmetric) a lane a row: an entry's mirror image then lies next to that of
    // the lane beside it.
    constexpr bool iteration = OUT == OUT_F16;
    const int out = iteration && p.out == OUT_BF16 ? OUT_BF16 : OUT;
    const bool sym = iteration && p.sym, mirror = sym && w.nb > w.mb;
    const int32_t log_r = 31 - __clz(share);
    const int32_t turns = sym ? share << log_g : R << log_g;
#pragma unroll 1
    for (int32_t i = static_cast<int32_t>(threadIdx.x); i < turns; i += C::THREADS) {
        const int32_t r = sym ? i & (share - 1) : i >> log_g, g = sym ? i >> log_r : i & ((1 << log_g) - 1);
        const int32_t row = row_at + r, col = col_at + 8 * g;
        const int32_t count = min(8, p.N - col);
        if (count <= 0 || r >= R) continue;
        const bool whole = count == 8 && p.store_bytes == 16;
        float a[8];
        if (p.aux) load8(p.aux, w.z * p.aux_matrix + row * p.ld_aux + col, OUT, whole, count, a);
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const uint32_t at = s_slot + (SWAP ? (r * share + 8 * g) * 4 : (2 * g * (share + 1) + r) * 16);
        const uint32_t next = SWAP ? 16 : (share + 1) * 16;            // the group's other four columns
        const uint32_t slot = SWAP ? BN * share * 4 : (BN / 4) * (share + 1) * 16;
#pragma unroll
        for (int c = 0; c < kMaxSplit; ++c) {
            if (c < p.split) {
                const uint4 t = ld_shared_v4(at + c * slot), v = ld_shared_v4(at + c * slot + next);
                x[0] += __uint_as_float(t.x), x[1] += __uint_as_float(t.y);
                x[2] += __uint_as_float(t.z), x[3] += __uint_as_float(t.w);
                x[4] += __uint_as_float(v.x), x[5] += __uint_as_float(v.y);
                x[6] += __uint_as_float(v.z), x[7] += __uint_as_float(v.w);
            }
        }
        if constexpr (iteration) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= p.alpha;
        }
        if (!iteration && p.bias) {
            float b[8];
            load8(p.bias, col, p.bias_f32 ? OUT_F32 : OUT_BF16, p.bias_vec && count == 8, count, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] += b[k];
        }
        if (!iteration && p.pre) store8(p.pre, row * p.ld_pre + col, OUT, whole, count, x);
        if (!iteration && p.slope) {
            with_act(p.act, [&](auto act) { apply_slope<decltype(act)::value>(x, a); });
        } else {
            if constexpr (!iteration) with_act(p.act, [&](auto act) { apply_act<decltype(act)::value>(x); });
            if (p.aux) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = iteration ? fmaf(p.beta, a[k], x[k]) : x[k] + a[k];
            }
        }
        store8(p.D, w.z * p.d_matrix + row * p.ldd + col, out, whole, count, x);
        if (mirror) {
            uint32_t o[4];
            pack8(out, x, o);
            uint16_t *const m = static_cast<uint16_t *>(p.D) + w.z * p.d_matrix + row;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < count) m[(col + k) * p.ldd] = static_cast<uint16_t>(o[k >> 1] >> (16 * (k & 1)));
        }
    }
}

}  // namespace ts
