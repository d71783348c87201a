// Orthogonalised updates of small matrices in one launch.
//
// The products of the iteration depend on each other, and for a matrix of some hundred rows each is
// over in 2 us, while a launch and its CTAs' prologue and exchange take 5 to 6.  Here a cooperative
// grid of one CTA per SM walks through the phases (sum of squares, normalisation, three products a
// step) with a barrier over the grid between them.  A product's tiles are 128 rows by 64 or 128
// columns, so that even small matrices occupy many SMs and a tile's whole K range is in flight at
// once or nearly so.  What bounds a phase: some 3 us (the barrier, the first loads' round trip, the
// epilogue's stores and the fences behind them), and the loads of a tile's K loop, 180 ns for 64 of K
// whether their turns hold 64 or 128.
//
// The barrier is a counter in global memory that every CTA adds to and polls, with a limit on the
// wait.  A phase's results are written by plain stores and read by TMA in the next: each writer
// orders its stores before later asynchronous reads (a proxy fence and a fence at GPU scope) before
// its CTA arrives, each reading CTA fences again behind the barrier.
//
// Warp roles (384 threads): warp 0 loads, warp 1 multiplies, warps 4 to 11 store; all of them
// normalise.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "linear_kernel.cuh"
#include "orth.cuh"

namespace ts {
namespace {

constexpr int kOneThreads = 384, kOneEpiWarps = 8;
constexpr int kOneBoxBytes = 64 * 64 * 2;
constexpr int kOneHalves = 2;  // K blocks of 64 in a stage: 2048 x 1024 142 us, with one 152
constexpr int kOneMaxStages = 4;
constexpr int kOneSmem = kSmemLimit - 1024;  // dynamic: some is static, the normalisation's sums

struct OneParams {
    OrthParams prep;
    int32_t g_f32, g_vec;
    int32_t batch, R, C, n, steps, tall;
    float a, b, c;
    uint16_t *X[2], *A, *B;
    int64_t ldx, ldn, x_matrix, n_matrix;
    uint16_t *O;
    int64_t ldo, o_matrix;
    int32_t o_vec;          // O's rows start on 16-byte boundaries
    int32_t bn, stages;     // columns of a tile; operand stages
    FastDiv div_tiles[2], div_cols[2];  // symmetric and last product: tiles of a matrix, of a row of tiles
    int32_t tiles[2];
    int32_t *barrier;
    uint64_t timeout_ns, drain_ns;
    unsigned long long *status;
};

}  // namespace
template <>
constexpr bool kCtaScope<OneParams> = true;
namespace {

// Tensor maps of X (two buffers), A and b A + c A^2, in boxes of 64 of K by 64 and by 128 rows; of X with
// its columns as the operand's rows, in boxes of 64 x 64.
struct OneMaps {
    CUtensorMap m[4][2], mn[2];
};

struct OnePhase {
    int32_t ma, mb;  // of the operands: 0, 1: X, 2: A, 3: b A + c A^2
    int32_t a_mn, b_mn, num_kb, sym, last;
    int32_t M, N;
    float alpha, beta;
    const uint16_t *aux;
    int64_t ld_aux, aux_matrix;
    uint16_t *D;
    int64_t ldd, d_matrix;
};

__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Arrive and wait until all CTAs have arrived `count` times; one thread.
__device__ __forceinline__ bool grid_barrier(const OneParams &p, int32_t count, volatile int *abort_flag) {
    __threadfence();
    const int32_t want = count * static_cast<int32_t>(gridDim.x);
    atomicAdd(p.barrier, 1);
    const uint64_t t0 = globaltimer();
    for (;;) {
        int32_t v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p.barrier) : "memory");
        if (v >= want) return true;
        if (globaltimer() - t0 > p.timeout_ns) {
            report_timeout(p, WAIT_GRID);
            *abort_flag = 1;
            return false;
        }
    }
}

__global__ void __launch_bounds__(kOneThreads, 1)
    orth_one_kernel(const __grid_constant__ OneMaps maps, const __grid_constant__ OneParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t stages = static_cast<uint32_t>(p.stages), bn = static_cast<uint32_t>(p.bn);
    const uint32_t b_boxes = bn / 64, half_bytes = (2 + b_boxes) * kOneBoxBytes, stage_bytes = kOneHalves * half_bytes;
    const uint32_t s_ring = base, s_bar = s_ring + stages * stage_bytes;
    auto full = [&](uint32_t s) { return s_bar + 8u * s; };
    auto empty = [&](uint32_t s) { return s_bar + 8u * (stages + s); };
    auto tfull = [&](uint32_t a) { return s_bar + 8u * (2 * stages + a); };
    auto tempty = [&](uint32_t a) { return s_bar + 8u * (2 * stages + 2 + a); };
    const uint32_t mma_done = s_bar + 8u * (2 * stages + 4);
    const uint32_t tail = s_bar + 8u * (2 * stages + 5);
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(gbase + (tail - base));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(gbase + (tail - base) + 4);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int32_t cta = static_cast<int32_t>(blockIdx.x), ctas = static_cast<int32_t>(gridDim.x);

    if (warp == 0 && lane == 0) {
        for (uint32_t s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull(a), 1);
            mbar_init(tempty(a), kOneEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        for (int i = 0; i < 8; ++i) prefetch_tmap(&maps.m[i >> 1][i & 1]);
        for (int i = 0; i < 2; ++i) prefetch_tmap(&maps.mn[i]);
    }
    if (warp == 1) {
        tmem_alloc<1>(tail, 256);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // ------------------------------------------------ normalisation
    int32_t arrivals = 0;
    // All threads; false: give up.  One thread decides for the CTA: a warp that read the flag for itself might
    // see what a quicker one sets in the phase behind the barrier, and leave the others alone at the next.
    // (By a word of its own, which the next call writes behind its first barrier; a barrier with a vote takes
    // 0.25 us longer.)
    __shared__ int stop;
    auto next_phase = [&] {
        fence_proxy_async_global();
        __syncthreads();
        if (threadIdx.x == 0) {
            const int given_up = *abort_flag;  // nobody else writes it before the next barrier
            stop = !grid_barrier(p, ++arrivals, abort_flag) || given_up;
        }
        __syncthreads();
        return stop == 0;
    };
    const int64_t shares = static_cast<int64_t>(p.batch) * p.prep.chunks;
    auto prepare = [&](auto type, auto vec) {
        using T = decltype(type);
        constexpr bool VEC = decltype(vec)::value;
        for (int64_t i = cta; i < shares; i += ctas)
            orth_norm<T, VEC, kOneThreads>(p.prep, i / p.prep.chunks, i % p.prep.chunks);
        if (!next_phase()) return false;
        for (int64_t i = cta; i < shares; i += ctas)
            orth_scale<T, VEC, kOneThreads>(p.prep, i / p.prep.chunks, i % p.prep.chunks);
        return true;
    };
    const bool prepared = p.g_f32 ? (p.g_vec ? prepare(float(), std::true_type()) : prepare(float(), std::false_type()))
                                  : (p.g_vec ? prepare(uint16_t(), std::true_type()) : prepare(uint16_t(), std::false_type()));

    // ------------------------------------------------ products
    uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, issued = 0;
    for (int32_t step = 0; prepared && step < 3 * p.steps; ++step) {
        if (!next_phase()) break;
        const int32_t which = step % 3, iter = step / 3;
        OnePhase f;
        const int32_t mx = iter & 1;
        f.last = 0;
        f.sym = which < 2;
        if (which == 0) {
            f.ma = f.mb = mx;
            f.a_mn = f.b_mn = p.tall;
            f.num_kb = ((p.tall ? p.R : p.C) + 64 * kOneHalves - 1) / (64 * kOneHalves);
            f.alpha = 1.f / kOrthScale;
            f.beta = 0.f;
            f.aux = nullptr;
            f.D = p.A;
        } else if (which == 1) {
            f.ma = f.mb = 2;
            f.a_mn = f.b_mn = 0;
            f.num_kb = (p.n + 64 * kOneHalves - 1) / (64 * kOneHalves);
            f.alpha = p.c / kOrthScale;
            f.beta = p.b;
            f.aux = p.A;
            f.D = p.B;
        } else {
            f.ma = p.tall ? mx : 3;
            f.mb = p.tall ? 3 : mx;
            f.a_mn = 0;
            f.b_mn = !p.tall;
            f.num_kb = (p.n + 64 * kOneHalves - 1) / (64 * kOneHalves);
            f.last = iter + 1 == p.steps;
            f.alpha = f.last ? 1.f / (kOrthScale * kOrthScale) : 1.f / kOrthScale;
            f.beta = f.last ? p.a / kOrthScale : p.a;
            f.aux = p.X[iter & 1];
            f.D = f.last ? p.O : p.X[(iter + 1) & 1];
        }
        f.M = f.sym ? p.n : p.R;
        f.N = f.sym ? p.n : p.C;
        f.ld_aux = f.sym ? p.ldn : p.ldx;
        f.aux_matrix = f.sym ? p.n_matrix : p.x_matrix;
        f.ldd = f.sym ? p.ldn : f.last ? p.ldo : p.ldx;
        f.d_matrix = f.sym ? p.n_matrix : f.last ? p.o_matrix : p.x_matrix;
        const int32_t units = p.tiles[f.sym ? 0 : 1] * p.batch;
        // tile u: rows 128 mb, columns bn nb of matrix z; symmetric, those on and right of the diagonal's blocks
        auto unit = [&](int32_t u, int32_t &mb, int32_t &nb, int32_t &z) {
            const int k = f.sym ? 0 : 1;
            z = fast_div(u, p.div_tiles[k]);
            const int32_t t = u - z * p.tiles[k];
            if (!f.sym) {
                mb = fast_div(t, p.div_cols[1]);
                nb = t - mb * ((f.N + p.bn - 1) / p.bn);
                return;
            }
            // a row of tiles after another; they get shorter by a block of 128
            const int32_t cols = (f.N + p.bn - 1) / p.bn, per = 128 / p.bn;
            int32_t left = t;
            for (mb = 0; left >= cols - mb * per; ++mb) left -= cols - mb * per;
            nb = mb * per + left;
        };

        if (warp == 0) {
            const bool leader = elect_one();
            bool alive = true;
            fence_proxy_async_global();  // the loads below come after what the barrier has made visible
            for (int32_t u = cta; u < units && alive; u += ctas) {
                int32_t mb, nb, z;
                unit(u, mb, nb, z);
                const int32_t a_row = mb * 128, b_row = nb * p.bn;
                for (int32_t kb = 0; kb < f.num_kb; ++kb) {
                    if (!wait_phase(empty(stage), phase ^ 1u, abort_flag, p, WAIT_PRODUCER_EMPTY)) {
                        alive = false;
                        break;
                    }
                    if (leader) {
                        mbar_arrive_expect_tx(full(stage), stage_bytes);
#pragma unroll
                        for (int i = 0; i < kOneHalves; ++i) {
                            const uint32_t at = s_ring + stage * stage_bytes + i * half_bytes;
                            const int32_t k = (kb * kOneHalves + i) * 64;
                            auto load = [&](uint32_t dst, int32_t m, bool mn, int32_t row, uint32_t boxes) {
                                if (mn) {  // boxes of 64 rows side by side
                                    for (uint32_t c = 0; c < boxes; ++c)
                                        tma_load_3d(dst + c * kOneBoxBytes, &maps.mn[m], full(stage), row + 64 * static_cast<int32_t>(c), k, z);
                                } else {
                                    tma_load_3d(dst, &maps.m[m][boxes - 1], full(stage), k, row, z);
                                }
                            };
                            load(at, f.ma, f.a_mn, a_row, 2);
                            load(at + 2 * kOneBoxBytes, f.mb, f.b_mn, b_row, b_boxes);
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
        } else if (warp == 1) {
            const bool leader = elect_one();
            const uint32_t idesc = (1u << 4) | (uint32_t(f.a_mn) << 15) | (uint32_t(f.b_mn) << 16) | ((bn >> 3) << 17) |
                                   ((128u >> 4) << 24);
            const uint32_t a_step = f.a_mn ? (16 * 128) >> 4 : 32 >> 4, b_step = f.b_mn ? (16 * 128) >> 4 : 32 >> 4;
            bool alive = true;
            for (int32_t u = cta; u < units && alive; u += ctas) {
                if (!wait_phase(tempty(acc), acc_phase ^ 1u, abort_flag, p, WAIT_MMA_TMEM_EMPTY)) break;
                tc_fence_after();
                for (int32_t kb = 0; kb < f.num_kb; ++kb) {
                    if (!wait_phase(full(stage), phase, abort_flag, p, WAIT_MMA_FULL)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int i = 0; i < kOneHalves; ++i) {
                            const uint32_t at = s_ring + stage * stage_bytes + i * half_bytes;
                            const uint64_t da = f.a_mn ? sw128_mn_desc(at) : sw128_kmajor_desc(at);
                            const uint64_t db = f.b_mn ? sw128_mn_desc(at + 2 * kOneBoxBytes) : sw128_kmajor_desc(at + 2 * kOneBoxBytes);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16<1>(tmem_base + acc * 128, da + a_step * kk, db + b_step * kk, idesc,
                                            kb != 0 || i != 0 || kk != 0);
                        }
                        mma_commit(empty(stage));
                    }
                    __syncwarp();
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!alive) break;
                if (leader) mma_commit(tfull(acc));
                __syncwarp();
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
        } else if (warp >= kRoleWarps) {
            const int j = warp - kRoleWarps, q = j & 3, h = j >> 2;
            for (int32_t u = cta; u < units; u += ctas) {
                int32_t mb, nb, z;
                unit(u, mb, nb, z);
                const int32_t row = mb * 128 + 32 * q + lane, col0 = nb * p.bn + h * (p.bn / 2);
                const uint16_t *const aux = f.aux ? f.aux + z * f.aux_matrix + row * f.ld_aux + col0 : nullptr;
                const int chunks = p.bn / 64;  // of 32 columns
                uint4 a[2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (aux && c < chunks && row < f.M && col0 + 32 * c + 8 * i < f.N)
                            a[c][i] = __ldcg(reinterpret_cast<const uint4 *>(aux + 32 * c + 8 * i));
                if (!wait_phase(tfull(acc), acc_phase, abort_flag, p, WAIT_EPI_TMEM_FULL)) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * 128 + h * (p.bn / 2);
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + 32 * c, v);
                    tmem_ld_wait();
                    if (c + 1 == chunks) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty(acc));
                    }
                    const int32_t col = col0 + 32 * c;
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0 = f.alpha * __uint_as_float(v[2 * i]), x1 = f.alpha * __uint_as_float(v[2 * i + 1]);
                        if (aux) {
                            const uint4 &t = a[0][i / 4];
                            const uint32_t w = i % 4 == 0 ? t.x : i % 4 == 1 ? t.y : i % 4 == 2 ? t.z : t.w;
                            x0 = fmaf(f.beta, f16_to_f32(static_cast<uint16_t>(w)), x0);
                            x1 = fmaf(f.beta, f16_to_f32(static_cast<uint16_t>(w >> 16)), x1);
                        }
                        o[i] = f.last ? pack_bf16x2(__float_as_uint(x0), __float_as_uint(x1))
                                      : pack_f16x2(__float_as_uint(x0), __float_as_uint(x1));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[0][i] = a[1][i];  // the next chunk's
                    uint16_t *const d = f.D + z * f.d_matrix + row * f.ldd + col;
                    if (row < f.M) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // rows of the workspace are padded to eight columns
                            if (!f.last || (p.o_vec && col + 8 * i + 8 <= f.N)) {
                                if (col + 8 * i < f.N)
                                    *reinterpret_cast<uint4 *>(d + 8 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (col + 8 * i + e < f.N)
                                        d[8 * i + e] = static_cast<uint16_t>(o[4 * i + e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                    if (f.sym && col >= (mb + 1) * 128) {
                        // the mirror image, two rows at once (as in the product kernel)
                        const int32_t r = mb * 128 + 32 * q + (lane & ~1), c0 = col + (lane & 1);
                        uint16_t *m = f.D + z * f.d_matrix + c0 * f.ldd + r;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, o[i], 1);
                            const uint32_t two = lane & 1 ? __byte_perm(got, o[i], 0x7632) : __byte_perm(o[i], got, 0x5410);
                            if (c0 + 2 * i < f.N) *reinterpret_cast<uint32_t *>(m) = two;  // r < M: left of the diagonal
                            m += 2 * f.ldd;
                        }
                    }
                }
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        __syncwarp();
    }
    // every load has landed and every MMA has completed before shared memory and TMEM are given up
    if (warp == 0) {
        const uint32_t n = issued < stages ? issued : stages;
        for (uint32_t i = 0; i < n; ++i) {
            if (stage == 0) {
                stage = stages;
                phase ^= 1u;
            }
            --stage;
            wait_drain(full(stage), phase, abort_flag, p);
        }
    } else if (warp == 1) {
        if (elect_one()) mma_commit(mma_done);
        __syncwarp();
        wait_drain(mma_done, 0, abort_flag, p);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(tmem_base, 256);
}

}  // namespace

// 64 columns while X's tiles then run at once: a tile's K loop is bound by its loads, and more, narrower
// tiles share them among more SMs.
OrthTiles orth_one_tiles(const OrthRun &r, int64_t sms) {
    OrthTiles t;
    t.bn = r.batch * cdiv(r.R, 128) * cdiv(r.C, 64) <= sms ? 64 : 128;
    t.x = cdiv(r.R, 128) * cdiv(r.C, t.bn);
    t.sym = 0;
    for (int64_t mb = 0; mb < cdiv(r.n, 128); ++mb) t.sym += cdiv(r.n, t.bn) - mb * (128 / t.bn);
    return t;
}

ts_status orth_one(const OrthRun &r) {
    const int64_t sms = device_sms(current_device());
    if (sms <= 0) return fail(TS_ERR_CUDA, "cannot query the SM count");
    OneParams p;
    std::memset(&p, 0, sizeof p);
    p.prep = r.prep;
    // a share of a matrix for each CTA, or more matrices than CTAs
    p.prep.chunks = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(r.prep.chunks, cdiv(sms, r.batch))));
    p.g_f32 = r.f32;
    p.g_vec = r.vec;
    p.batch = static_cast<int32_t>(r.batch);
    p.R = static_cast<int32_t>(r.R);
    p.C = static_cast<int32_t>(r.C);
    p.n = static_cast<int32_t>(r.n);
    p.steps = r.steps;
    p.tall = r.R > r.C;
    p.a = r.a;
    p.b = r.b;
    p.c = r.c;
    for (int i = 0; i < 2; ++i) p.X[i] = r.X[i];
    p.A = r.A;
    p.B = r.B;
    p.ldx = r.ldx;
    p.ldn = r.ldn;
    p.x_matrix = r.R * r.ldx;
    p.n_matrix = r.ldn * r.ldn;
    p.O = static_cast<uint16_t *>(r.O);
    p.ldo = r.ldo;
    p.o_matrix = r.o_matrix;
    p.o_vec = reinterpret_cast<uintptr_t>(r.O) % 16 == 0 && (r.R <= 1 || r.ldo % 8 == 0) && (r.batch <= 1 || r.o_matrix % 8 == 0);
    const OrthTiles tiles = orth_one_tiles(r, sms);
    p.bn = tiles.bn;
    const int stage_bytes = kOneHalves * (2 + p.bn / 64) * kOneBoxBytes;
    p.stages = std::min(kOneMaxStages, (kOneSmem - 1024 - 256) / stage_bytes);
    p.tiles[0] = static_cast<int32_t>(tiles.sym);
    p.tiles[1] = static_cast<int32_t>(tiles.x);
    for (int i = 0; i < 2; ++i) p.div_tiles[i] = fast_div_for(p.tiles[i]);
    p.div_cols[1] = fast_div_for(cdiv(r.C, p.bn));
    p.barrier = r.barrier;
    const double tmo = r.timeout_s > 0 ? r.timeout_s : 2.0;
    p.timeout_ns = std::max<uint64_t>(1, static_cast<uint64_t>(std::min(tmo, 60.0) * 1e9));
    p.drain_ns = 200ull * 1000 * 1000;
    ts_status s;
    p.status = device_status_word(&s);
    if (!p.status) return s;
    OneMaps maps;
    const uint16_t *const at[4] = {r.X[0], r.X[1], r.A, r.B};
    for (int i = 0; i < 4; ++i) {
        const int64_t rows = i < 2 ? r.R : r.n, cols = i < 2 ? r.C : r.n, ld = i < 2 ? r.ldx : r.ldn;
        const int64_t strides[2] = {ld * 2, (i < 2 ? r.R : r.ldn) * ld * 2};
        auto encode = [&](CUtensorMap &m, int64_t width, int box_rows) {
            const int64_t dims[3] = {width, rows, r.batch};
            const int box[3] = {64, box_rows, 1};
            return encode_map(&m, at[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box);
        };
        for (int j = 0; j < 2; ++j)
            if ((s = encode(maps.m[i][j], cols, 64 << j)) != TS_OK) return s;
        // to the end of a sector, as in the products' maps
        if (i < 2 && (s = encode(maps.mn[i], cdiv(cols, 16) * 16, 64)) != TS_OK) return s;
    }
    static std::atomic<uint64_t> prepared{0};  // devices
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    cudaError_t e = cudaSuccess;
    if (!bit || !(prepared.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(orth_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneSmem);
        if (e != cudaSuccess) return cuda_fail(e, "one-launch orthogonalisation");
        if (bit) prepared.fetch_or(bit, std::memory_order_acq_rel);
    }
    e = cudaMemsetAsync(r.barrier, 0, sizeof(int32_t), r.stream);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the grid barrier");
    cudaLaunchConfig_t cfg = {};
    // as many CTAs as the widest phase has work for
    const int64_t work = std::max<int64_t>(p.tiles[1] * r.batch, std::max<int64_t>(p.tiles[0] * r.batch, p.prep.chunks * r.batch));
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(sms, work)), 1, 1);
    cfg.blockDim = dim3(kOneThreads, 1, 1);
    cfg.dynamicSmemBytes = 1024 + p.stages * stage_bytes + 256;
    cfg.stream = r.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, orth_one_kernel, maps, p);
    return e == cudaSuccess ? TS_OK : cuda_fail(e, "one-launch orthogonalisation");
}

}  // namespace ts
