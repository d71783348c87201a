// Host launcher for one instantiation of the fused-epilogue product kernel (one translation unit each).
#pragma once
#include <atomic>

#include "common.h"
#include "linear_kernel.cuh"

namespace ts {
namespace {

template <int BN, int CG, int MODE, int OUT>
cudaError_t linear_launch(const LinLaunch &L) {
    using C = LinCfg<BN, CG, MODE == LIN_PRE>;
    auto *kernel = linear_kernel<BN, CG, MODE, OUT>;
    static std::atomic<uint64_t> prepared{0};  // devices
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(prepared.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        if (bit) prepared.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(L.grid), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::smem_bytes(L.p.stages, L.p.bufs);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (CG == 2) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, L.a, L.b, L.d, L.aux, L.pre, L.p);
}

template <int BN, int CG, int MODE>
int linear_stages(int bufs) {
    return LinCfg<BN, CG, MODE == LIN_PRE>::stages(bufs);
}

template <int BN, int CG, int MODE>
constexpr auto iteration_launch() -> cudaError_t (*)(const LinLaunch &) {
    if constexpr (MODE == LIN_BARE)
        return &linear_launch<BN, CG, MODE, OUT_F16>;
    else
        return nullptr;
}

}  // namespace
}  // namespace ts

// One for each type of D.
#define TS_LINEAR_VARIANT(NAME, BN, CG, MODE)                                                                     \
    namespace ts {                                                                                                \
    extern const LinVariant NAME;                                                                                 \
    const LinVariant NAME = {BN, CG, MODE,                                                                        \
                             {&linear_launch<BN, CG, MODE, OUT_BF16>, &linear_launch<BN, CG, MODE, OUT_F32>,      \
                              iteration_launch<BN, CG, MODE>()},                                                  \
                             &linear_stages<BN, CG, MODE>};                                                       \
    }
