// Host launcher for one instantiation of the fused-epilogue product kernel (one translation unit each).
#pragma once
#include <atomic>

#include "common.h"
#include "linear_kernel.cuh"

namespace ts {
namespace {

template <int BN, int CG, int PRE>
cudaError_t linear_launch(const LinLaunch &L) {
    using C = LinCfg<BN, CG, PRE>;
    auto *kernel = linear_kernel<BN, CG, PRE>;
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

template <int BN, int CG, int PRE>
int linear_stages(int bufs) {
    return LinCfg<BN, CG, PRE>::stages(bufs);
}

}  // namespace
}  // namespace ts

#define TS_LINEAR_VARIANT(NAME, BN, CG, PRE)                                                               \
    namespace ts {                                                                                         \
    extern const LinVariant NAME;                                                                          \
    const LinVariant NAME = {BN, CG, PRE, &linear_launch<BN, CG, PRE>, &linear_stages<BN, CG, PRE>};       \
    }
