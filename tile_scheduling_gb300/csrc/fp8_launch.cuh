// Host launcher for one instantiation of the 8-bit product kernel (one translation unit each).
#pragma once
#include <atomic>

#include "common.h"
#include "fp8_kernel.cuh"

namespace ts {
namespace {

template <int BN, int CG, bool ROWS, bool GROUPED, int SC, int AR>
cudaError_t fp8_launch(const Fp8Launch &L) {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>;
    auto *kernel = fp8_gemm_kernel<BN, CG, ROWS, GROUPED, SC, AR>;
    static std::atomic<uint64_t> done{0};  // cudaFuncSetAttribute once per device
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (C::SHIFT_REGS) {
            // the promotion warps wait for registers that the block must have been launched with
            cudaFuncAttributes a;
            e = cudaFuncGetAttributes(&a, kernel);
            if (e != cudaSuccess) return e;
            if (a.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
        }
        if (bit) done.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(L.grid), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(L.cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, L.a, L.b, L.d, L.p);
}

}  // namespace
}  // namespace ts

#define TS_FP8_VARIANT(NAME, BN, CG, ROWS, GROUPED, SC, AR)                                          \
    namespace ts {                                                                                   \
    extern const Fp8Variant NAME;                                                                    \
    const Fp8Variant NAME = {BN, CG, ROWS, GROUPED, AR, &fp8_launch<BN, CG, ROWS, GROUPED, SC, AR>}; \
    }
