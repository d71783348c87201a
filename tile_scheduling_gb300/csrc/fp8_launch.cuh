// Host launcher for one instantiation of the 8-bit product kernel (one translation unit each).
#pragma once
#include <atomic>

#include "common.h"
#include "fp8_kernel.cuh"

namespace ts {
namespace {

// What the kernel needs set before its first launch on a device.
template <int BN, int CG, bool ROWS, bool GROUPED, int SC, int AR>
cudaError_t fp8_prepare() {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>;
    auto *kernel = fp8_gemm_kernel<BN, CG, ROWS, GROUPED, SC, AR>;
    static std::atomic<uint64_t> done{0};  // devices
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
    return cudaSuccess;
}

template <int BN, int CG, bool ROWS, bool GROUPED, int SC, int AR>
cudaError_t fp8_launch(const Fp8Launch &L) {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>;
    auto *kernel = fp8_gemm_kernel<BN, CG, ROWS, GROUPED, SC, AR>;
    const cudaError_t e = fp8_prepare<BN, CG, ROWS, GROUPED, SC, AR>();
    if (e != cudaSuccess) return e;
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

// Clusters of `size` CTAs that run at once (0: none, or an error), asked once per size.
template <int BN, int CG, bool ROWS, bool GROUPED, int SC, int AR>
int fp8_clusters(int size) {
    using C = Fp8Cfg<BN, CG, ROWS, GROUPED, SC, AR>;
    static std::atomic<int> known[kMaxCluster + 1];  // their number + 1; devices of a process are alike
    if (const int n = known[size].load(std::memory_order_relaxed)) return n - 1;
    if (fp8_prepare<BN, CG, ROWS, GROUPED, SC, AR>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<BN, CG, ROWS, GROUPED, SC, AR>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[size].store(n + 1, std::memory_order_relaxed);
    return n;
}

}  // namespace
}  // namespace ts

#define TS_FP8_VARIANT(NAME, BN, CG, ROWS, GROUPED, SC, AR)                                         \
    namespace ts {                                                                                  \
    extern const Fp8Variant NAME;                                                                   \
    const Fp8Variant NAME = {BN, CG, ROWS, GROUPED, AR, &fp8_launch<BN, CG, ROWS, GROUPED, SC, AR>, \
                             &fp8_clusters<BN, CG, ROWS, GROUPED, SC, AR>};                         \
    }
