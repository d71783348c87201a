// Launchers of the split product (linear_split.cuh).
#include <atomic>

#include "linear_split.cuh"

namespace ts {
namespace {

template <int BN, bool SWAP>
cudaError_t split_prepare() {
    static std::atomic<uint64_t> prepared{0};  // devices
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit && (prepared.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(linear_split_kernel<BN, SWAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemLimit);
    if (e == cudaSuccess && bit) prepared.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int BN, bool SWAP>
cudaError_t split_launch(const LinLaunch &L) {
    using C = SplitCfg<BN, SWAP>;
    const cudaError_t e = split_prepare<BN, SWAP>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(L.grid), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::smem_bytes(L.p.stages, L.p.split);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.p.split > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(L.p.split);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<BN, SWAP>, L.a, L.b, L.p);
}

// Clusters of `size` CTAs that run at once with one or two of them on an SM (0: none, or an error),
// asked once per size.
template <int BN, bool SWAP>
int split_clusters(int size, int ctas) {
    using C = SplitCfg<BN, SWAP>;
    static std::atomic<int> known[2][kMaxSplit + 1];  // their number + 1; devices of a process are alike
    if (const int n = known[ctas - 1][size].load(std::memory_order_relaxed)) return n - 1;
    if (split_prepare<BN, SWAP>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::smem_bytes(C::stages(size, ctas), size);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, linear_split_kernel<BN, SWAP>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[ctas - 1][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int BN, bool SWAP>
int split_stages(int split, int ctas) {
    return SplitCfg<BN, SWAP>::stages(split, ctas);
}

}  // namespace

extern const SplitVariant split_128, split_swap_64, split_swap_32;
const SplitVariant split_128 = {128, 0, &split_launch<128, false>, &split_clusters<128, false>,
                                &split_stages<128, false>};
const SplitVariant split_swap_64 = {64, 1, &split_launch<64, true>, &split_clusters<64, true>,
                                &split_stages<64, true>};
const SplitVariant split_swap_32 = {32, 1, &split_launch<32, true>, &split_clusters<32, true>,
                                &split_stages<32, true>};

}  // namespace ts
