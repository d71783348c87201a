// Launchers of the split product (linear_split.cuh).
#include <atomic>

#include "linear_split.cuh"

namespace ts {
namespace {

template <int BN, bool SWAP, int OUT>
cudaError_t split_prepare() {
    static std::atomic<uint64_t> prepared{0};  // devices
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit && (prepared.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(linear_split_kernel<BN, SWAP, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemLimit);
    if (e == cudaSuccess && bit) prepared.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int BN, bool SWAP, int OUT>
cudaError_t split_launch(const LinLaunch &L) {
    using C = SplitCfg<BN, SWAP>;
    const cudaError_t e = split_prepare<BN, SWAP, OUT>();
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
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<BN, SWAP, OUT>, L.a, L.b, L.p);
}

// Clusters of `size` CTAs that run at once with one or two of them on an SM (0: none, or an error),
// asked once per size.
template <int BN, bool SWAP, int OUT>
int split_clusters(int size, int ctas) {
    using C = SplitCfg<BN, SWAP>;
    static std::atomic<int> known[2][kMaxSplit + 1];  // their number + 1; devices of a process are alike
    if (const int n = known[ctas - 1][size].load(std::memory_order_relaxed)) return n - 1;
    if (split_prepare<BN, SWAP, OUT>() != cudaSuccess) return 0;
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
    if (cudaOccupancyMaxActiveClusters(&n, linear_split_kernel<BN, SWAP, OUT>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[ctas - 1][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int BN, bool SWAP, int OUT>
int split_stages(int split, int ctas) {
    return SplitCfg<BN, SWAP>::stages(split, ctas);
}

template <int BN, bool SWAP, int OUT>
constexpr SplitVariant variant() {
    return {BN, SWAP, &split_launch<BN, SWAP, OUT>, &split_clusters<BN, SWAP, OUT>, &split_stages<BN, SWAP, OUT>};
}

}  // namespace

extern const SplitVariant split_128[3], split_swap_64[3], split_swap_32[3];
const SplitVariant split_128[3] = {variant<128, false, 0>(), variant<128, false, 1>(), variant<128, false, 2>()};
const SplitVariant split_swap_64[3] = {variant<64, true, 0>(), variant<64, true, 1>(), variant<64, true, 2>()};
const SplitVariant split_swap_32[3] = {variant<32, true, 0>(), variant<32, true, 1>(), variant<32, true, 2>()};

}  // namespace ts
