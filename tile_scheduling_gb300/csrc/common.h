// Host-side helpers shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tsgemm.h"
#include "gemm_params.h"

namespace ts {

// Record a thread-local error message and return `s`.
ts_status fail(ts_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Map a CUDA runtime error to TS_ERR_CUDA with context.
ts_status cuda_fail(cudaError_t e, const char *what);

int current_device();
int device_sms(int dev);
int device_smem_optin(int dev);
// Device address of the library-owned status word on the current device.
unsigned long long *device_status_word(ts_status *err);

// One compiled GEMM variant (tile shape, cluster size, output type).
struct GemmLaunch {
    CUtensorMap a, b, d;
    GemmParams p;
    int grid;
    cudaStream_t stream;
};

// Encode a tiled tensor map: `rank` dimensions of
// `dims` elements (innermost first), strides in bytes of dimensions 1.., boxes
// of `box` elements.  Out-of-range elements of a load read as zero.
ts_status encode_map(CUtensorMap *m, const void *ptr, CUtensorMapDataType dt, int rank, const int64_t *dims,
                     const int64_t *strides, const int *box,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// Launch a kernel as a programmatic dependent of the previous kernel in its
// stream (it calls grid_dep_wait before its first global memory access).
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Multiplier and shift of FastDiv for divisor d (1 <= d < 2^31; an empty grid's
// divisor 0 is taken as 1, it divides nothing).
inline FastDiv fast_div_for(int64_t d) {
    if (d < 1) d = 1;
    int l = 0;
    while ((int64_t{1} << l) < d) ++l;
    FastDiv f;
    f.s = 31 + l;
    f.m = ((uint64_t{1} << f.s) + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d);
    f.pad = 0;
    return f;
}

inline bool ranges_overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

struct GemmVariant {
    int bn, cg, out, epi_warps, merge, log, stages, smem_bytes;
    ts_gemm_protocol protocol;  // barrier layout and arrival counts of this variant
    cudaError_t (*launch)(const GemmLaunch &);
    // Workers (CTAs, or 2-CTA clusters) that can be resident at once.
    cudaError_t (*max_workers)(int *);
};

// log = 1: the protocol-logging instantiation (a test instrument; few shapes have one).
const GemmVariant *find_variant(int bn, int cg, int out, int epi_warps, int merge, int log = 0);

}  // namespace ts
