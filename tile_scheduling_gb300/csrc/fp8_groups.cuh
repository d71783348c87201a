// Row ranges of a grouped 8-bit product, read and checked on the device.
#pragma once
#include "fp8_params.h"

namespace ts {

// Rows [lo, hi) of group g, or an empty range when the offsets are not ordered in [0, M].
__device__ __forceinline__ bool group_rows(const Fp8Params &p, int32_t g, int64_t &lo, int64_t &hi) {
    lo = p.offsets[g];
    hi = p.offsets[g + 1];
    if (lo < 0 || hi < lo || hi > p.M) {
        lo = hi = 0;
        return false;
    }
    return true;
}

__device__ __forceinline__ void report_group(const Fp8Params &p, int32_t g) {
    if (atomicCAS(&p.status[0], 0ull, 4ull) == 0ull) atomicExch(&p.status[1], static_cast<unsigned long long>(g));
    atomicAdd(&p.status[2], 1ull);
}

}  // namespace ts
