// Bounded mbarrier waits of the persistent kernels.  P is a kernel's parameter
// block: it holds timeout_ns and drain_ns (the limits of a wait) and status (the
// device status word a wait that gives up is reported in).
#pragma once
#include <cstdint>

#include "gemm_params.h"
#include "ptx.cuh"

namespace ts {

template <class P>
__device__ __forceinline__ void report_timeout(const P &p, int where) {
    const unsigned long long info = (static_cast<unsigned long long>(where) << 32) | blockIdx.x;
    if (atomicCAS(&p.status[0], 0ull, 1ull) == 0ull) atomicExch(&p.status[1], info);
    atomicAdd(&p.status[2], 1ull);
}

// Bounded phase wait.  honor_abort: give up as soon as another role aborted
// (role loops); drains pass false and rely on their own limit alone.
template <class P>
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int *abort_flag,
                                       bool honor_abort, const P &p, int where) {
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (honor_abort && *abort_flag) return false;
            if (globaltimer() - t0 > limit_ns) {
                report_timeout(p, where);
                *abort_flag = 1;
                return false;
            }
        }
    }
}

template <class P>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                           const P &p, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, p.timeout_ns, abort_flag, true, p, where);
}

// A wait of few instructions and without a function call, for loops whose registers
// and instruction-cache lines are scarce.  It gives up when another role of the CTA
// has (a role that waits with a time limit, and that this wait's end depends on or
// that depends on it) or, should none, after kLeanPolls polls, whatever that limit: a few
// seconds at least (a poll tries the barrier and reads the abort flag, two dependent loads
// of shared memory).  The caller reports it then.
constexpr uint32_t kLeanPolls = 1u << 27;
__device__ __forceinline__ bool wait_lean(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t n = 0; n < kLeanPolls; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    return false;
}

// Bounded wait for roles whose waits last about a tile and whose wake-up is not
// on the critical path (epilogue warps waiting for an accumulator, the CLC
// scheduler waiting for a free slot): it sleeps between polls, leaving the
// issue slots and shared-memory port of its SM sub-partition to the producer
// and the MMA issuer.  Measured: 0.5-1 % faster at 8192^3 than polling.
template <class P>
static __device__ __noinline__ bool wait_long_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                                   const P &p, int where) {
    const uint64_t t0 = globaltimer();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > p.timeout_ns) {
            report_timeout(p, where);
            *abort_flag = 1;
            return false;
        }
        __nanosleep(500);
    }
}

template <class P>
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          const P &p, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_long_slow(bar, parity, abort_flag, p, where);
}

template <class P>
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                           const P &p) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, p.drain_ns, abort_flag, false, p, WAIT_DRAIN);
}

}  // namespace ts
