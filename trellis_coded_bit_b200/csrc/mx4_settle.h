// mx4_settle.h -- what is left to do on a pair's stage barriers when one of its
// roles stopped early (mx4_gemm.cu).  No CUDA in here: a host test runs it over
// every way that the roles can stop.
//
// The leader's barrier full[i % stages] completes step i when the leader's
// producer (which announces the bytes of both CTAs) and the four scale warps of
// the pair have arrived and the bytes of both CTAs have landed.  Every role does
// its steps in order, and no role begins a step before all have done the one
// `stages` before it.  So from the number of steps that each role has done, known
// once all have stopped, follows what step i lacks: the arrivals that never come,
// and the bytes that were announced and not sent, or sent and not announced.
// With that made up, the barrier completes exactly when the copies that were
// begun have landed, and the pair may leave.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EXL3_HD __host__ __device__ __forceinline__
#else
#define EXL3_HD inline
#endif

namespace exl3 {

// The roles: the producers of the leader and of its peer, then the scale warps.
constexpr int kMxRoles = 6;

struct MxDebt {
    uint32_t arrivals;  // that nobody makes any more
    int32_t tx;         // bytes to announce (> 0) or to strike off (< 0)
};

// The first step whose copies may still be in flight, and the end of all steps
// that were begun.
EXL3_HD void mx_debt_range(const uint32_t *steps, uint32_t stages, uint32_t &first, uint32_t &end)
{
    end = steps[0] > steps[1] ? steps[0] : steps[1];
    first = end > stages ? end - stages : 0;
}

// What step i lacks; `bytes`: of one CTA in a step.
EXL3_HD MxDebt mx_debt(const uint32_t *steps, uint32_t i, uint32_t bytes)
{
    MxDebt d = {0u, 0};
    d.arrivals = steps[0] <= i;
    for (int r = 2; r < kMxRoles; ++r)
        d.arrivals += steps[r] <= i;
    if (steps[0] <= i && steps[1] > i)
        d.tx = (int32_t)bytes;  // the peer's are on their way, unannounced
    else if (steps[0] > i && steps[1] <= i)
        d.tx = -(int32_t)bytes;
    return d;
}

}  // namespace exl3
