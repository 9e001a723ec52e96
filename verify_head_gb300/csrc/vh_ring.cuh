// The end of a ring of copies after a wait has expired.
//
// A stage's barrier takes one arrival per operand (W, X), made by CTA 0 when it asks for its copy and expecting the bytes of
// every CTA of the group; the copies give those bytes.  When a wait expires, those who ask stop, each where it is: then some
// stages have been asked for by some of them only, and their phase would never end, though copies into them may still be on
// their way.  lack() says what such a phase is short of; settle() makes up for it and waits, so that no CTA leaves before what
// was asked for has landed.
#pragma once
#include <stdint.h>

#if defined(__CUDACC__)
#define VH_RING_HD __host__ __device__ __forceinline__
#else
#define VH_RING_HD inline
#endif

namespace vh {
namespace ring {

struct Lack {
    uint32_t arrive;  // arrivals that are missing: CTA 0 has not asked
    uint32_t expect;  // bytes that nobody expects and that will come
    uint32_t give;    // bytes that are expected and will not come
};

// One operand of use j of the ring: CTA c has asked for asked[c] uses so far, of `bytes` each.
template <int CTAS>
VH_RING_HD Lack lack(uint32_t j, const uint32_t (&asked)[CTAS], uint32_t bytes) {
    Lack l = {j < asked[0] ? 0u : 1u, 0u, 0u};
    for (int c = 1; c < CTAS; ++c) {
        if (l.arrive && j < asked[c]) l.expect += bytes;
        if (!l.arrive && j >= asked[c]) l.give += bytes;
    }
    return l;
}

}  // namespace ring
}  // namespace vh

#if defined(__CUDACC__)
#include "vh_ptx.cuh"

namespace vh {
namespace ring {

// Bytes that no copy will bring count as here.
__device__ __forceinline__ void mbar_give(unsigned long long* bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(ptx::smem_u32(bar)), "r"(bytes) : "memory");
}

// By one thread of CTA 0, when nobody asks any more.  Nobody is further ahead of another than the ring is long: a stage is
// free for its next use only when all had asked for this one.
template <int STAGES, int CTAS>
__device__ __forceinline__ void settle(unsigned long long* full, const uint32_t (&w)[CTAS], const uint32_t (&x)[CTAS], uint32_t w_bytes,
                                       uint32_t x_bytes) {
    uint32_t least = 0xFFFFFFFFu, most = 0u;
    for (int c = 0; c < CTAS; ++c) {
        least = min(least, min(w[c], x[c]));
        most = max(most, max(w[c], x[c]));
    }
    for (uint32_t j = least; j < most; ++j)
        for (int operand = 0; operand < 2; ++operand) {
            const Lack l = lack<CTAS>(j, operand ? x : w, operand ? x_bytes : w_bytes);
            unsigned long long* bar = full + j % STAGES;
            if (l.give > 0u) mbar_give(bar, l.give);
            if (l.arrive && l.expect > 0u)
                ptx::mbar_arrive_expect_tx(bar, l.expect);
            else if (l.arrive)
                ptx::mbar_arrive(bar);
        }
    for (uint32_t j = most > (uint32_t)STAGES ? most - STAGES : 0u; j < most; ++j) ptx::mbar_drain(full + j % STAGES, (j / STAGES) & 1u);
}

}  // namespace ring
}  // namespace vh
#endif
