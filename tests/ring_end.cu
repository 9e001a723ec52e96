// A ring of copies whose askers stop at different places, settled by vh_ring.cuh: every phase that anybody has asked for ends, and
// only after the bytes have landed.  The copies of a second CTA are made by this one.  Nothing is taken from the ring here, so
// no count passes its length.
#include "vh_ring.cuh"

constexpr int kStages = 4, kBytes = 4096;  // per operand and CTA

template <int CTAS>
__global__ void k_ring_end(const uint8_t* src, const uint32_t* counts, uint32_t* done, uint8_t* out) {
    extern __shared__ __align__(128) uint8_t ring[];  // [stage][operand][CTA][kBytes]
    __shared__ __align__(8) unsigned long long full[kStages];
    const int total = kStages * 2 * CTAS * kBytes;
    for (int i = threadIdx.x; i < total; i += blockDim.x) ring[i] = 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) vh::ptx::mbar_init(full + s, 2);
        vh::ptx::fence_barrier_init();
    }
    __syncthreads();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros come before the copies
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t asked[2][CTAS];
        for (int o = 0; o < 2; ++o)
            for (int c = 0; c < CTAS; ++c) asked[o][c] = counts[o * CTAS + c];
        const unsigned long long policy = vh::ptx::policy_evict_first();
        for (uint32_t j = 0; j < kStages; ++j)
            for (int o = 0; o < 2; ++o)
                for (int c = 0; c < CTAS; ++c) {
                    if (j >= asked[o][c]) continue;
                    const int at = ((j * 2 + o) * CTAS + c) * kBytes;
                    if (c == 0) vh::ptx::mbar_arrive_expect_tx(full + j, CTAS * kBytes);
                    vh::ptx::bulk_load(ring + at, src + at, kBytes, full + j, policy);
                }
        vh::ring::settle<kStages, CTAS>(full, asked[0], asked[1], kBytes, kBytes);
        for (int j = 0; j < kStages; ++j) done[j] = vh::ptx::mbar_try_wait(full + j, 0u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += blockDim.x) out[i] = ring[i];
}

// counts: of W by each CTA, of X by each CTA; at most kStages.
extern "C" __attribute__((visibility("default"))) int ring_end(const uint8_t* src, const uint32_t* counts, int ctas, uint32_t* done, uint8_t* out) {
    const int smem = kStages * 2 * ctas * kBytes;
    auto kernel = ctas == 1 ? k_ring_end<1> : k_ring_end<2>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 1;
    kernel<<<1, 128, smem>>>(src, counts, done, out);
    return cudaGetLastError() != cudaSuccess;
}
