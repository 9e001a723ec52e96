// Product of two block-scaled 4-bit matrices: y[t][v] = gx(t) gw(v) sum_h X[t,h] W[v,h], both in the tiled layout.
//
// The contraction runs on the 4-bit tensor cores (tcgen05.mma kind::mxf4nvf4, one e4m3 scale per 16 elements of either
// operand, fp32 accumulators in TMEM).  A = 128 rows of W per CTA, B = up to 128 rows of X, K = 64 per MMA.  A record of the
// tiled layout is the operand's shared-memory image, so a stage of the ring is two bulk copies of W and X (codes and scales
// lie together), without tensor maps.  The scales go from there to TMEM by tcgen05.cp, each ring stage to columns of its
// own: they are written again only when the stage's MMAs have been committed.
//
// Epilogue: an accumulator lane is a row of W and a column a row of X, so a warp's 32 lanes write 32 neighbours of a row of y.
//
// Every wait is bounded; on expiry the CTA's flag is set, the tiles concerned become NaN, copies in flight are waited for, and
// TMEM is freed.
#include <algorithm>
#include <atomic>

#include "vh_nvfp4_tiles.h"
#include "vh_row_kernels.h"
#include "vh_rows.cuh"
#include "vh_tc.cuh"

namespace vh {
namespace mm4 {

using namespace tc;
using ptx::bulk_load;
using ptx::mbar_arrive;
using ptx::mbar_arrive_expect_tx;
using ptx::mbar_drain;
using ptx::mbar_init;
using ptx::mbar_wait;
using ptx::policy_evict_first;
using ptx::policy_evict_last;

constexpr int kTileM = kTileRows;
constexpr int kEpiWarps = 8;  // two per quarter of the TMEM lanes, on alternate blocks of 32 rows of X
constexpr int kThreadsM = 32 * (2 + kEpiWarps);
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;
constexpr int kScaleCol = 256;   // behind two accumulators of 128 columns
constexpr int kScaleCols = 32;   // per stage: 4 x 4 of W, 4 x 4 of X
static_assert(kScaleCol + kMaxStages * kScaleCols <= kTmemCols, "scales of every stage");

struct alignas(8) Bars {
    unsigned long long full[kMaxStages];
    unsigned long long empty[kMaxStages];
    unsigned long long tmem_full[2];
    unsigned long long tmem_empty[2];
    unsigned long long mma_done;
    unsigned int tmem_base;
    unsigned int err;
};

struct Args {
    const uint8_t *x, *w;
    float x_scale, w_scale;
    const float *x_scales, *w_scales;
    int T, V, H;
    int records;  // per row of records
    int n_w, n_x; // tiles of W and of X
    void* y;
    long long y_stride;
};

// Instruction descriptor, kind::mxf4nvf4: e2m1 A and B, e4m3 scales, K = 64, both K-major.
__host__ __device__ constexpr uint32_t idesc_nvf4(int M, int N) {
    return (1u << 7)                      // A format: e2m1
           | (1u << 10)                   // B format: e2m1
           | ((uint32_t)(N >> 3) << 17)   // N / 8
           | ((uint32_t)(M >> 7) << 27);  // M / 128
}

template <int CTAS>
__device__ __forceinline__ void mma_nvf4(uint32_t tmem_d, unsigned long long adesc, unsigned long long bdesc, uint32_t idesc,
                                         uint32_t scale_a, uint32_t scale_b, uint32_t accumulate) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate)
            : "memory");
}

// 32 lines of 16 bytes (512 in a row) to 4 columns of each quarter of the TMEM lanes.
__device__ __forceinline__ unsigned long long scale_desc(uint32_t saddr) {
    return (unsigned long long)((saddr >> 4) & 0x3FFFu)  // no swizzle: 8 lines of 16 bytes, then
           | (unsigned long long)(128u >> 4) << 32       // the next 8 lines
           | 1ull << 46;
}
template <int CTAS>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, unsigned long long desc) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else  // in both CTAs, each from its own shared memory
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

template <int NMAX>
struct Config {
    static constexpr int kStageX = NMAX * 128 + kTileScales;
    static constexpr int kStage = kTileBytes + kStageX;
    static constexpr int kStages = std::min(kMaxStages, (226 * 1024 - 2048) / kStage);
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + sizeof(Bars);
};

template <typename TO, int NMAX>
__global__ void __launch_bounds__(kThreadsM, 1) k_matmul(const Args a) {
    using C = Config<NMAX>;
    constexpr int STAGES = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // stage s: W codes and scales, X codes (NMAX lines) and scales
    Bars* bars = reinterpret_cast<Bars*>(smem + (size_t)STAGES * C::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n_tiles = (long long)a.n_w * a.n_x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->tmem_full[i], 1);
            mbar_init(&bars->tmem_empty[i], kEpiWarps);
        }
        mbar_init(&bars->mma_done, 1);
        bars->err = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    // rows of X of tile `tx`, as the MMA takes them
    auto cols = [&](int tx) { return min(NMAX, (a.T - tx * NMAX + 15) / 16 * 16); };

    if (warp == 0) {
        if (lane == 0) {
            // W is read before the previous kernel is waited for, X after.
            const unsigned long long pol_w = a.n_x > 1 ? policy_evict_last() : policy_evict_first(), pol_x = policy_evict_last();
            uint32_t it = 0;
            bool ok = true, waited = false;
            auto load_x = [&](uint32_t j, int tx, int kt) {
                const int s = j % STAGES;
                uint8_t* to = smem + (size_t)s * C::kStage + kTileBytes;
                // NMAX of a record's 128 lines, and all of its scales
                const uint8_t* from = a.x + ((size_t)(tx * NMAX / kTileRows) * a.records + kt) * kTileBytes;
                bulk_load(to, from + (tx * NMAX % kTileRows) * 128, cols(tx) * 128, &bars->full[s], pol_x);
                bulk_load(to + NMAX * 128, from + kTileCodes, kTileScales, &bars->full[s], pol_x);
            };
            auto release_first_ring = [&](uint32_t n) {  // all of one tile of X, or of several: by their order
                rows_wait();
                rows_fence_async();
                for (uint32_t j = 0; j < n; ++j) {
                    const long long tile = blockIdx.x + (long long)(j / a.records) * gridDim.x;
                    load_x(j, (int)(tile % a.n_x), (int)(j % a.records));
                }
                waited = true;
            };
            for (long long tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
                const int tw = (int)(tile / a.n_x), tx = (int)(tile % a.n_x);
                for (int kt = 0; kt < a.records; ++kt, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&bars->empty[s], ((it / STAGES) & 1u) ^ 1u, &bars->err)) { ok = false; break; }
                    mbar_arrive_expect_tx(&bars->full[s], (uint32_t)(kTileBytes + cols(tx) * 128 + kTileScales));
                    bulk_load(smem + (size_t)s * C::kStage, a.w + ((size_t)tw * a.records + kt) * kTileBytes, kTileBytes,
                              &bars->full[s], pol_w);
                    if (waited)
                        load_x(it, tx, kt);
                    else if (it + 1 == (uint32_t)STAGES)
                        release_first_ring(it + 1);
                }
            }
            if (!waited) release_first_ring(it);
            for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0); j < it; ++j)
                mbar_drain(&bars->full[j % STAGES], (j / STAGES) & 1u);
        }
    } else if (warp == 1) {
        // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers; one lane issues.  (With the
        // loop in one lane every instruction's operands were moved there first: 12 instructions took 1,400 cycles a stage.)
        const bool leader = elect_one();
        const uint32_t base = smem_u32(smem);
        uint32_t it = 0, local = 0;
        bool ok = true;
        for (long long tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++local) {
            const uint32_t idesc = idesc_nvf4(kTileM, cols((int)(tile % a.n_x)));
            const uint32_t buf = local & 1u;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->tmem_empty[buf], ((local >> 1) & 1u) ^ 1u, &bars->err))) break;
            tc_fence_after();
            for (int kt = 0; kt < a.records; ++kt, ++it) {
                const int s = it % STAGES;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->full[s], (it / STAGES) & 1u, &bars->err))) { ok = false; break; }
                tc_fence_after();
                const uint32_t sw = base + s * C::kStage, sx = sw + kTileBytes;
                const uint32_t tw = tmem_base + kScaleCol + s * kScaleCols, tx = tw + 16, td = tmem_base + buf * 128u;
                const unsigned long long dw = smem_desc_sw128(sw), dx = smem_desc_sw128(sx);
                const unsigned long long gw = scale_desc(sw + kTileCodes), gx = scale_desc(sx + NMAX * 128);
                const int steps = min(4, (a.H - kt * kTileElems + 63) / 64);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps) {
                            scales_to_tmem<1>(tw + ks * 4, gw + ks * 32);
                            scales_to_tmem<1>(tx + ks * 4, gx + ks * 32);
                        }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps)
                            mma_nvf4<1>(td, dw + ks * 2, dx + ks * 2, idesc, tw + ks * 4, tx + ks * 4, (kt > 0 || ks > 0) ? 1u : 0u);
                    mma_commit(&bars->empty[s]);
                }
                __syncwarp();
            }
            if (ok && leader) mma_commit(&bars->tmem_full[buf]);
            __syncwarp();
        }
        if (leader) {
            mma_commit(&bars->mma_done);
            mbar_drain(&bars->mma_done, 0u);
        }
        __syncwarp();
    } else {
        rows_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint32_t local = 0;
        bool ok = true;
        for (long long tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++local) {
            const uint32_t buf = local & 1u;
            const int tw = (int)(tile / a.n_x), tx = (int)(tile % a.n_x);
            const int v = tw * kTileM + quarter * 32 + lane, t0 = tx * NMAX;
            const float gw = a.w_scales != nullptr ? (v < a.V ? a.w_scales[v] : 0.0f) : a.w_scale;
            const int blocks = (cols(tx) + 31) / 32;
            if (ok) ok = mbar_wait(&bars->tmem_full[buf], (local >> 1) & 1u, &bars->err);
            tc_fence_after();
            for (int g = half; g < blocks; g += 2) {
                const int t = t0 + g * 32;
                float acc[32];
                tmem_ld32(tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * 128u + g * 32u, acc);
                float gx = a.x_scale;
                if (a.x_scales != nullptr) gx = t + lane < a.T ? a.x_scales[t + lane] : 0.0f;
                if (!ok) gx = quiet_nan();
                TO* y = static_cast<TO*>(a.y) + (long long)t * a.y_stride + v;
                const int n = min(32, a.T - t);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float f = acc[j] * __shfl_sync(0xFFFFFFFFu, gx, j) * gw;
                    if (j < n && v < a.V) y[(long long)j * a.y_stride] = from_f32<TO>(f);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->tmem_empty[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------
// More rows of X: CTA pairs (cta_group::2) on 256 rows of W x 256 rows of X, two records, or up to 128 at X's end, where each
// CTA has half the lines of the last record.  Each CTA stages its record of W, its lines of X and the scales of both records; the
// leader issues; each CTA's TMEM has the accumulators of its own rows of W and the scales of all rows of X, 32 rows to a column
// and a record's in four columns (tcgen05.cp writes four at a time, at a multiple of four).  Per stage a CTA takes in 38 KiB for 512 cycles of MMAs, a little more than an SM is given by L2 (64 bytes a cycle).
// Two accumulators of 256 columns would leave the scales no room: there is one, and the epilogue takes all of it into registers
// (128 a thread) before it hands it back and begins to write.
//
// The records come by tensor maps over the buffer's bytes, since those copies may signal the leader's barrier.

constexpr int kStages2 = 5;
constexpr int kScales2 = 256, kScaleCols2 = 48;  // columns: behind the accumulator; per stage 4 x 4 of W, 4 x 8 of X
constexpr int kStageB2 = kTileBytes + kTileCodes + 2 * kTileScales;
constexpr int kMapRow = 256;                      // bytes of a row of the tensor maps
static_assert(kScales2 + kStages2 * kScaleCols2 <= kTmemCols, "scales of every stage");
constexpr size_t kSmem2 = 1024 + (size_t)kStages2 * kStageB2 + sizeof(Bars);

template <typename TO>
__global__ void __launch_bounds__(kThreadsM, 1)
    k_matmul_pair(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_codes,
                  const __grid_constant__ CUtensorMap map_scales, const Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // stage: W (codes, scales), codes of X, scales of both records of X
    Bars* bars = reinterpret_cast<Bars*>(smem + (size_t)kStages2 * kStageB2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const long long n_tiles = (long long)a.n_w * a.n_x;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages2; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->tmem_full[0], 1);
        mbar_init(&bars->tmem_empty[0], 2 * kEpiWarps);  // of both CTAs
        mbar_init(&bars->mma_done, 1);
        bars->err = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    // rows of X of a tile, as the MMA takes them: two records, or some lines of one
    auto cols = [&](int tx) { return a.T - tx * 256 > kTileRows ? 256 : (a.T - tx * 256 + 31) / 32 * 32; };

    if (warp == 0) {
        if (lane == 0) {
            // W is read before the previous kernel is waited for, X after.
            const unsigned long long pol_w = a.n_x > 1 ? policy_evict_last() : policy_evict_first(), pol_x = policy_evict_last();
            uint32_t it = 0;
            bool ok = true, waited = false;
            auto load_x = [&](uint32_t j, int tx, int kt) {
                const int s = j % kStages2;
                const uint32_t bar = map_to_rank(smem_u32(&bars->full[s]), 0);
                uint8_t* to = smem + (size_t)s * kStageB2 + kTileBytes;
                auto row = [&](int r) { return ((2 * tx + r) * a.records + kt) * (kTileBytes / kMapRow); };  // r: of the two records
                const int n = cols(tx);  // of one record: the other half of its lines, and what lies behind them
                tma_load_2d_pair(to, &map_codes, bar, 0, n == 256 ? row((int)rank) : row(0) + (int)rank * (n / 2 * 128 / kMapRow), pol_x);
                tma_load_2d_pair(to + kTileCodes, &map_scales, bar, 0, row(0) + kTileCodes / kMapRow, pol_x);
                tma_load_2d_pair(to + kTileCodes + kTileScales, &map_scales, bar, 0, row(1) + kTileCodes / kMapRow, pol_x);
            };
            auto release_first_ring = [&](uint32_t n) {
                rows_wait();
                rows_fence_async();
                for (uint32_t j = 0; j < n; ++j) {
                    const long long tile = pair + (long long)(j / a.records) * pairs;
                    load_x(j, (int)(tile % a.n_x), (int)(j % a.records));
                }
                waited = true;
            };
            for (long long tile = pair; tile < n_tiles && ok; tile += pairs) {
                const int tw = (int)(tile / a.n_x) * 2 + (int)rank, tx = (int)(tile % a.n_x);
                for (int kt = 0; kt < a.records; ++kt, ++it) {
                    const int s = it % kStages2;
                    if (!mbar_wait(&bars->empty[s], ((it / kStages2) & 1u) ^ 1u, &bars->err)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2u * kStageB2);
                    tma_load_2d_pair(smem + (size_t)s * kStageB2, &map_w, map_to_rank(smem_u32(&bars->full[s]), 0), 0,
                                     (tw * a.records + kt) * (kTileBytes / kMapRow), pol_w);
                    if (waited)
                        load_x(it, tx, kt);
                    else if (it + 1 == (uint32_t)kStages2)
                        release_first_ring(it + 1);
                }
            }
            if (!waited) release_first_ring(it);
            if (rank == 0)  // the leader's barriers see both CTAs' loads
                for (uint32_t j = (it > (uint32_t)kStages2 ? it - kStages2 : 0); j < it; ++j)
                    mbar_drain(&bars->full[j % kStages2], (j / kStages2) & 1u);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            uint32_t it = 0, local = 0;
            bool ok = true;
            for (long long tile = pair; tile < n_tiles && ok; tile += pairs, ++local) {
                const uint32_t idesc = idesc_nvf4(2 * kTileM, cols((int)(tile % a.n_x)));
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->tmem_empty[0], (local & 1u) ^ 1u, &bars->err))) break;
                tc_fence_after();
                for (int kt = 0; kt < a.records; ++kt, ++it) {
                    const int s = it % kStages2;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->full[s], (it / kStages2) & 1u, &bars->err))) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = base + s * kStageB2, sx = sw + kTileBytes;
                    const uint32_t tw = tmem_base + kScales2 + s * kScaleCols2, tx = tw + 16;
                    const unsigned long long dw = smem_desc_sw128(sw), dx = smem_desc_sw128(sx);
                    const unsigned long long gw = scale_desc(sw + kTileCodes), gx = scale_desc(sx + kTileCodes);
                    const int steps = min(4, (a.H - kt * kTileElems + 63) / 64);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < steps) {
                                scales_to_tmem<2>(tw + ks * 4, gw + ks * 32);
                                scales_to_tmem<2>(tx + ks * 8, gx + ks * 32);
                                scales_to_tmem<2>(tx + ks * 8 + 4, gx + kTileScales / 16 + ks * 32);
                            }
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < steps)
                                mma_nvf4<2>(tmem_base, dw + ks * 2, dx + ks * 2, idesc, tw + ks * 4, tx + ks * 8,
                                            (kt > 0 || ks > 0) ? 1u : 0u);
                        mma_commit_pair(&bars->empty[s]);
                    }
                    __syncwarp();
                }
                if (ok && leader) mma_commit_pair(&bars->tmem_full[0]);
                __syncwarp();
            }
            if (leader) {
                mma_commit_pair(&bars->mma_done);
                mbar_drain(&bars->mma_done, 0u);
            }
            __syncwarp();
        }
    } else {
        rows_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t empty = map_to_rank(smem_u32(&bars->tmem_empty[0]), 0);
        uint32_t local = 0;
        bool ok = true;
        for (long long tile = pair; tile < n_tiles; tile += pairs, ++local) {
            const int tw = (int)(tile / a.n_x) * 2 + (int)rank, tx = (int)(tile % a.n_x);
            const int v = tw * kTileM + quarter * 32 + lane, t0 = tx * 256;
            const int blocks = cols(tx) / 32;  // this warp has half, half + 2, ..
            const float gw = a.w_scales != nullptr ? (v < a.V ? a.w_scales[v] : 0.0f) : a.w_scale;
            float gx[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int t = t0 + (2 * g + half) * 32 + lane;
                gx[g] = a.x_scales != nullptr ? (t < a.T ? a.x_scales[t] : 0.0f) : a.x_scale;
            }
            if (ok) ok = mbar_wait(&bars->tmem_full[0], local & 1u, &bars->err);
            tc_fence_after();
            float acc[4][32];
            const uint32_t at = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * 32);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (2 * g + half < blocks) tmem_ld32(at + g * 64u, acc[g]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(empty);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int t = t0 + (2 * g + half) * 32;
                if (2 * g + half >= blocks || t >= a.T) break;
                TO* y = static_cast<TO*>(a.y) + (long long)t * a.y_stride + v;
                const int n = min(32, a.T - t);
                const float gt = ok ? gx[g] : quiet_nan();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float f = acc[g][j] * __shfl_sync(0xFFFFFFFFu, gt, j) * gw;
                    if (j < n && v < a.V) y[(long long)j * a.y_stride] = from_f32<TO>(f);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------

static int sm_count() {
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    int n = cache[dev & 63].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
        cache[dev & 63].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <typename TO, int NMAX>
static cudaError_t run_n(Args a, cudaStream_t s) {
    using C = Config<NMAX>;
    auto kernel = k_matmul<TO, NMAX>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    a.n_w = (int)(((long long)a.V + kTileM - 1) / kTileM);
    a.n_x = (int)(((long long)a.T + NMAX - 1) / NMAX);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>((long long)a.n_w * a.n_x, sm_count()));
    cfg.blockDim = dim3(kThreadsM);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// A buffer of records as rows of kMapRow bytes, copied `box` rows at a time; past its end zeros.
static bool byte_map(CUtensorMap* m, const void* base, size_t bytes, int box) {
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kMapRow, (cuuint64_t)(bytes / kMapRow)};
    cuuint64_t strides[1] = {(cuuint64_t)kMapRow};
    cuuint32_t boxes[2] = {(cuuint32_t)kMapRow, (cuuint32_t)box};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs that are resident at once, per device.
template <typename TO>
static int resident_pairs() {
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    int n = cache[dev & 63].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaFuncSetAttribute(k_matmul_pair<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem2) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
    cfg.blockDim = dim3(kThreadsM);
    cfg.dynamicSmemBytes = kSmem2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_matmul_pair<TO>, &cfg) != cudaSuccess) return 0;
    cache[dev & 63].store(n, std::memory_order_relaxed);
    return n;
}

template <typename TO>
static cudaError_t run_pair(Args a, int pairs, cudaStream_t s) {
    a.n_w = (int)(((long long)a.V + 2 * kTileM - 1) / (2 * kTileM));
    a.n_x = (int)(((long long)a.T + 255) / 256);
    alignas(64) CUtensorMap mw, mc, ms;
    if (!byte_map(&mw, a.w, nvfp4_tiles_bytes(a.V, a.H), kTileBytes / kMapRow) ||
        !byte_map(&mc, a.x, nvfp4_tiles_bytes(a.T, a.H), kTileCodes / kMapRow) ||
        !byte_map(&ms, a.x, nvfp4_tiles_bytes(a.T, a.H), kTileScales / kMapRow))
        return cudaErrorNotSupported;
    const cudaError_t e =
        cudaFuncSetAttribute(k_matmul_pair<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem2);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<long long>((long long)a.n_w * a.n_x, pairs)));
    cfg.blockDim = dim3(kThreadsM);
    cfg.dynamicSmemBytes = kSmem2;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_matmul_pair<TO>, mw, mc, ms, a);
}

template <typename TO>
static cudaError_t run(const Nvfp4MatmulArgs& m, cudaStream_t s) {
    Args a{};
    a.x = m.x;
    a.w = m.w;
    a.x_scale = m.x_scale;
    a.w_scale = m.w_scale;
    a.x_scales = m.x_scales;
    a.w_scales = m.w_scales;
    a.T = m.T;
    a.V = m.V;
    a.H = m.H;
    a.records = tiles_per_row(m.H);
    a.y = m.y;
    a.y_stride = m.y_stride;
    if (a.T <= 32) return run_n<TO, 32>(a, s);
    if (a.T <= kTileRows) return run_n<TO, 128>(a, s);
    // rows of tiles of bytes / 256 in 31 bits (549 GB)
    const int pairs = resident_pairs<TO>();
    return pairs > 0 ? run_pair<TO>(a, pairs, s) : run_n<TO, 128>(a, s);
}

}  // namespace mm4

cudaError_t launch_nvfp4_matmul(const Nvfp4MatmulArgs& a, int dtype, cudaStream_t s) {
    return dtype == VH_F32    ? mm4::run<float>(a, s)
           : dtype == VH_BF16 ? mm4::run<__nv_bfloat16>(a, s)
                              : mm4::run<__half>(a, s);
}

}  // namespace vh
