// Product of two block-scaled 4-bit matrices: y[t][v] = gx(t) gw(v) sum_h X[t,h] W[v,h], both in the tiled layout.
//
// The contraction runs on the 4-bit tensor cores (tcgen05.mma kind::mxf4nvf4, one e4m3 scale per 16 elements of either
// operand, fp32 accumulators in TMEM).  A = 128 rows of W per CTA, B = up to 128 rows of X, K = 64 per MMA.  A record of the
// tiled layout is the operand's shared-memory image, so a stage of the ring is two bulk copies of W and X (codes and scales
// lie together), without tensor maps.  The scales go from there to TMEM by tcgen05.cp, each ring stage to columns of its
// own: they are written again only when the stage's MMAs have been committed.
//
// Epilogue: an accumulator lane is a row of W and a column a row of X.  A warp turns its 32 x 32 blocks in shared memory and
// writes 64 or 128 bytes of each of 32 rows of y in 16-byte pieces; where y's rows are not aligned for that, its 32 lanes write 32
// neighbours of a row.  (One row after the other for all, the rows' scales by shuffles: 256 x 248320 x 2048 took 113 us, and
// 104 with a quarter of the contraction: the epilogue set the pace.)
//
// Bound: the stream of W for few rows (4 x 248320 x 2048 44.5 us, 0.97 of the copy rate); for many no unit's limit but the waits of
// the pairs below (4096 x 8192 x 8192 94 us, 5.9 PFLOP/s).  Up to 32 rows of X a stage has 32 lines of X and there are eight stages of W, so
// that enough of it is on its way; with few tiles a cluster shares the records of one (1 x 4096 x 4096 5.9 us, 9.9 with a CTA each).
//
// Every wait is bounded, by a limit that begins when the previous kernel has ended; on expiry the CTA's flag is set, the tiles
// concerned become NaN, copies in flight are waited for (vh_ring.cuh), and TMEM is freed.
#include <algorithm>
#include <atomic>

#include "vh_nvfp4_tiles.h"
#include "vh_ring.cuh"
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
constexpr int kEpiWarps = 8;  // two per quarter of the TMEM lanes, on every other block of 32 rows of X
constexpr int kShare = kEpiWarps / 4;
constexpr int kXWarp = 2 + kEpiWarps;  // asks for X
constexpr int kThreadsM = 32 * (kXWarp + 1);
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
    unsigned int asked[2][2];  // records of W and of X that each CTA of a pair has asked for (in the leader's)
    unsigned int peer_err;
};

struct Args {
    const uint8_t *x, *w;
    float x_scale, w_scale;
    const float *x_scales, *w_scales;
    int T, V, H;
    int records;  // per row of records
    int n_w, n_x; // tiles of W and of X
    int split;    // CTAs that share a tile's records (a cluster), with up to 32 rows of X
    void* y;
    long long y_stride;
    bool wide;    // y's rows are 16-byte aligned
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
// Arrival that orders no memory: the accumulators have been read when it is made.  (With release semantics at cluster scope it
// waits for the warp's stores of the tile before.)
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

constexpr int kTurnBytes = 32 * 32 * 4;  // a turned block, per epilogue warp
constexpr int kEpiBytes = kEpiWarps * kTurnBytes;

// 32 lanes x 32 columns of fp32 from TMEM, without waiting for them; and the wait, before which nothing uses them.
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
template <int G>
__device__ __forceinline__ void tmem_wait(float (&v)[G][32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[g][i]));
}

// A warp's block of y: rows t.. (n of them), columns v0.. (nv of them); lane = column, acc[j] row t + j, whose scale lane j has.
// Turned in shared memory: of odd rows the 16-byte halves of each 32 bytes are swapped, so that eight lanes read two rows' 16-byte
// pieces 32 bytes apart from all banks.
template <typename TO>
__device__ __forceinline__ void write_block(const float (&acc)[32], float gx, float gw, TO* y, long long stride, int n, int nv,
                                            bool wide, float* turn) {
    const int lane = threadIdx.x & 31;
    if (wide && nv == 32) {
        constexpr int LANES = 2 * (int)sizeof(TO);     // of a row: 16 bytes of y each
        constexpr int ROWS = 32 / LANES, E = 16 / (int)sizeof(TO);
        const int row = lane / LANES, piece = lane % LANES;
        TO* to = y + row * stride + piece * E;
#pragma unroll
        for (int j = 0; j < 32; ++j) turn[j * 32 + (lane ^ ((j & 1) << 2))] = acc[j] * gw;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += ROWS) {
            const int r = i + row;
            const float g = __shfl_sync(0xFFFFFFFFu, gx, r);
            RawVec<TO, E> o;
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(turn + r * 32 + ((piece * E + h * 4) ^ ((r & 1) << 2)));
                if constexpr (sizeof(TO) == 4) {
                    o.u[0] = __float_as_uint(q.x * g);
                    o.u[1] = __float_as_uint(q.y * g);
                    o.u[2] = __float_as_uint(q.z * g);
                    o.u[3] = __float_as_uint(q.w * g);
                } else {
                    o.set2(2 * h, q.x * g, q.y * g);
                    o.set2(2 * h + 1, q.z * g, q.w * g);
                }
            }
            if (r < n) o.store(to);
            to += ROWS * stride;
        }
        __syncwarp();
    } else {
        TO* to = y + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float f = acc[j] * gw * __shfl_sync(0xFFFFFFFFu, gx, j);
            if (j < n && lane < nv) *to = from_f32<TO>(f);
            to += stride;
        }
    }
}

// The scales that a warp's blocks of a tile want: asked for a tile ahead.  First row of W v0, first row of X t0; the warp has blocks
// share, share + kShare, .. of 32 rows of X.
template <int G>
struct TileScales {
    float gx[G], gw;
    __device__ __forceinline__ void ask(const Args& a, int v0, int t0, int share) {
        const int lane = threadIdx.x & 31;
        gw = a.w_scales != nullptr ? (v0 + lane < a.V ? a.w_scales[v0 + lane] : 0.0f) : a.w_scale;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int t = t0 + (kShare * g + share) * 32 + lane;
            gx[g] = a.x_scales != nullptr ? (t < a.T ? a.x_scales[t] : 0.0f) : a.x_scale;
        }
    }
};

template <int NMAX>
struct Config {
    static constexpr int kStageX = NMAX * 128 + kTileScales;
    static constexpr int kStage = kTileBytes + kStageX;
    static constexpr int kStages = std::min(kMaxStages, (226 * 1024 - 2048 - kEpiBytes) / kStage);
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpiBytes + sizeof(Bars);
};

// Which CTA of a cluster of `split` adds up a quarter of a tile's rows of W, and the quarter's place there.
__device__ __forceinline__ int owner_of(int quarter, int split) { return split == 2 ? quarter >> 1 : quarter; }
__device__ __forceinline__ int slot_of(int quarter, int split) { return split == 2 ? quarter & 1 : 0; }
constexpr int kMaxSplit = 8;
static_assert(kMaxSplit * kTurnBytes <= kEpiBytes, "partial sums of a quarter from every CTA, in place of the turned blocks");

template <typename TO, int NMAX>
__global__ void __launch_bounds__(kThreadsM, 1) k_matmul(const Args a) {
    using C = Config<NMAX>;
    constexpr int STAGES = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // stage s: W codes and scales, X codes (NMAX lines) and scales
    uint8_t* turn = smem + (size_t)STAGES * C::kStage;
    Bars* bars = reinterpret_cast<Bars*>(turn + kEpiBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n_tiles = (long long)a.n_w * a.n_x;
    // With few tiles a cluster shares the records of one; its partial sums meet below.
    const int split = NMAX == 32 ? a.split : 1;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int k0 = (int)((long long)a.records * rank / split), k1 = (int)((long long)a.records * (rank + 1) / split);
    const long long first_tile = blockIdx.x / split, step = gridDim.x / split;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 2);  // W and X are asked for by a warp each
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
    if (split > 1)
        cluster_sync();  // every CTA of the cluster runs: the others may write to its shared memory
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    // rows of X of tile `tx`, as the MMA takes them
    auto cols = [&](int tx) { return min(NMAX, (a.T - tx * NMAX + 15) / 16 * 16); };

    if (warp == 0 || warp == kXWarp) {
        // As with the issue of MMAs below, the whole warp runs the loop.  W waits for the previous kernel as X does: a head is made by
        // calls (nvfp4_tile, nvfp4_quantize_tiles) whose next one may be its product, and only the wait orders their writes before
        // these reads.  (4 x 65536 x 2048 with its quantisation 17.7 us, 17.8 with W unordered: what comes before does not signal.)
        const bool leader = elect_one(), is_w = warp == 0;
        const unsigned long long policy = is_w && a.n_x == 1 ? policy_evict_first() : policy_evict_last();
        rows_wait();
        rows_fence_async();
        uint32_t it = 0;
        bool ok = true;
        for (long long tile = first_tile; tile < n_tiles && ok; tile += step) {
            const int tw = (int)(tile / a.n_x), tx = (int)(tile % a.n_x);
            const uint32_t x_bytes = (uint32_t)cols(tx) * 128u;
            // of X, NMAX of a record's 128 lines, and all of its scales
            const uint8_t* from = is_w ? a.w + (size_t)tw * a.records * kTileBytes : a.x + (size_t)(tx * NMAX / kTileRows) * a.records * kTileBytes;
            from += (size_t)k0 * kTileBytes;
            const int line = is_w ? 0 : tx * NMAX % kTileRows * 128;
            for (int kt = k0; kt < k1; ++kt, ++it, from += kTileBytes) {
                const int s = it % STAGES;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->empty[s], ((it / STAGES) & 1u) ^ 1u, &bars->err))) { ok = false; break; }
                uint8_t* to = smem + (size_t)s * C::kStage;
                if (leader) {
                    if (is_w) {
                        mbar_arrive_expect_tx(&bars->full[s], kTileBytes);
                        bulk_load(to, from, kTileBytes, &bars->full[s], policy);
                    } else {
                        mbar_arrive_expect_tx(&bars->full[s], x_bytes + kTileScales);
                        bulk_load(to + kTileBytes, from + line, x_bytes, &bars->full[s], policy);
                        bulk_load(to + kTileBytes + NMAX * 128, from + kTileCodes, kTileScales, &bars->full[s], policy);
                    }
                }
                __syncwarp();
            }
        }
        if (leader) bars->asked[is_w ? 0 : 1][0] = it;
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers; one lane issues.  (With the
        // loop in one lane every instruction's operands were moved there first: 12 instructions took 1,400 cycles a stage.)
        rows_wait();  // nothing comes before: else the first wait's limit would count the previous kernel's time
        const bool leader = elect_one();
        const uint32_t base = smem_u32(smem);
        uint32_t it = 0, local = 0;
        bool ok = true;
        for (long long tile = first_tile; tile < n_tiles && ok; tile += step, ++local) {
            const uint32_t idesc = idesc_nvf4(kTileM, cols((int)(tile % a.n_x)));
            const uint32_t buf = local & 1u;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->tmem_empty[buf], ((local >> 1) & 1u) ^ 1u, &bars->err))) break;
            tc_fence_after();
            for (int kt = k0; kt < k1; ++kt, ++it) {
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
                            mma_nvf4<1>(td, dw + ks * 2, dx + ks * 2, idesc, tw + ks * 4, tx + ks * 4, (kt > k0 || ks > 0) ? 1u : 0u);
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
        const int quarter = warp & 3, share = (warp - 2) >> 2;
        constexpr int G = (NMAX + 32 * kShare - 1) / (32 * kShare);  // blocks per warp
        uint32_t local = 0;
        bool ok = true;
        TileScales<G> now, next;
        auto ask = [&](long long tile, TileScales<G>& to) {
            if (tile < n_tiles) to.ask(a, (int)(tile / a.n_x) * kTileM + quarter * 32, (int)(tile % a.n_x) * NMAX, share);
        };
        ask(first_tile, next);
        for (long long tile = first_tile; tile < n_tiles; tile += step, ++local) {
            const uint32_t buf = local & 1u;
            const int v0 = (int)(tile / a.n_x) * kTileM + quarter * 32, tx = (int)(tile % a.n_x), t0 = tx * NMAX;
            const int blocks = (cols(tx) + 31) / 32;
            now = next;
            ask(tile + step, next);
            if (ok) ok = mbar_wait(&bars->tmem_full[buf], (local >> 1) & 1u, &bars->err);
            tc_fence_after();
            float acc[G][32];
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (kShare * g + share < blocks)
                    tmem_ask32(tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * 128u + (kShare * g + share) * 32u, acc[g]);
            tmem_wait(acc);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->tmem_empty[buf]);
            if (NMAX == 32 && split > 1) {
                // to the CTA that adds this quarter up
                if (share == 0) {
                    const uint32_t to = map_to_rank(smem_u32(turn), (uint32_t)owner_of(quarter, split)) +
                                        (uint32_t)((slot_of(quarter, split) * split + rank) * kTurnBytes + lane * 4);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < a.T)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + j * 128), "f"(ok ? acc[0][j] : quiet_nan()) : "memory");
                }
                continue;
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int t = t0 + (kShare * g + share) * 32;
                if (kShare * g + share < blocks && t < a.T && v0 < a.V)
                    write_block(acc[g], ok ? now.gx[g] : quiet_nan(), now.gw, static_cast<TO*>(a.y) + t * a.y_stride + v0, a.y_stride,
                                min(32, a.T - t), min(32, a.V - v0), a.wide, reinterpret_cast<float*>(turn + (warp - 2) * kTurnBytes));
            }
        }
    }
    if (NMAX == 32 && split > 1) {
        __syncwarp();
        cluster_sync();  // every CTA's sums are where they are added
        const int quarter = warp & 3;
        if (warp >= 2 && warp < 6 && owner_of(quarter, split) == rank) {
            const float* from = reinterpret_cast<const float*>(turn + slot_of(quarter, split) * split * kTurnBytes) + lane;
            const int v0 = (int)first_tile * kTileM + quarter * 32;
            TileScales<1> scales;
            scales.ask(a, v0, 0, 0);
#pragma unroll 4
            for (int j = 0; j < a.T; ++j) {  // in the order of the ranks
                float f = from[j * 32];
                for (int r = 1; r < split; ++r) f += from[r * (kTurnBytes / 4) + j * 32];
                f = f * scales.gw * __shfl_sync(0xFFFFFFFFu, scales.gx[0], j);
                if (v0 + lane < a.V) static_cast<TO*>(a.y)[(long long)j * a.y_stride + v0 + lane] = from_f32<TO>(f);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (bars->err != 0u) {
        if (threadIdx.x == 0) ring::settle<STAGES, 1>(bars->full, {bars->asked[0][0]}, {bars->asked[1][0]}, 0u, 0u);
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Many rows of X: CTA pairs (cta_group::2) on 256 rows of W x two records of X, or some lines of one at X's end.  Each CTA stages
// its record of W, half of the tile's lines of X (of two records one each) and the scales of all of them; the leader issues; each
// CTA's TMEM has the accumulators of its own rows of W and the scales of all rows of X, 32 rows to a column and a record's in four
// columns (tcgen05.cp writes four at a time, at a multiple of four).
//
// A stage is 38 KiB per CTA for 512 cycles of MMAs and takes about 700.  Two accumulators of 256 columns would leave the scales no
// room: there is one, and the epilogue takes all of it into registers, in two halves, the second before it hands it back; every
// tile waits for that and the writing of the first, about 2.2 us of the 13.4 that one takes with 32 records (4096 x 8192 x 8192, seven
// tiles to a pair).  No unit is at its limit there: tensor pipe 60% busy, L2 to SM 35% of its rate (1.3 GB, 45 bytes a cycle and
// SM), L2 slices 45%.  (Pairs on one record, with two accumulators: 4096 x 8192 x 8192 138 us, 88 with two records in the same run;
// 256 x 248320 x 2048 84 and 87; what one CTA per tile does as well.)
//
// The records come by tensor maps over the buffer's bytes, since those copies may signal the leader's barrier.

constexpr int kMapRow = 256;  // bytes of a row of the tensor maps
constexpr int kCols2 = 2 * kTileRows;  // rows of X of a tile
constexpr int kStage2 = kTileBytes + kTileCodes + 2 * kTileScales;
constexpr int kStages2 = 5;
constexpr int kScales2 = 256, kScaleCols2 = 48;  // columns: behind the accumulator; per stage 4 x 4 of W, 4 x 8 of X
constexpr size_t kSmem2 = 1024 + (size_t)kStages2 * kStage2 + kEpiBytes + sizeof(Bars);
static_assert(kScales2 + kStages2 * kScaleCols2 <= kTmemCols && kStages2 <= kMaxStages && kStage2 % 1024 == 0, "room");
static_assert(kSmem2 <= 227 * 1024, "shared memory");

template <typename TO>
__global__ void __launch_bounds__(kThreadsM, 1)
    k_matmul_pair(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_codes,
                  const __grid_constant__ CUtensorMap map_scales, const Args a) {
    constexpr int STAGES = kStages2, kStage = kStage2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // stage: W (codes, scales), codes of X, scales of X
    uint8_t* turn = smem + (size_t)STAGES * kStage;
    Bars* bars = reinterpret_cast<Bars*>(turn + kEpiBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const long long n_tiles = (long long)a.n_w * a.n_x;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 2);  // W and X are asked for by a warp each
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->tmem_full[0], 1);
        mbar_init(&bars->tmem_empty[0], 2 * kEpiWarps);  // of both CTAs
        mbar_init(&bars->mma_done, 1);
        bars->err = bars->peer_err = 0u;
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
    // rows of X of a tile, as the MMA takes them: two records, or some lines of one, half of them in each CTA
    auto cols = [&](int tx) {
        const int left = a.T - tx * kCols2;
        return left > kTileRows ? 256 : (left + 31) / 32 * 32;
    };

    if (warp == 0 || warp == kXWarp) {
        const bool leader = elect_one(), is_w = warp == 0;
        const unsigned long long policy = is_w && a.n_x == 1 ? policy_evict_first() : policy_evict_last();
        rows_wait();
        rows_fence_async();
        const uint32_t full0 = map_to_rank(smem_u32(&bars->full[0]), 0);  // the leader's; 8 bytes on the next
        uint32_t it = 0;
        bool ok = true;
        for (long long tile = pair; tile < n_tiles && ok; tile += pairs) {
            const int tw = (int)(tile / a.n_x) * 2 + (int)rank, tx = (int)(tile % a.n_x);
            const int n = cols(tx);
            int row_w = tw * a.records * (kTileBytes / kMapRow), row_x = 2 * tx * a.records * (kTileBytes / kMapRow);
            // of one record: the CTA's half of its lines, and what lies behind them
            const int codes = (int)rank * (n == 256 ? a.records * (kTileBytes / kMapRow) : n / 2 * 128 / kMapRow);
            for (int kt = 0; kt < a.records; ++kt, ++it, row_w += kTileBytes / kMapRow, row_x += kTileBytes / kMapRow) {
                const int s = it % STAGES;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->empty[s], ((it / STAGES) & 1u) ^ 1u, &bars->err))) { ok = false; break; }
                uint8_t* to = smem + (size_t)s * kStage;
                const uint32_t bar = full0 + s * 8u;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2u * (is_w ? kTileBytes : kStage - kTileBytes));
                    if (is_w) {
                        tma_load_2d_pair(to, &map_w, bar, 0, row_w, policy);
                    } else {
                        tma_load_2d_pair(to + kTileBytes, &map_codes, bar, 0, row_x + codes, policy);
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            tma_load_2d_pair(to + kTileBytes + kTileCodes + r * kTileScales, &map_scales, bar, 0,
                                             row_x + (r * a.records) * (kTileBytes / kMapRow) + kTileCodes / kMapRow, policy);
                    }
                }
                __syncwarp();
            }
        }
        if (leader)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&bars->asked[is_w ? 0 : 1][rank]), 0)), "r"(it)
                         : "memory");
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            rows_wait();
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            uint32_t it = 0, local = 0;
            bool ok = true;
            for (long long tile = pair; tile < n_tiles && ok; tile += pairs, ++local) {
                const uint32_t idesc = idesc_nvf4(2 * kTileM, cols((int)(tile % a.n_x)));
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->tmem_empty[0], (local & 1u) ^ 1u, &bars->err))) break;
                tc_fence_after();
                for (int kt = 0; kt < a.records; ++kt, ++it) {
                    const int s = it % STAGES;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars->full[s], (it / STAGES) & 1u, &bars->err))) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = base + s * kStage, sx = sw + kTileBytes;
                    const uint32_t tw = tmem_base + kScales2 + s * kScaleCols2, tx = tw + 16;
                    const unsigned long long dw = smem_desc_sw128(sw), dx = smem_desc_sw128(sx);
                    const unsigned long long gw = scale_desc(sw + kTileCodes), gx = scale_desc(sx + kTileCodes);
                    const int steps = min(4, (a.H - kt * kTileElems + 63) / 64);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < steps) {
                                scales_to_tmem<2>(tw + ks * 4, gw + ks * 32);
#pragma unroll
                                for (int r = 0; r < 2; ++r)
                                    scales_to_tmem<2>(tx + (ks * 2 + r) * 4, gx + r * (kTileScales / 16) + ks * 32);
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
        const int quarter = warp & 3, share = (warp - 2) >> 2;
        const uint32_t empty = map_to_rank(smem_u32(&bars->tmem_empty[0]), 0);
        constexpr int G = kCols2 / (32 * kShare);  // blocks of 32 columns per warp
        static_assert(G == 4, "two and two");
        uint32_t local = 0;
        bool ok = true;
        TileScales<G> now, next;
        auto ask = [&](long long tile, TileScales<G>& to) {
            if (tile < n_tiles)
                to.ask(a, ((int)(tile / a.n_x) * 2 + (int)rank) * kTileM + quarter * 32, (int)(tile % a.n_x) * kCols2, share);
        };
        ask(pair, next);
        for (long long tile = pair; tile < n_tiles; tile += pairs, ++local) {
            const int v0 = ((int)(tile / a.n_x) * 2 + (int)rank) * kTileM + quarter * 32, tx = (int)(tile % a.n_x), t0 = tx * kCols2;
            const int blocks = cols(tx) / 32;  // this warp has share, share + kShare, ..
            now = next;
            ask(tile + pairs, next);
            if (ok) ok = mbar_wait(&bars->tmem_full[0], local & 1u, &bars->err);
            tc_fence_after();
            const uint32_t at = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(share * 32);
            // two blocks at a time: four do not fit the registers, and there is no first-level cache left to spill to
#pragma unroll 1
            for (int g0 = 0; g0 < G; g0 += 2) {
                float acc[2][32];
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    if (kShare * (g0 + g) + share < blocks) tmem_ask32(at + (g0 + g) * (32u * kShare), acc[g]);
                tmem_wait(acc);
                if (g0 + 2 >= G) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed(empty);
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int block = kShare * (g0 + g) + share, t = t0 + block * 32;
                    if (block < blocks && t < a.T && v0 < a.V)
                        write_block(acc[g], ok ? now.gx[g] : quiet_nan(), now.gw, static_cast<TO*>(a.y) + t * a.y_stride + v0, a.y_stride,
                                    min(32, a.T - t), min(32, a.V - v0), a.wide, reinterpret_cast<float*>(turn + (warp - 2) * kTurnBytes));
                }
                now.gx[0] = now.gx[2];
                now.gx[1] = now.gx[3];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && bars->err != 0u)  // both have to know
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&bars->peer_err), rank ^ 1u)), "r"(1u) : "memory");
    __syncwarp();
    cluster_sync();  // no CTA leaves while its peer may still signal or read it
    if ((bars->err | bars->peer_err) != 0u) {
        if (rank == 0 && threadIdx.x == 0)  // the leader's barriers see both CTAs' copies
            ring::settle<STAGES, 2>(bars->full, bars->asked[0], bars->asked[1], kTileBytes, kStage - kTileBytes);
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------

static long long tiles_of(int n, int per) { return ((long long)n + per - 1) / per; }

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
    a.n_w = (int)tiles_of(a.V, kTileM);
    a.n_x = (int)tiles_of(a.T, NMAX);
    const long long tiles = (long long)a.n_w * a.n_x;
    // Clusters while there are SMs for all of them, and two records or more for each CTA.
    a.split = 1;
    while (NMAX == 32 && a.split < kMaxSplit && tiles * a.split * 2 <= sm_count() && a.records >= a.split * 4) a.split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? tiles * a.split : std::min<long long>(tiles, sm_count())));
    cfg.blockDim = dim3(kThreadsM);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
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
    a.n_w = (int)tiles_of(a.V, 2 * kTileM);
    a.n_x = (int)tiles_of(a.T, kCols2);
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
    a.wide = reinterpret_cast<uintptr_t>(m.y) % 16 == 0 && (m.T == 1 || m.y_stride * sizeof(TO) % 16 == 0);
    if (a.T <= 32) return run_n<TO, 32>(a, s);
    if (a.T <= kTileRows) return run_n<TO, 128>(a, s);
    // One CTA per 128 x 128 rows, or pairs: by what a tile takes (us, measured) and the waves of tiles.  A tile takes its
    // contraction and the wait for the accumulators, or the writing of the one before, whichever is longer.
    const long long w = tiles_of(a.V, kTileM), x = tiles_of(a.T, kTileRows);
    const int pairs = resident_pairs<TO>();
    auto waves = [](long long tiles, int at_once) { return (float)((tiles + at_once - 1) / at_once); };
    const float one = waves(w * x, sm_count()) * std::max(1.75f, a.records * 0.325f + 0.7f);
    const float two = waves(tiles_of(a.V, 2 * kTileM) * tiles_of(a.T, kCols2), std::max(pairs, 1)) * std::max(3.3f, a.records * 0.39f + 2.2f) + 2.0f;
    return pairs > 0 && two < one ? run_pair<TO>(a, pairs, s) : run_n<TO, 128>(a, s);
}

}  // namespace mm4

cudaError_t launch_nvfp4_matmul(const Nvfp4MatmulArgs& a, int dtype, cudaStream_t s) {
    return dtype == VH_F32    ? mm4::run<float>(a, s)
           : dtype == VH_BF16 ? mm4::run<__nv_bfloat16>(a, s)
                              : mm4::run<__half>(a, s);
}

}  // namespace vh
