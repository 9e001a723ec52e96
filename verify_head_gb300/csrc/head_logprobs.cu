// Log probabilities of given tokens straight from hidden rows and the output
// head: the scores S = W Xt come from the tensor cores (tcgen05 + TMEM + TMA)
// and are reduced to each row's softmax statistics as they leave TMEM.
//
//     S[r,v] = sum_h X[r,h] W[v,h]     lse, logprob, entropy, alternatives of S[r,:]
//
// Contraction.  As in verification: A = 128 head rows per CTA (K-major, ring
// of 64-element K stages by TMA), B = the hidden rows, fp32 accumulators in
// two TMEM buffers, so that the epilogue of a tile runs under the MMAs of the
// next.  Up to 128 hidden rows: one CTA per tile of 128 head rows.  More: CTA
// pairs (cta_group::2) on 256 head rows x 256 hidden rows, and up to four
// groups of 256 hidden rows per pass over the head: pair p takes row group
// p % groups, so the pairs that need the same head tile ask for it at about
// the same time and it comes from HBM once.
//
// Epilogue.  An accumulator lane is a head row and a column a hidden row, but
// a row's softmax runs over head rows.  Each warp turns its 32 x 32 blocks in
// shared memory and then lane = hidden row: 32 scores in registers, a running
// maximum and the sums of Stat per hidden row, kept across tiles.  A warp
// loads, turns and sums one block after the other, so a tile's epilogue is a
// chain of waits and not of instructions: two warps per scheduler hide it
// under the MMAs of long rows (H from 512 up), but not of short ones (584 rows
// of 65,536 x 256: 43 us, with 20 alternatives 73 us, against 114 us with four
// warps and 80 us with sixteen on blocks of 16 hidden rows).
//
// Alternatives.  Where they are wanted each block of 32 head rows (a segment)
// leaves its maximum per hidden row in the workspace, and its 32 scores unless
// n larger ones are known.  The n largest scores of a row lie in the n segments
// with the largest maxima (select_top), so the finishing kernel reads the
// maxima and about n blocks of 128 bytes per row.
//
// Every wait is bounded; on expiry the workspace error word is set and the
// CTA drains its copies, frees TMEM and returns.
#include <algorithm>
#include <atomic>

#include "vh_kernels.h"
#include "vh_row_kernels.h"
#include "vh_rows.cuh"
#include "vh_tc.cuh"

namespace vh {
namespace hlp {

using namespace tc;
using ptx::mbar_arrive;
using ptx::mbar_arrive_expect_tx;
using ptx::mbar_drain;
using ptx::mbar_init;
using ptx::mbar_wait;
using ptx::policy_evict_first;
using ptx::policy_evict_last;

constexpr int kTileM = 128;             // head rows per CTA and tile
constexpr int kPairTile = 2 * kTileM;   // head rows per pair and tile
constexpr int kGroup = 256;             // hidden rows per row group (MMA N)
constexpr int kMaxGroups = 4;           // row groups per pass over the head
constexpr int kPassRows = kGroup * kMaxGroups;
constexpr int kOneCtaRows = 128;
constexpr int kEpiWarps = 8;            // two per quarter of the TMEM lanes, on alternate blocks of 32 hidden rows
constexpr int kBoundWarp = 2 + kEpiWarps;
constexpr int kThreadsH = 32 * (kBoundWarp + 1);
constexpr int kMaxStages = 8;
constexpr int kStageW = kTileM * kBlockK * 2;  // 16 KiB
constexpr int kTmemCols = 512;
constexpr int kSeg = 32;                // head rows per segment
constexpr int kTransBytes = 32 * 32 * 4;  // a transposed block, per epilogue warp
constexpr int kMaxParts = 512;          // CTAs that leave statistics of one row
static_assert(kGroup / 2 * 3 * 4 <= kTransBytes, "a warp's statistics fit its block");

struct alignas(8) Bars {
    unsigned long long full[kMaxStages];
    unsigned long long empty[kMaxStages];
    unsigned long long tmem_full[2];
    unsigned long long tmem_empty[2];
    unsigned long long mma_done;
    unsigned int tmem_base;
    uint32_t done;             // an epilogue warp has finished its last tile
    uint32_t bounds[kGroup];   // of the row group's rows: see find_bounds
};

struct Args {
    int R;       // hidden rows of this pass
    int Rp;      // row pitch of the workspace arrays
    int N;       // hidden rows of a row group, rounded up to 16: MMA N
    int H, V;
    int groups;  // row groups (pairs)
    const int32_t* tokens;
    float* tok_score;  // [Rp]
    float4* part;      // [CTA of the row group][Rp]: c, s, t
    float* seg_max;    // [Rp][segments], null: no alternatives
    float* scores;     // [segment][Rp][32]
    int segs, top_n;
    uint32_t* bound;   // [Rp]: see Bound, zero between calls
    uint32_t* seen;    // [kMaxGroups]: epilogue warps that have left their first tile's maxima
    unsigned int* err;
};

// A row group: hidden rows [begin, end) of the pass.
struct Rows {
    int group, begin, end;
};

__host__ __device__ constexpr size_t smem_bytes(int stages, int nmax) {
    return 1024 + (size_t)stages * (kStageW + (size_t)nmax * kBlockK * 2) + sizeof(Bars) + kEpiWarps * kTransBytes + 64;
}

// ---------------------------------------------------------------------------
// Which blocks of scores are kept for the alternatives.  Each epilogue warp
// counts itself in `seen` once the maxima of its first tile are written.  A
// warp of its own in every CTA looks at the count; when all have counted, the
// CTAs of the row group share out the hidden rows, and each finds a
// value that n of a row's first maxima reach: blocks whose maximum is below it need not be written any more.  At 248,320 head rows that
// leaves about a sixth of the scores to write.  The epilogue never waits for a
// bound: it reads what the CTA has so far from shared memory (0 = none).  In a
// warp of the epilogue itself the same search cost the 64-row call 8 us.
// The bound is rounded down to 16 bits of the ordered float.

constexpr int kFirstSegs = 1024;
constexpr int kMinFirstSegs = 64;   // so that each of the 64 groups below has one
constexpr int kTries = 256;         // looks at the count, and at the bounds
constexpr unsigned int kTryNs = 500;

// A value that n <= 32 of the m <= kFirstSegs values p[0..m) reach, by one warp, as ord_f32 rounded down: the n-th
// largest maximum of 64 groups of them (two per lane).
__device__ __forceinline__ uint32_t nth_largest(const float* p, int m, int n) {
    const int lane = threadIdx.x & 31;
    float x[kFirstSegs / 32];
#pragma unroll
    for (int i = 0; i < kFirstSegs / 32; ++i) x[i] = i * 32 + lane < m ? __ldcg(p + i * 32 + lane) : quiet_nan();
    float lo = x[0], hi = x[1];
#pragma unroll
    for (int i = 2; i < kFirstSegs / 32; i += 2) {
        lo = fmaxf(lo, x[i]);
        hi = fmaxf(hi, x[i + 1]);
    }
    const uint32_t a = lo == lo ? ord_f32(lo) >> 16 : 0u, b = hi == hi ? ord_f32(hi) >> 16 : 0u;  // NaN: no value
    uint32_t t = 0u;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
        const uint32_t u = t | (1u << bit);
        const int c = __popc(__ballot_sync(0xFFFFFFFFu, a >= u)) + __popc(__ballot_sync(0xFFFFFFFFu, b >= u));
        t = c >= n ? u : t;
    }
    return t << 16;
}

// The bounds of a row group, by one warp of each of its n_cta CTAs; `first_segs`: the segments of their first tiles.
// bounds: the CTA's copy (shared, zero at the start); *done: the CTA's epilogue has finished.
__device__ __forceinline__ void find_bounds(const Args& a, const Rows& rw, int cta, int n_cta, int first_segs,
                                            volatile uint32_t* bounds, volatile uint32_t* done) {
    first_segs = min(first_segs, kFirstSegs);
    // no later tiles (this CTA's, at least), or too few maxima
    if (a.seg_max == nullptr || first_segs >= a.segs || first_segs < kMinFirstSegs) return;
    const int lane = threadIdx.x & 31;
    const int row0 = rw.begin, rows = rw.end - rw.begin;
    volatile uint32_t* seen = a.seen + rw.group;
    volatile uint32_t* shared = a.bound + row0;
    bool all = false;
    for (int i = 0; i < kTries && !all && *done == 0u; ++i) {
        if (i > 0) __nanosleep(kTryNs);
        all = __shfl_sync(0xFFFFFFFFu, lane == 0 ? *seen : 0u, 0) == (uint32_t)(kEpiWarps * n_cta);
    }
    if (!all) return;
    __threadfence();  // lane 0 saw the count: what the epilogue warps wrote before is then seen by all lanes
    __syncwarp();
    for (int r = cta; r < rows; r += n_cta) {
        const uint32_t b = nth_largest(a.seg_max + (size_t)(row0 + r) * a.segs, first_segs, a.top_n);
        if (lane == 0) shared[r] = b;
    }
    all = false;
    for (int i = 0; i < kTries && !all && *done == 0u; ++i) {
        if (i > 0) __nanosleep(kTryNs);
        bool have = true;
        for (int r = lane; r < rows; r += 32) {
            const uint32_t b = shared[r];
            bounds[r] = b;
            have = have && b != 0u;
        }
        all = __all_sync(0xFFFFFFFFu, have);
    }
}

// ---------------------------------------------------------------------------
// Epilogue of one warp: blocks `half`, half + 2, ... of 32 hidden rows (row = begin + 32 block + lane), NB at most.
// A block is turned in shared memory; 16-byte pieces of hidden row j lie at piece p ^ (j % 8), so that the rows are
// written (lane = head row) and read (lane = hidden row, four floats) without bank conflicts.

template <int NB>
struct Epilogue {
    Stat st[NB];
    int tok[NB];
    float* tr;
    int half;
    volatile uint32_t* bounds;  // of the row group's rows

    __device__ __forceinline__ static int place(int j, int c) { return j * 32 + ((((c >> 2) ^ j) & 7) << 2 | (c & 3)); }

    __device__ __forceinline__ void begin(const Args& a, const Rows& rw, float* tr_, int half_, volatile uint32_t* bounds_) {
        tr = tr_;
        half = half_;
        bounds = bounds_;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int row = rw.begin + (2 * k + half) * 32 + lane;
            st[k] = stat_none();
            tok[k] = (a.tokens != nullptr && row < rw.end) ? a.tokens[row] : -1;
        }
    }

    // After the warp's first tile: its maxima are there (see find_bounds).
    __device__ __forceinline__ void first_done(const Args& a, const Rows& rw) {
        if (a.seg_max == nullptr) return;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) rows_take_ticket(a.seen + rw.group);
    }

    // v[j]: the score of head row v0 + lane for hidden row j of this warp's k-th block.
    __device__ __forceinline__ void block(const Args& a, const Rows& rw, int k, int v0, const float (&v)[32]) {
        const int lane = threadIdx.x & 31;
        const int in_group = (2 * k + half) * 32 + lane, row = rw.begin + in_group;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) tr[place(j, lane)] = v[j];
        __syncwarp();
        float x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(tr + place(lane, 4 * i));
            x[4 * i] = q.x;
            x[4 * i + 1] = q.y;
            x[4 * i + 2] = q.z;
            x[4 * i + 3] = q.w;
        }
        const int n = a.V - v0;  // head rows of this block
        const unsigned int at = (unsigned int)(tok[k] - v0);
        if (at < 32u && (int)at < n && row < rw.end) a.tok_score[row] = tr[place(lane, (int)at)];
        if (n < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i >= n) x[i] = neg_inf();
        }
        float m = neg_inf();
#pragma unroll
        for (int i = 0; i < 32; ++i) m = fmaxf(m, x[i]);
        if (a.seg_max != nullptr) {
            const int seg = v0 / kSeg;
            if (row < rw.end && vh_guard(seg < a.segs, a.err)) a.seg_max[(size_t)row * a.segs + seg] = m;
            // rows whose scores are kept: 128 bytes each, lane = head row again
            const uint32_t keep = __ballot_sync(0xFFFFFFFFu, row < rw.end && ord_f32(m) >= bounds[in_group]);
            float* p = a.scores + ((size_t)seg * a.Rp + row - lane) * kSeg + lane;
            if (keep != 0u) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if ((keep >> j) & 1u) p[j * kSeg] = v[j];
            }
        }
        Stat2 run{st[k].c, f2(st[k].s, 0.f), f2(st[k].t, 0.f)};
        run.raise(m);
        if (fabsf(run.c) < kFar) {
            const F2 mcl = run.minus_cl();
#pragma unroll
            for (int i = 0; i < 32; i += 2) run.add_plain(fmaxf(x[i], kLift), fmaxf(x[i + 1], kLift), mcl);
        } else if (run.c != neg_inf()) {
#pragma unroll 1
            for (int i = 0; i < n && i < 32; i += 2)
                run.add_far(tr[place(lane, i)], i + 1 < n ? tr[place(lane, i + 1)] : neg_inf());
        }
        st[k] = run.get();
    }

    // The accumulators of one tile, of whose 32 lanes (`taddr`: the first one's) lane 0 is head row v0; `free` hands
    // them back once this warp has read its blocks of them.
    template <typename Free>
    __device__ __forceinline__ void tile(const Args& a, const Rows& rw, uint32_t taddr, int v0, Free free) {
        const int blocks = (a.N + 31) / 32;
        if (half >= blocks) free();
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int g = 2 * k + half;
            if (g < blocks) {
                float v[32];
                tmem_ld32(taddr + g * 32u, v);
                if (g + 2 >= blocks) free();
                if (v0 < a.V && rw.begin + g * 32 < rw.end) block(a, rw, k, v0, v);
            }
        }
    }

    // The warp's statistics of its hidden rows, for the CTA to join.
    __device__ __forceinline__ void leave() {
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            float* p = tr + (k * 32 + lane) * 3;
            p[0] = st[k].c;
            p[1] = st[k].s;
            p[2] = st[k].t;
        }
    }
};

// The transposition buffer of the epilogue warp of a lane quarter and a half of the blocks.
__device__ __forceinline__ float* trans_of(float* trans, int quarter, int half) {
    return trans + (half * 4 + quarter) * (kTransBytes / 4);
}

// After __syncthreads: join the four quarters' statistics of the group's rows.
__device__ __forceinline__ void publish(const Args& a, const Rows& rw, float* trans, int slot) {
    for (int r = threadIdx.x; r < rw.end - rw.begin; r += blockDim.x) {
        const int g = r >> 5;
        Stat s = stat_none();
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float* p = trans_of(trans, w, g & 1) + ((g >> 1) * 32 + (r & 31)) * 3;
            s = stat_join(s, Stat{p[0], p[1], p[2]});
        }
        a.part[(size_t)slot * a.Rp + rw.begin + r] = make_float4(s.c, s.s, s.t, 0.f);
    }
}

__device__ __forceinline__ void init_bars(Bars* b, int stages, int empty_arrivals) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&b->full[s], 1);
            mbar_init(&b->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b->tmem_full[i], 1);
            mbar_init(&b->tmem_empty[i], empty_arrivals);
        }
        mbar_init(&b->mma_done, 1);
        ptx::fence_barrier_init();
        b->done = 0u;
    }
    for (int i = threadIdx.x; i < kGroup; i += blockDim.x) b->bounds[i] = 0u;
}

// ---------------------------------------------------------------------------
// Up to 128 hidden rows: one CTA per tile.  Warp 0 = TMA producer, warp 1 =
// TMEM owner and MMA issuer, warps 2..9 = epilogue (TMEM lane quarter = warp % 4),
// warp 10 = the alternatives' bounds.

template <int STAGES, int NMAX>
__global__ void __launch_bounds__(kThreadsH, 1)
    k_head_logprobs(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
    constexpr int kStageX = NMAX * kBlockK * 2;
    constexpr int NB = (NMAX / 32 + 1) / 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stage_w = smem;
    uint8_t* stage_x = smem + (size_t)STAGES * kStageW;
    float* trans = reinterpret_cast<float*>(stage_x + (size_t)STAGES * kStageX);
    Bars* bars = reinterpret_cast<Bars*>(reinterpret_cast<uint8_t*>(trans) + kEpiWarps * kTransBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k_stages = (a.H + kBlockK - 1) / kBlockK;  // TMA fills past H with zeros
    const int n_tiles = (a.V + kTileM - 1) / kTileM;

    const Rows rw{0, 0, a.R};
    init_bars(bars, STAGES, kEpiWarps);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    rows_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            // The head is read before the previous kernel is waited for, everything else after.
            const unsigned long long pol_w = policy_evict_first(), pol_x = policy_evict_last();
            uint32_t it = 0;
            bool ok = true, waited = false;
            auto release_first_ring = [&](uint32_t n) {
                rows_wait();
                rows_fence_async();
                for (uint32_t j = 0; j < n; ++j)
                    tma_load_2d(stage_x + (size_t)j * kStageX, &map_x, &bars->full[j], (int)(j % k_stages) * kBlockK, 0,
                                pol_x);
                waited = true;
            };
            for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
                for (int ks = 0; ks < k_stages; ++ks, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&bars->empty[s], ((it / STAGES) & 1u) ^ 1u, a.err)) { ok = false; break; }
                    mbar_arrive_expect_tx(&bars->full[s], (uint32_t)(kStageW + a.N * kBlockK * 2));
                    tma_load_2d(stage_w + (size_t)s * kStageW, &map_w, &bars->full[s], ks * kBlockK, tile * kTileM, pol_w);
                    if (waited)
                        tma_load_2d(stage_x + (size_t)s * kStageX, &map_x, &bars->full[s], ks * kBlockK, 0, pol_x);
                    else if (it + 1 == (uint32_t)STAGES)
                        release_first_ring(it + 1);
                }
            }
            if (!waited) release_first_ring(it);
            for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0); j < it; ++j)
                mbar_drain(&bars->full[j % STAGES], (j / STAGES) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(kTileM, a.N);
            uint32_t it = 0, local = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++local) {
                const uint32_t buf = local & 1u;
                if (!mbar_wait(&bars->tmem_empty[buf], ((local >> 1) & 1u) ^ 1u, a.err)) break;
                tc_fence_after();
                for (int ks = 0; ks < k_stages; ++ks, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&bars->full[s], (it / STAGES) & 1u, a.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = smem_u32(stage_w + (size_t)s * kStageW);
                    const uint32_t sx = smem_u32(stage_x + (size_t)s * kStageX);
#pragma unroll
                    for (int kk = 0; kk < kBlockK / 16; ++kk)
                        mma_bf16(tmem_base + buf * 256u, smem_desc_sw128(sw + kk * 32), smem_desc_sw128(sx + kk * 32),
                                 idesc, (ks > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&bars->empty[s]);
                }
                if (ok) mma_commit(&bars->tmem_full[buf]);
            }
            mma_commit(&bars->mma_done);
            mbar_drain(&bars->mma_done, 0u);
        }
    } else if (warp == kBoundWarp) {
        rows_wait();
        find_bounds(a, rw, blockIdx.x, gridDim.x, (int)gridDim.x * (kTileM / kSeg), bars->bounds, &bars->done);
    } else {
        rows_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        Epilogue<NB> ep;
        ep.begin(a, rw, trans_of(trans, quarter, half), half, bars->bounds);
        uint32_t local = 0;
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++local) {
            const uint32_t buf = local & 1u;
            if (!mbar_wait(&bars->tmem_full[buf], (local >> 1) & 1u, a.err)) break;
            tc_fence_after();
            ep.tile(a, rw, tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * 256u, tile * kTileM + quarter * 32, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tmem_empty[buf]);
            });
            if (local == 0) ep.first_done(a, rw);
        }
        ep.leave();
        *const_cast<volatile uint32_t*>(&bars->done) = 1u;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                     : "memory");
    }
    rows_wait();
    publish(a, rw, trans, blockIdx.x);
}

// ---------------------------------------------------------------------------
// More hidden rows: CTA pairs.  Each CTA stages its 128 head rows and half of
// the row group's hidden rows; the leader issues the MMAs; each CTA's TMEM
// holds the accumulators of its own head rows.

constexpr int kStages2 = 6;
constexpr int kStageX2 = 128 * kBlockK * 2;

__global__ void __launch_bounds__(kThreadsH, 1)
    k_head_logprobs_pair(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                         const Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stage_w = smem;
    uint8_t* stage_x = smem + (size_t)kStages2 * kStageW;
    float* trans = reinterpret_cast<float*>(stage_x + (size_t)kStages2 * kStageX2);
    Bars* bars = reinterpret_cast<Bars*>(reinterpret_cast<uint8_t*>(trans) + kEpiWarps * kTransBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int group = pair % a.groups, row0 = group * a.N;
    const Rows rw{group, row0, min(row0 + a.N, a.R)};
    const int tile0 = pair / a.groups, step = (int)(gridDim.x >> 1) / a.groups;
    const int n_tiles = (a.V + kPairTile - 1) / kPairTile;
    const int k_stages = (a.H + kBlockK - 1) / kBlockK;

    init_bars(bars, kStages2, 2 * kEpiWarps);  // of both CTAs
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    rows_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            const unsigned long long pol_w = policy_evict_first(), pol_x = policy_evict_last();
            uint32_t it = 0;
            bool ok = true, waited = false;
            auto load_x = [&](uint32_t j) {
                const int s = j % kStages2;
                tma_load_2d_pair(stage_x + (size_t)s * kStageX2, &map_x, map_to_rank(smem_u32(&bars->full[s]), 0),
                                 (int)(j % k_stages) * kBlockK, row0 + (int)rank * (a.N / 2), pol_x);
            };
            auto release_first_ring = [&](uint32_t n) {
                rows_wait();
                rows_fence_async();
                for (uint32_t j = 0; j < n; ++j) load_x(j);
                waited = true;
            };
            for (int tile = tile0; tile < n_tiles && ok; tile += step) {
                for (int ks = 0; ks < k_stages; ++ks, ++it) {
                    const int s = it % kStages2;
                    if (!mbar_wait(&bars->empty[s], ((it / kStages2) & 1u) ^ 1u, a.err)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(&bars->full[s], 2u * kStageW + (uint32_t)(a.N * kBlockK * 2));
                    tma_load_2d_pair(stage_w + (size_t)s * kStageW, &map_w, map_to_rank(smem_u32(&bars->full[s]), 0),
                                     ks * kBlockK, tile * kPairTile + (int)rank * kTileM, pol_w);
                    if (waited)
                        load_x(it);
                    else if (it + 1 == (uint32_t)kStages2)
                        release_first_ring(it + 1);
                }
            }
            if (!waited) release_first_ring(it);
            if (leader)  // the leader's barriers see both CTAs' loads
                for (uint32_t j = (it > (uint32_t)kStages2 ? it - kStages2 : 0); j < it; ++j)
                    mbar_drain(&bars->full[j % kStages2], (j / kStages2) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            const uint32_t idesc = idesc_bf16(kPairTile, a.N);
            uint32_t it = 0, local = 0;
            bool ok = true;
            for (int tile = tile0; tile < n_tiles && ok; tile += step, ++local) {
                const uint32_t buf = local & 1u;
                if (!mbar_wait(&bars->tmem_empty[buf], ((local >> 1) & 1u) ^ 1u, a.err)) break;
                tc_fence_after();
                for (int ks = 0; ks < k_stages; ++ks, ++it) {
                    const int s = it % kStages2;
                    if (!mbar_wait(&bars->full[s], (it / kStages2) & 1u, a.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = smem_u32(stage_w + (size_t)s * kStageW);
                    const uint32_t sx = smem_u32(stage_x + (size_t)s * kStageX2);
#pragma unroll
                    for (int kk = 0; kk < kBlockK / 16; ++kk)
                        mma_bf16_pair(tmem_base + buf * 256u, smem_desc_sw128(sw + kk * 32),
                                      smem_desc_sw128(sx + kk * 32), idesc, (ks > 0 || kk > 0) ? 1u : 0u);
                    mma_commit_pair(&bars->empty[s]);
                }
                if (ok) mma_commit_pair(&bars->tmem_full[buf]);
            }
            mma_commit_pair(&bars->mma_done);
            mbar_drain(&bars->mma_done, 0u);
        }
    } else if (warp == kBoundWarp) {
        rows_wait();
        find_bounds(a, rw, tile0 * 2 + (int)rank, step * 2, step * (kPairTile / kSeg), bars->bounds, &bars->done);
    } else {
        rows_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        Epilogue<kGroup / 64> ep;
        ep.begin(a, rw, trans_of(trans, quarter, half), half, bars->bounds);
        const uint32_t empty0 = map_to_rank(smem_u32(&bars->tmem_empty[0]), 0);
        const uint32_t empty1 = map_to_rank(smem_u32(&bars->tmem_empty[1]), 0);
        uint32_t local = 0;
        for (int tile = tile0; tile < n_tiles; tile += step, ++local) {
            const uint32_t buf = local & 1u;
            if (!mbar_wait(&bars->tmem_full[buf], (local >> 1) & 1u, a.err)) break;
            tc_fence_after();
            ep.tile(a, rw, tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * 256u,
                    tile * kPairTile + (int)rank * kTileM + quarter * 32, [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(buf ? empty1 : empty0);
                    });
            if (local == 0) ep.first_done(a, rw);
        }
        ep.leave();
        *const_cast<volatile uint32_t*>(&bars->done) = 1u;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                     : "memory");
    }
    rows_wait();
    publish(a, rw, trans, tile0 * 2 + (int)rank);
}

// ---------------------------------------------------------------------------
// One CTA per hidden row: join the statistics, pick the alternatives.

constexpr int kThreadsF = kSelThreads;

struct FinishArgs {
    int Rp, V, n_parts, segs, top_n;
    bool signal;  // no ids are written, or this call's next pass follows
    const int32_t* tokens;
    const float* tok_score;
    const float4* part;
    const float* seg_max;
    const float* scores;
    uint32_t* bound;
    uint32_t* seen;
    float *logprob, *entropy, *lse;
    int32_t* top_ids;
    float* top_logprobs;
};

// A row's blocks of scores for select_top.
struct Blocks {
    static constexpr bool kLane = false;
    using Item = float;
    const FinishArgs& a;
    int row;
    __device__ __forceinline__ float max(int g) const { return a.seg_max[(size_t)row * a.segs + g]; }
    __device__ __forceinline__ float load(int g) const {
        return a.scores[((size_t)g * a.Rp + row) * kSeg + (threadIdx.x & 31)];
    }
    __device__ __forceinline__ float peak(float x) const { return fmaxf(x, neg_inf()); }
    template <typename F>
    __device__ __forceinline__ void each(float x, int g, float b, F take) const {
        const long long v = (long long)g * kSeg + (threadIdx.x & 31);
        if (!(x < b) && v < a.V) take(make_key(x, (uint32_t)v));
    }
    static constexpr int kBatches = 1;
    __device__ __forceinline__ unsigned long long key(int g, int) const {
        const long long v = (long long)g * kSeg + (threadIdx.x & 31);
        return v < a.V ? make_key(load(g), (uint32_t)v) : 0ull;
    }
};

__global__ void __launch_bounds__(kThreadsF) k_head_logprobs_finish(const FinishArgs a) {
    constexpr int kHeld = 5;  // shares of the statistics a lane of the joining warp loads at once (152 CTAs)
    constexpr int kJoiner = kSelWarps - 1;
    __shared__ SelectSmem s_sel;
    __shared__ RowStat s_rs;
    if (a.signal) rows_launch_dependents();
    rows_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x;
    float4 p[kHeld];
    const int tok = a.tokens != nullptr ? a.tokens[row] : -1;
    const bool given = tok >= 0 && tok < a.V;
    const float tok_score = given ? a.tok_score[row] : 0.f;
    if (warp == kJoiner) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int q = i * 32 + lane;
            p[i] = q < a.n_parts ? a.part[(size_t)q * a.Rp + row] : make_float4(neg_inf(), 0.f, 0.f, 0.f);
        }
    }
    auto join = [&] {
        Stat st = stat_none();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) st = stat_join(st, Stat{p[i].x, p[i].y, p[i].z});
        for (int q = kHeld * 32 + lane; q < a.n_parts; q += 32) {
            const float4 o = a.part[(size_t)q * a.Rp + row];
            st = stat_join(st, Stat{o.x, o.y, o.z});
        }
        const RowStat rs = stat_finish(stat_warp(st));
        if (lane == 0) {
            s_rs = rs;
            if (a.logprob != nullptr) a.logprob[row] = given ? stat_logprob(rs, tok_score) : 0.f;
            if (a.entropy != nullptr) a.entropy[row] = rs.entropy;
            if (a.lse != nullptr) a.lse[row] = rs.lse;
        }
    };
    if (a.top_n == 0) {
        if (warp == kJoiner) join();
        return;
    }
    const uint32_t floor = a.bound[row];
    select_top<32>(s_sel, a.segs, a.top_n, floor, Blocks{a, row}, join, [&](int i, unsigned long long k) {
        const size_t o = (size_t)row * a.top_n + i;
        a.top_ids[o] = k != 0ull ? (int32_t)key_gid(k) : -1;
        a.top_logprobs[o] = k != 0ull ? stat_logprob(s_rs, key_score(k)) : neg_inf();
    });
    if (threadIdx.x == 0) {  // for the next call
        a.bound[row] = 0u;
        if (row < kMaxGroups) a.seen[row] = 0u;
    }
}

// ---------------------------------------------------------------------------

struct Layout {
    int Rp, segs;
    size_t tok, part, seg_max, scores, total;
};
// Bounds and counts at a fixed place, so that a workspace serves calls of any size.
constexpr size_t kBoundAt = kWsHeaderBytes + kMaxGroups * 4;
constexpr size_t kZeroed = 8192;
static_assert(kBoundAt + (size_t)kPassRows * 4 <= kZeroed, "zeroed part of the workspace");
static Layout layout(int R, int V, int top_n) {
    Layout l;
    l.Rp = (std::min(R, kPassRows) + 31) / 32 * 32;
    l.segs = (int)(((long long)V + kSeg - 1) / kSeg);
    l.tok = kZeroed;
    l.part = l.tok + (size_t)l.Rp * 4;
    l.seg_max = l.part + (size_t)kMaxParts * l.Rp * 16;
    l.scores = l.seg_max + (top_n > 0 ? (size_t)l.segs * l.Rp * 4 : 0);
    l.total = l.scores + (top_n > 0 ? (size_t)l.segs * l.Rp * kSeg * 4 : 0);
    return l;
}

template <typename K>
static cudaError_t launch_tc(K kernel, int grid, size_t smem, int cluster, cudaStream_t s, const CUtensorMap& mw,
                             const CUtensorMap& mx, const Args& a) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreadsH);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mw, mx, a);
}

// CTA pairs that are resident at once, per device.
static int resident_pairs() {
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    int n = cache[dev & 63].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const size_t smem = smem_bytes(kStages2, 128);
    if (cudaFuncSetAttribute(k_head_logprobs_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
    cfg.blockDim = dim3(kThreadsH);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_head_logprobs_pair, &cfg) != cudaSuccess) return 0;
    cache[dev & 63].store(n, std::memory_order_relaxed);
    return n;
}

// One pass over the head for nr <= kPassRows hidden rows.
static cudaError_t pass(const HeadLogprobArgs& h, int r0, int nr, cudaStream_t s) {
    const Layout l = layout(h.R, h.V, h.top_n);
    uint8_t* base = static_cast<uint8_t*>(h.ws);
    Args a{};
    a.R = nr;
    a.Rp = l.Rp;
    a.H = h.H;
    a.V = h.V;
    a.tokens = h.tokens ? h.tokens + r0 : nullptr;
    a.tok_score = reinterpret_cast<float*>(base + l.tok);
    a.part = reinterpret_cast<float4*>(base + l.part);
    a.seg_max = h.top_n > 0 ? reinterpret_cast<float*>(base + l.seg_max) : nullptr;
    a.scores = reinterpret_cast<float*>(base + l.scores);
    a.segs = l.segs;
    a.top_n = h.top_n;
    a.seen = reinterpret_cast<uint32_t*>(base + kWsHeaderBytes);
    a.bound = reinterpret_cast<uint32_t*>(base + kBoundAt);
    a.err = reinterpret_cast<unsigned int*>(base + kWsErrorOffset);
    const uint16_t* x = h.x + (size_t)r0 * h.H;
    alignas(64) CUtensorMap mw, mx;
    if (!make_map(&mw, h.W, h.V, h.H, kTileM)) return cudaErrorNotSupported;
    int n_parts;
    cudaError_t e;
    if (nr <= kOneCtaRows) {
        a.N = (nr + 15) / 16 * 16;
        if (!make_map(&mx, x, nr, h.H, a.N)) return cudaErrorNotSupported;
        n_parts = std::min({sm_count(), (int)(((long long)h.V + kTileM - 1) / kTileM), kMaxParts});
        e = a.N <= 64 ? launch_tc(k_head_logprobs<8, 64>, n_parts, smem_bytes(8, 64), 1, s, mw, mx, a)
                      : launch_tc(k_head_logprobs<6, 128>, n_parts, smem_bytes(6, 128), 1, s, mw, mx, a);
    } else {
        // groups of even size: the MMA's time goes with N (369 rows of 137,667 x 2560: 219 us in two groups of 192, 237 us
        // in groups of 256)
        a.groups = (nr + kGroup - 1) / kGroup;
        a.N = ((nr + a.groups - 1) / a.groups + 15) / 16 * 16;
        if (!make_map(&mx, x, nr, h.H, a.N / 2)) return cudaErrorNotSupported;
        const int pairs = resident_pairs();
        const int tiles = (int)(((long long)h.V + kPairTile - 1) / kPairTile);
        const int per = std::min({pairs / a.groups, tiles, kMaxParts / 2});  // pairs of one row group
        if (per < 1) return cudaErrorNotSupported;
        n_parts = 2 * per;
        e = launch_tc(k_head_logprobs_pair, 2 * per * a.groups, smem_bytes(kStages2, 128), 2, s, mw, mx, a);
    }
    if (e != cudaSuccess) return e;
    FinishArgs f{};
    f.Rp = l.Rp;
    f.V = h.V;
    f.n_parts = n_parts;
    f.segs = l.segs;
    f.top_n = h.top_n;
    f.signal = h.top_n == 0 || r0 + nr < h.R;
    f.tokens = a.tokens;
    f.tok_score = a.tok_score;
    f.part = a.part;
    f.seg_max = a.seg_max;
    f.scores = a.scores;
    f.seen = a.seen;
    f.bound = a.bound;
    f.logprob = h.logprob ? h.logprob + r0 : nullptr;
    f.entropy = h.entropy ? h.entropy + r0 : nullptr;
    f.lse = h.lse ? h.lse + r0 : nullptr;
    f.top_ids = h.top_ids ? h.top_ids + (size_t)r0 * h.top_n : nullptr;
    f.top_logprobs = h.top_logprobs ? h.top_logprobs + (size_t)r0 * h.top_n : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nr);
    cfg.blockDim = dim3(kThreadsF);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_head_logprobs_finish, f);
}

}  // namespace hlp

size_t head_logprobs_ws_bytes(int R, int V, int top_n) { return hlp::layout(R, V, top_n).total; }

cudaError_t launch_head_logprobs(const HeadLogprobArgs& a, cudaStream_t s) {
    for (int r0 = 0; r0 < a.R; r0 += hlp::kPassRows) {
        const cudaError_t e = hlp::pass(a, r0, std::min(hlp::kPassRows, a.R - r0), s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace vh
