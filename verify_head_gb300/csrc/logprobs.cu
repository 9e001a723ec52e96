// Log probabilities of given tokens from logits, with the entropy of each row
// and its largest alternatives, and the gradient.
//
//     lse = log sum_v e^x_v      logprob = x_token - lse      entropy = lse - sum_v p_v x_v
//     dx_v = g_lp ([v = token] - p_v) - g_ent p_v (log p_v + entropy)
//
// Forward: one pass over the logits.  A row is cut into slots of 32 aligned
// bytes and segments of 32 slots (one warp load of 1 KiB).  Each thread keeps
// a running maximum and the two sums of Stat; where alternatives are wanted
// the maxima of segments, or of slots, are written too, and one CTA per row
// picks the alternatives from the units with the largest maxima (select_top),
// reading about n units again.
//
// Rows are cut into pieces for about one resident wave of CTAs, or all rows'
// segments are shared out evenly over it (see plan).  A row of several pieces
// meets in the workspace, where the last of its CTAs (a ticket, left zero
// again) finishes it, the choice included (129 x 40001 fp16 with 5
// alternatives: 10.5 us, against 11.5 us with the choice in a second kernel;
// 9.6 us since the statistics are joined while the listed units are read).
// With even ranges a CTA may be the last one of two rows and more: then the
// choice is a second kernel's.
//
// Bound: memory (the logits once; the gradient also writes them once).
#include <algorithm>

#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace lp {

constexpr int kThreadsL = kSelThreads;
constexpr int kWarpsL = kThreadsL / 32;
constexpr int kUnroll = 2;             // segments in flight per warp (and two more requested); three: 50.1 us for the same
// CTAs per SM.  Four for statistics alone (2048 x 65536 bf16: 46.9 against 48.1 us with three); with alternatives
// the rows are few and three, with more registers each, are faster (129 x 40001 fp16, 5 of them, with even ranges: 12.7 against 13.2 us).
constexpr int kPerSm = 4, kPerSmTop = 3;
constexpr int kTargetCtas = 152 * kPerSm;
constexpr int kMinSegs = 2 * kWarpsL;  // segments per CTA below which the work is not cut further
constexpr int kShortSegs = 64;         // segments per CTA up to which a call is short
constexpr int kWholeSegs = 64, kRowSegs = 129;  // see plan

// A row as aligned 32-byte slots: slot v holds elements [v * kSlot - shift, +kSlot).
constexpr int kSlotBytes = 32;
template <typename T>
constexpr int kSlot = kSlotBytes / (int)sizeof(T);
template <typename T>
struct Row {
    const uint8_t* base;  // row address rounded down to 32 bytes
    int shift;            // elements before the row's first one in slot 0
    int V;
    __device__ __forceinline__ Row(const T* p, int V_) : V(V_) {
        const uintptr_t u = reinterpret_cast<uintptr_t>(p);
        base = reinterpret_cast<const uint8_t*>(u & ~uintptr_t(kSlotBytes - 1));
        shift = (int)((u & (kSlotBytes - 1)) / sizeof(T));
    }
    __device__ __forceinline__ int slots() const { return (int)(((long long)V + shift + kSlot<T> - 1) / kSlot<T>); }
    __device__ __forceinline__ long long first(int slot) const { return (long long)slot * kSlot<T> - shift; }
    // Elements of a slot; places outside the row (and whole slots past the end) read as -inf.
    __device__ __forceinline__ void load(int slot, RawVec<T, kSlot<T>>& r) const {
        const long long e0 = first(slot);
        if (e0 >= 0 && e0 + kSlot<T> <= V) {
            r.load(reinterpret_cast<const T*>(base + (size_t)slot * kSlotBytes));
        } else {
            const T* p = reinterpret_cast<const T*>(base) + (long long)slot * kSlot<T>;
            r.fill_lowest();
#pragma unroll
            for (int i = 0; i < kSlot<T>; ++i)
                if (e0 + i >= 0 && e0 + i < V) r.put(i, p[i]);
        }
    }
};

// A row's units for select_top: segments, or single slots.
template <typename T, bool SLOTS>
struct RowUnits {
    static constexpr bool kLane = SLOTS;
    using Item = RawVec<T, kSlot<T>>;
    const Row<T>& x;
    const float* maxima;
    __device__ __forceinline__ int slot(int g) const { return SLOTS ? g : g * 32 + (threadIdx.x & 31); }
    __device__ __forceinline__ float max(int g) const { return __ldcg(maxima + g); }
    __device__ __forceinline__ Item load(int g) const {
        Item it;
        x.load(slot(g), it);
        return it;
    }
    __device__ __forceinline__ float peak(const Item& it) const { return it.max(); }
    template <typename F>
    __device__ __forceinline__ void each(const Item& it, int g, float b, F take) const {
        const long long e0 = x.first(slot(g));
#pragma unroll
        for (int j = 0; j < kSlot<T>; ++j)
            if (!(it.get(j) < b) && e0 + j >= 0 && e0 + j < x.V) take(make_key(it.get(j), (uint32_t)(e0 + j)));
    }
    static constexpr int kBatches = SLOTS ? 1 : kSlot<T>;
    __device__ __forceinline__ unsigned long long key(int g, int i) const {
        const int lane = threadIdx.x & 31;
        const long long e = x.first(SLOTS ? g : g * 32) + i * 32 + lane;
        if (e < 0 || e >= x.V || (SLOTS && lane >= kSlot<T>)) return 0ull;
        return make_key(to_f32((reinterpret_cast<const T*>(x.base) + x.shift)[e]), (uint32_t)e);
    }
};

// Upper bound of the segments of a row of V elements of `size` bytes, whatever its alignment: what the call's rows are
// counted by.  It is one more than an aligned row of whole segments has (65 for 32,768 elements of 16 bits, 129 for 65,536).
__host__ __device__ inline int max_segs(int V, int size) {
    const long long per = 32 * kSlotBytes / size;
    return (int)(((long long)V + kSlotBytes / size - 1 + per - 1) / per);
}

// The call's units are the R x segs segments, cut into one range per CTA: every CTA has the same work to within a
// segment, whatever R and V.  A range holds whole rows and, at its ends, pieces of rows that other CTAs share.
// Rows of up to kSlotSegs segments keep the maximum of every slot for the alternatives, longer ones that of every
// segment: there have to be clearly more units than alternatives.  At the limit the two cost the same (64 to 300 rows of
// 131,072 bf16 and 1024 of 65,536 fp32, of 257 segments each, with 20 alternatives: within 2% either way).
constexpr int kSlotSegs = 256;
__host__ __device__ inline int row_units(int row_segs) { return row_segs <= kSlotSegs ? row_segs * 32 : row_segs; }

struct Ws {
    unsigned int* ticket;  // [kTargetCtas], zero between calls: by the first CTA of a shared row
    float4* part;          // [kTargetCtas][2]: c, s, t of the CTA's first piece of a row begun before it, and of its last
    float* unit_max;       // [R][row_units], alternatives only
    float4* row;           // [R]: c, s, t of rows that are not shared, alternatives only
};
constexpr size_t kTicketEnd = kWsHeaderBytes + (size_t)kTargetCtas * 4;
constexpr size_t kPartEnd = kTicketEnd + (size_t)kTargetCtas * 2 * 16;

// The CTAs of the scan, and into how many pieces each row is cut (0: the units are, whatever the rows).
// With pieces of rows a CTA finishes one row or piece; with even ranges up to two pieces and the rows between them, one
// after the other, but all CTAs have the same work.  So rows are cut for short calls (231 x 32768 bf16: 7.9 against
// 10.0 us) and where that fills three quarters of the SMs' places (600 x 65536: 14.6 against 18.9 us; with half of
// them, 310 x 131072, 23.8 against 19.0 us).
// More rows than places: a CTA each up to kRowSegs segments, which rows of 65,536 elements of 16 bits have (1645 x 32768:
// 21.9 against 24.5 us, 1024 x 65536: 25.9 against 27.7 us, 2048 x 65536: 46.1 against 47.3 us; 610 x 65536, hardly more
// rows than places, 19.6 against 18.9 us), even ranges above, where a last wave of few CTAs would weigh more; with
// alternatives, whose calls write every unit's maximum, even ranges (1645 x 32768: 39.8 against 40.2 us).
// The last piece's CTA joins a row, which takes 1.2 us: rows of up to kWholeSegs segments stay whole (44 x 21479: 4.5
// against 5.7 us; whole rows of 65 segments, 32,768 bf16: 231 rows 9.0 against 8.2 us cut, 304 rows 6.6 against 8.1 us,
// 16 rows 5.0 against 4.8 us).
inline void plan(int R, int segs, bool top, int& n, int& k) {
    const long long units = (long long)R * segs;
    const int wave = 152 * (top ? kPerSmTop : kPerSm);
    k = segs > kWholeSegs ? std::max(1, std::min(wave / R, segs / kMinSegs)) : 1;
    n = R * k;
    if (R > wave && !top && segs <= kRowSegs) return;
    if (R > wave || (units > (long long)wave * kShortSegs && n < wave / 4 * 3)) {
        k = 0;
        n = (int)std::min((long long)wave, std::max((long long)R, units / kMinSegs));
    }
}

// A range of segments of one row.
template <typename T>
struct Piece {
    Row<T> x;
    int row, g0, g1;   // segments [g0, g1) of the row, of row_segs
    int segs;          // segments that the row has
    int in0, in1;      // those of the range that hold whole slots only
    const T* p;        // this thread's slot of segment in0 + warp
    __device__ __forceinline__ Piece(const LogprobArgs& a, int row_, int g0_, int g1_)
        : x(static_cast<const T*>(a.logits) + (long long)row_ * a.stride, a.V), row(row_), g0(g0_), g1(g1_) {
        segs = (x.slots() + 31) / 32;
        in0 = max(g0, x.shift != 0 ? 1 : 0);
        in1 = min(g1, (int)(((long long)x.V + x.shift) / (32 * kSlot<T>)));
        p = reinterpret_cast<const T*>(x.base + ((size_t)in0 * 32 + threadIdx.x) * kSlotBytes);
    }
    __device__ __forceinline__ int first() const { return in0 + (threadIdx.x >> 5); }  // this warp's first whole segment
};

// kUnroll segments of a piece per warp, from segment g on; places past the piece read as -inf.
template <typename T>
struct Block {
    RawVec<T, kSlot<T>> r[kUnroll];
    __device__ __forceinline__ void request(const Piece<T>& pc, int g) {
        if (g >= pc.in1) return;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (g + u * kWarpsL < pc.in1)
                r[u].load(pc.p + (size_t)(g - pc.first() + u * kWarpsL) * (32 * kSlot<T>));
            else
                r[u].fill_lowest();
        }
    }
};

// Statistics of a piece by one thread, and the maxima of its segments.  `next` holds the piece's first block;
// request_after() puts the first block of the next piece there: loads are in flight while a block, or a row, is
// summed up.
template <typename T, bool TOP, typename F>
__device__ __forceinline__ Stat scan(const Piece<T>& pc, Block<T>& next, float* unit_max, bool slots, F request_after) {
    constexpr int VEC = kSlot<T>;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    constexpr float lift = kHalf ? kLiftHalf : kLift, lift_from = kHalf ? kLiftFromHalf : kLiftFrom;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Stat2 run;
    run.clear();
    auto keep_max = [&](int g, float m) {
        if (TOP) {
            if (slots) {
                unit_max[g * 32 + lane] = m;
            } else {
                float w;
                asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(w) : "f"(m));
                if (lane == 0) unit_max[g] = w;
            }
        }
    };
    // The row's ends, element by element: the first segment by warp 0, the last by warp 1.
    const int g1 = min(pc.g1, pc.segs);
    const int end = warp == 0 ? (pc.g0 < pc.in0 ? pc.g0 : -1) : warp == 1 ? (g1 > pc.in1 && g1 > pc.in0 ? g1 - 1 : -1) : -1;
    if (end >= 0) {
        RawVec<T, VEC> f;
        pc.x.load(end * 32 + lane, f);
        const float m = f.max();
        keep_max(end, m);
        run.raise(m);
        if (run.c != neg_inf()) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) run.add(f.get(i), f.get(i + 1));
        }
    }
    int g = pc.first();
    if (g >= pc.in1) request_after();
    for (; g < pc.in1; g += kWarpsL * kUnroll) {
        Block<T> b = next;
        if (g + kWarpsL * kUnroll < pc.in1)
            next.request(pc, g + kWarpsL * kUnroll);
        else
            request_after();
        float m = neg_inf();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const float mu = b.r[u].max();
            m = fmaxf(m, mu);
            if (g + u * kWarpsL < pc.in1) keep_max(g + u * kWarpsL, mu);
        }
        run.raise(m);
        if (run.c > lift_from && run.c < kFar) {
            const F2 mcl = run.minus_cl();
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                b.r[u].lift(lift);
#pragma unroll
                for (int i = 0; i < VEC; i += 2) run.add_plain(b.r[u].get(i), b.r[u].get(i + 1), mcl);
            }
        } else if (run.c != neg_inf()) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                for (int i = 0; i < VEC; i += 2) run.add(b.r[u].get(i), b.r[u].get(i + 1));
        }
    }
    return run.get();
}

// a / b for a, b >= 0; the 64-bit division takes several times as long.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// How the units are cut into ranges of n CTAs: `per` units each, the first `more` CTAs one more; or, with k > 0, every
// row of `segs` units by itself into k ranges.
struct Split {
    long long per, more;
    int segs, k;
    __device__ __forceinline__ Split(int rows, int segs_, int n, int k_) : segs(segs_), k(k_) {
        const long long units = (long long)rows * segs;
        per = k > 0 ? 0 : quotient(units, n);
        more = units - per * n;
    }
    __device__ __forceinline__ long long begin(int c) const {
        if (k > 0) {
            const int row = (int)((uint32_t)c / (uint32_t)k);
            return (long long)row * segs + quotient((long long)(c - row * k) * segs, k);
        }
        return c * per + min((long long)c, more);
    }
    __device__ __forceinline__ int cta_of(long long u) const {  // whose range holds unit u
        const long long big = more * (per + 1);
        return (int)(u < big ? quotient(u, per + 1) : more + quotient(u - big, per));
    }
    // the CTAs that share a row
    __device__ __forceinline__ int first(int row) const { return k > 0 ? row * k : cta_of((long long)row * segs); }
    __device__ __forceinline__ int last(int row) const { return k > 0 ? row * k + k - 1 : cta_of((long long)(row + 1) * segs - 1); }
};

__device__ __forceinline__ float4 pack(const Stat& st) { return make_float4(st.c, st.s, st.t, 0.f); }
__device__ __forceinline__ Stat unpack(float4 v) { return Stat{v.x, v.y, v.z}; }

// The pieces of a row that CTAs first .. last share, by one warp; `held`: what the lane has of them already.
__device__ __forceinline__ float4 lane_piece(const Ws& ws, int first, int c, int last) {
    return c <= last ? __ldcg(ws.part + c * 2 + (c == first)) : pack(stat_none());
}
__device__ __forceinline__ Stat join_pieces(const Ws& ws, int first, int last, float4 held) {
    Stat st = unpack(held);
    for (int c = first + 32 + (threadIdx.x & 31); c <= last; c += 32) st = stat_join(st, unpack(lane_piece(ws, first, c, last)));
    return stat_warp(st);
}

__device__ __forceinline__ void write_row(const LogprobArgs& a, int row, const RowStat& rs, bool given, float tok_score) {
    if (a.logprob != nullptr) a.logprob[row] = given ? stat_logprob(rs, tok_score) : 0.f;
    if (a.entropy != nullptr) a.entropy[row] = rs.entropy;
    if (a.lse != nullptr) a.lse[row] = rs.lse;
}

// A row's statistics (request(): what the lane reads of them, stat(): those of the whole row, by one warp) and its
// alternatives, by all threads of a CTA.  EARLY: what a warp reads of the statistics and the token is requested before
// the choice, not during it.  Many rows at once gain by it (the second kernel, 1024 x 65536 bf16 with 20 alternatives:
// 40.8 against 42.6 us), a row by itself loses, as the warp's share of the maxima waits (9 x 1365: 6.7 against 6.3 us).
template <typename T, bool SLOTS, bool EARLY, typename Request, typename GetStat>
__device__ __forceinline__ void choose(SelectSmem& s_sel, RowStat& s_rs, const LogprobArgs& a, const Ws& ws, int row, int row_segs,
                                       Request request, GetStat stat) {
    constexpr int kHeld = SLOTS ? 16 : 4;
    const T* p = static_cast<const T*>(a.logits) + (long long)row * a.stride;
    const Row<T> x(p, a.V);
    float4 held;
    bool given = false;
    float tok_score = 0.f;
    auto read = [&] {
        const int tok = a.logprob != nullptr ? a.tokens[row] : -1;
        held = request();
        given = tok >= 0 && tok < a.V;
        if (given) tok_score = to_f32(p[tok]);
    };
    if (EARLY && threadIdx.x >= kSelThreads - 32) read();
    auto finish = [&] {
        if (!EARLY) read();
        const RowStat rs = stat_finish(stat(held));
        if ((threadIdx.x & 31) == 0) {
            s_rs = rs;
            write_row(a, row, rs, given, tok_score);
        }
    };
    select_top<kHeld>(
        s_sel, SLOTS ? x.slots() : (x.slots() + 31) / 32, a.top_n, 0u,
        RowUnits<T, SLOTS>{x, ws.unit_max + (size_t)row * row_units(row_segs)}, finish,
        [&](int i, unsigned long long k) {
            const size_t o = (size_t)row * a.top_n + i;
            a.top_ids[o] = k != 0ull ? (int32_t)key_gid(k) : -1;
            a.top_logprobs[o] = k != 0ull ? stat_logprob(s_rs, key_score(k)) : neg_inf();
        });
}

// What a scan does besides the statistics: nothing; the units' maxima, for the second kernel; or the choice itself, by the
// last CTA of a row, where every CTA has one row or piece (by slots or by segments).
enum Mode { kStats, kMaxima, kChooseSlots, kChooseSegs };

// Everything after a row's scan is warp 0's; the other warps go on with the next row.  Without alternatives the last
// CTA of a row joins the pieces and writes the results.
template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreadsL, MODE != kStats ? kPerSmTop : kPerSm)
    k_logprobs(const LogprobArgs a, const Ws ws, const int row_segs, const int pieces) {
    constexpr bool TOP = MODE != kStats, CHOOSE = MODE == kChooseSlots || MODE == kChooseSegs;
    __shared__ float4 s_part[2][kWarpsL];
    if (!CHOOSE) rows_launch_dependents();
    rows_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Split split(a.R, row_segs, gridDim.x, pieces);
    const long long u0 = split.begin(blockIdx.x), u1 = split.begin(blockIdx.x + 1);
    const int row0 = (int)quotient(u0, row_segs), first_g = (int)(u0 - (long long)row0 * row_segs);
    long long left = u1 - u0;  // units from the current piece on
    int row = row0, g0 = first_g;
    Block<T> next;
    {
        const Piece<T> pc(a, row, g0, (int)min((long long)row_segs, g0 + left));
        next.request(pc, pc.first());
    }
    for (int buf = 0; left > 0; buf ^= 1, ++row, g0 = 0) {
        const int g1 = (int)min((long long)row_segs, g0 + left);
        left -= g1 - g0;
        const T* p = static_cast<const T*>(a.logits) + (long long)row * a.stride;
        float* unit_max = TOP ? ws.unit_max + (size_t)row * row_units(row_segs) : nullptr;
        float tok_score = 0.f;  // requested before the scan, used after it
        bool given = false;
        if (!TOP && threadIdx.x == 0 && a.logprob != nullptr) {
            const int tok = a.tokens[row];
            given = tok >= 0 && tok < a.V;
            if (given) tok_score = to_f32(p[tok]);
        }
        Stat st = stat_warp(scan<T, TOP>(Piece<T>(a, row, g0, g1), next, unit_max, row_segs <= kSlotSegs, [&] {
            if (left > 0) {
                const Piece<T> after(a, row + 1, 0, (int)min((long long)row_segs, left));
                next.request(after, after.first());
            }
        }));
        if (lane == 0) s_part[buf][warp] = pack(st);
        __syncthreads();
        if constexpr (CHOOSE) {
            __shared__ SelectSmem s_sel;
            __shared__ RowStat s_rs;
            __shared__ bool s_last;
            const bool shared_row = g1 - g0 < row_segs;
            const int first = split.first(row), last = split.last(row);
            auto mine = [&] { return stat_warp(lane < kWarpsL ? unpack(s_part[buf][lane]) : stat_none()); };
            if (shared_row) {
                if (warp == 0) {
                    st = mine();
                    if (lane == 0) {
                        __stcg(ws.part + blockIdx.x * 2 + ((int)blockIdx.x == first), pack(st));
                        s_last = rows_take_ticket(ws.ticket + first) == (unsigned)(last - first);
                        if (s_last) __stcg(ws.ticket + first, 0u);
                    }
                }
                __syncthreads();
                if (!s_last) return;
            }
            choose<T, MODE == kChooseSlots, false>(
                s_sel, s_rs, a, ws, row, row_segs,
                [&] { return shared_row ? lane_piece(ws, first, first + lane, last) : pack(stat_none()); },
                [&](float4 held) { return shared_row ? join_pieces(ws, first, last, held) : mine(); });
            return;
        }
        if (warp != 0) continue;
        st = stat_warp(lane < kWarpsL ? unpack(s_part[buf][lane]) : stat_none());
        if (g1 - g0 < row_segs) {
            const int first = split.first(row);
            float4* part = ws.part + blockIdx.x * 2 + ((int)blockIdx.x == first);
            if (TOP) {
                if (lane == 0) *part = pack(st);
                continue;
            }
            // the last of the row's CTAs to get here joins the pieces
            const int last = split.last(row);
            int done = 0;
            if (lane == 0) {
                __stcg(part, pack(st));
                done = rows_take_ticket(ws.ticket + first) == (unsigned)(last - first);
                if (done) __stcg(ws.ticket + first, 0u);
            }
            if (__shfl_sync(0xFFFFFFFFu, done, 0) == 0) continue;
            __syncwarp();
            st = join_pieces(ws, first, last, lane_piece(ws, first, first + lane, last));
        }
        if (lane == 0) {
            if (TOP)
                ws.row[row] = pack(st);
            else
                write_row(a, row, stat_finish(st), given, tok_score);
        }
    }
}

// One row per CTA: its statistics and its alternatives, after k_logprobs<T, kMaxima> of n_scan CTAs.
template <typename T, bool SLOTS>
__global__ void __launch_bounds__(kSelThreads, 3)
    k_logprobs_top(const LogprobArgs a, const Ws ws, const int row_segs, const int n_scan) {
    __shared__ SelectSmem s_sel;
    __shared__ RowStat s_rs;
    rows_wait();
    const int row = blockIdx.x;
    const Split split(a.R, row_segs, n_scan, 0);
    const int first = split.first(row), last = split.last(row), lane = threadIdx.x & 31;
    choose<T, SLOTS, true>(
        s_sel, s_rs, a, ws, row, row_segs,
        [&] { return first == last ? ws.row[row] : lane_piece(ws, first, first + lane, last); },
        [&](float4 held) { return first == last ? unpack(held) : join_pieces(ws, first, last, held); });
}

// ---------------------------------------------------------------------------
// Gradient: every thread takes kGradUnroll slots of its row.

constexpr int kGradUnroll = 4;

// VEC: elements of a 16-byte slot, as the forward pass cuts a row (both tensors' rows lie alike in their slots), or 1.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreadsL) k_logprobs_grad(const LogprobGradArgs a, int chunks) {
    rows_wait();
    const int row = (int)(blockIdx.x / chunks);
    const int chunk = (int)(blockIdx.x % chunks);
    const T* x = static_cast<const T*>(a.logits) + (long long)row * a.stride;
    T* d = static_cast<T*>(a.dlogits) + (long long)row * a.d_stride;
    const int shift = VEC == 1 ? 0 : (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const long long e0 = ((long long)chunk * kThreadsL * kGradUnroll + threadIdx.x) * VEC - shift;
    constexpr long long kStep = (long long)kThreadsL * VEC;
    RawVec<T, VEC> r[kGradUnroll];
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
        const long long e = e0 + u * kStep;
        if (e >= 0 && e + VEC <= a.V) r[u].load(x + e);
    }
    const float lse = a.lse[row];
    const int tok = a.tokens != nullptr ? a.tokens[row] : -1;
    const bool given = tok >= 0 && tok < a.V;
    float gl = (given && a.g_logprob != nullptr) ? a.g_logprob[row] : 0.f;
    const float ge = a.g_entropy != nullptr ? a.g_entropy[row] : 0.f;
    const float ent = a.g_entropy != nullptr ? a.entropy[row] : 0.f;
    const bool empty = lse == neg_inf();
    // dx = p (k0 - ge2 y) with y = log2 p: -g_lp p - g_ent p (ln2 y + entropy)
    const float k0 = empty ? 0.f : (lse != lse ? quiet_nan() : -gl - ge * ent);
    const float ge2 = empty ? 0.f : ge * kLn2;
    if (empty) gl = 0.f;
    auto of = [&](float v) {
        const float y = fmaxf((v - lse) * kLog2e, kFloorY);
        return (empty ? 0.f : ex2(y)) * fmaf(-ge2, y, k0);
    };
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
        const long long e = e0 + u * kStep;
        if (e >= 0 && e + VEC <= a.V) {
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = of(r[u].get(i));
            if (given && tok >= e && tok < e + VEC) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] += e + i == tok ? gl : 0.f;
            }
            RawVec<T, VEC> o;
            pack_vec<T, VEC>(o, f);
            o.store(d + e);
        } else if (VEC > 1 && e < a.V && e + VEC > 0) {  // a row's ends
            for (int i = 0; i < VEC; ++i)
                if (e + i >= 0 && e + i < a.V)
                    d[e + i] = from_f32<T>(of(to_f32(x[e + i])) + (given && e + i == tok ? gl : 0.f));
        }
    }
}

template <typename... P, typename... A>
static cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
static cudaError_t forward(const LogprobArgs& a, cudaStream_t s) {
    const int segs = max_segs(a.V, (int)sizeof(T));
    Ws ws;
    uint8_t* p = static_cast<uint8_t*>(a.ws);
    ws.ticket = reinterpret_cast<unsigned int*>(p + kWsHeaderBytes);
    ws.part = reinterpret_cast<float4*>(p + kTicketEnd);
    ws.row = reinterpret_cast<float4*>(p + kPartEnd);
    ws.unit_max = reinterpret_cast<float*>(p + kPartEnd + (size_t)a.R * 16);
    int n, k;
    plan(a.R, segs, a.top_n > 0, n, k);
    const dim3 grid((unsigned)n);
    const dim3 block(kThreadsL);
    const bool slots = segs <= kSlotSegs;
    if (a.top_n == 0) return launch(k_logprobs<T, kStats>, grid, block, s, a, ws, segs, k);
    if (k > 0)
        return slots ? launch(k_logprobs<T, kChooseSlots>, grid, block, s, a, ws, segs, k)
                     : launch(k_logprobs<T, kChooseSegs>, grid, block, s, a, ws, segs, k);
    const cudaError_t e = launch(k_logprobs<T, kMaxima>, grid, block, s, a, ws, segs, 0);
    if (e != cudaSuccess) return e;
    const dim3 rows((unsigned)a.R), sel(kSelThreads);
    return slots ? launch(k_logprobs_top<T, true>, rows, sel, s, a, ws, segs, n)
                 : launch(k_logprobs_top<T, false>, rows, sel, s, a, ws, segs, n);
}

template <typename T, int VEC>
static cudaError_t grad_vec(const LogprobGradArgs& a, cudaStream_t s) {
    const long long per = (long long)kThreadsL * kGradUnroll * VEC;
    const long long chunks = ((long long)a.V + VEC - 1 + per - 1) / per;  // up to VEC - 1 places before the first element
    const long long rows_max = std::max(1LL, 2147483647LL / chunks);
    for (long long r0 = 0; r0 < a.R; r0 += rows_max) {
        LogprobGradArgs b = a;
        const int nr = (int)std::min(rows_max, a.R - r0);
        b.logits = static_cast<const T*>(a.logits) + r0 * a.stride;
        b.dlogits = static_cast<T*>(a.dlogits) + r0 * a.d_stride;
        b.tokens = a.tokens ? a.tokens + r0 : nullptr;
        b.lse = a.lse + r0;
        b.entropy = a.entropy ? a.entropy + r0 : nullptr;
        b.g_logprob = a.g_logprob ? a.g_logprob + r0 : nullptr;
        b.g_entropy = a.g_entropy ? a.g_entropy + r0 : nullptr;
        cudaError_t e = launch(k_logprobs_grad<T, VEC>, dim3((unsigned)(chunks * nr)), dim3(kThreadsL), s, b, (int)chunks);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
static cudaError_t grad(const LogprobGradArgs& a, cudaStream_t s) {
    constexpr int V = kVecOf<T>;
    const bool alike = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.dlogits)) & 15) == 0 &&
                       (a.stride - a.d_stride) % V == 0;
    return alike ? grad_vec<T, V>(a, s) : grad_vec<T, 1>(a, s);
}

}  // namespace lp

size_t logits_logprobs_ws_bytes(int R, int V, int top_n) {
    const int units = std::max(lp::row_units(lp::max_segs(V, 4)), lp::row_units(lp::max_segs(V, 2)));
    return lp::kPartEnd + (top_n > 0 ? (size_t)R * 16 + round16((size_t)R * units * 4) : 0);
}

cudaError_t launch_logits_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s) {
    if (dtype == VH_BF16) return lp::forward<__nv_bfloat16>(a, s);
    if (dtype == VH_F16) return lp::forward<__half>(a, s);
    return lp::forward<float>(a, s);
}

cudaError_t launch_logits_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s) {
    if (dtype == VH_BF16) return lp::grad<__nv_bfloat16>(a, s);
    if (dtype == VH_F16) return lp::grad<__half>(a, s);
    return lp::grad<float>(a, s);
}

}  // namespace vh
