// Device helpers shared by the row operators (norm, log probabilities):
// element types, 16-byte vectors, base-2 softmax statistics and the sorted
// top list of a warp.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "vh_common.cuh"

namespace vh {

// Lets the next kernel in the stream start.  The head kernels read their weight table, and the read-only path their ids
// and rows, without regard to kernels that are still running: a kernel signals only if it writes neither rows nor ids
// that a caller could hand on (workspaces and fp32 vectors are read after the wait), or if a kernel of the same call,
// which waits for it, follows.
__device__ __forceinline__ void rows_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void rows_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Before bulk or tensor copies read what kernels before this one wrote.
__device__ __forceinline__ void rows_fence_async() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Adds one to a counter, after everything that this thread wrote or (by a barrier) saw written and before everything that
// it reads from then on: one ordered operation instead of full fences on both sides.
__device__ __forceinline__ uint32_t rows_take_ticket(uint32_t* p) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// ---------------------------------------------------------------------------
// Element types and vectors of VEC elements (16 bytes, or one element).

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T>
constexpr int kVecOf = 16 / (int)sizeof(T);

template <typename T, int VEC>
struct RawVec;  // VEC elements as loaded
template <typename T>
struct RawVec<T, 1> {
    T v;
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
    __device__ __forceinline__ void set(int, float f) { v = from_f32<T>(f); }
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
};
template <typename T, int VEC>
struct RawVec {
    static constexpr int N = VEC * (int)sizeof(T) / 4;  // 32-bit words
    static_assert(N == 4 || N == 8, "one vector of 16 or 32 bytes");
    uint32_t u[N];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(u[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            return (i & 1) ? bf_hi(u[i >> 1]) : bf_lo(u[i >> 1]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i >> 1]));
            return (i & 1) ? f.y : f.x;
        }
    }
    __device__ __forceinline__ void set2(int i, float lo, float hi) {  // elements 2i, 2i+1 (16-bit types)
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(lo, hi);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (N == 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            u[0] = q.x;
            u[1] = q.y;
            u[2] = q.z;
            u[3] = q.w;
        } else {
            // read once: no L1 allocation, first out of L2; not the read-only path, since a kernel of this library that
            // let this one start early may have written the row
            asm volatile(
                "ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                : "l"(p));
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        static_assert(N == 4, "stores are of 16 bytes");
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void put(int i, T v) {  // element i as it is
        if constexpr (sizeof(T) == 4) {
            u[i] = __float_as_uint(v);
        } else {
            const uint32_t h = *reinterpret_cast<const uint16_t*>(&v);
            u[i >> 1] = (i & 1) ? (u[i >> 1] & 0xFFFFu) | (h << 16) : (u[i >> 1] & 0xFFFF0000u) | h;
        }
    }
    __device__ __forceinline__ void fill_lowest() {  // -inf
#pragma unroll
        for (int i = 0; i < N; ++i)
            u[i] = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __nv_bfloat16>::value ? 0xFF80FF80u : 0xFC00FC00u;
    }
    // Elements below `lo` and NaN become `lo`: two per instruction for the 16-bit types.
    __device__ __forceinline__ void lift(float lo) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = __float_as_uint(fmaxf(__uint_as_float(u[i]), lo));
        } else {
            using P = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
            P b;
            b.x = b.y = from_f32<T>(lo);
            P* p = reinterpret_cast<P*>(u);
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = __hmax2(p[i], b);
        }
    }
    // The largest element, NaN left out (-inf if there is nothing else).
    __device__ __forceinline__ float max() const {
        const float lowest = -__int_as_float(0x7f800000);
        if constexpr (sizeof(T) == 4) {
            float m = lowest;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, get(i));
            return m;
        } else {
            using P = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
            const P* p = reinterpret_cast<const P*>(u);
            P m = p[0];
#pragma unroll
            for (int i = 1; i < N; ++i) m = __hmax2(m, p[i]);
            return fmaxf(fmaxf(to_f32(m.x), to_f32(m.y)), lowest);
        }
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void pack_vec(RawVec<T, VEC>& r, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        r.set(0, f[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) r.set2(i, f[2 * i], f[2 * i + 1]);
    }
}

// ---------------------------------------------------------------------------
// Two floats in one register pair: the packed fp32 instructions issue once for both.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// ---------------------------------------------------------------------------
// Softmax statistics relative to a running maximum c: s = sum 2^y, t = sum
// 2^y y with y = log2(e) (x - c) <= 0.  Then lse = c + ln s, log p = (x - c)
// - ln s and entropy = ln2 (log2 s - t / s): the entropy's terms are small
// where the row is peaked, so nothing cancels.  c = -inf: nothing summed yet
// (s = t = 0).  A +inf score leaves c = +inf and the row's statistics are NaN.
//
// Where |c| < kFar, y is taken as fma(x, log2e, -round(c log2e)); every use of
// such a c rounds that product the same way, and what the rounding took
// (stat_rest, a sixteenth at most) is given back at the end.  The rounding
// grows with |c|: from about 1e9 it is an exponent that 2^y cannot hold, and a
// row with nothing but a mask value in it (-1e10, -1e30, the type's lowest)
// has such a maximum.  From kFar on y is (x - c) log2e, which costs a
// subtraction more per score.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = 1048576.0f;
// Scores below kLift carry no probability beside a maximum above kLiftFrom and may be lifted to it.  A type whose
// lowest value is above kLift is lifted to that value, beside a maximum that is well above it.
constexpr float kLift = -1e30f, kLiftFrom = -kFar;
constexpr float kLiftHalf = -65504.f, kLiftFromHalf = -60000.f;
// y below this is lifted to it: 2^y is 0 in either case and y * 2^y must not
// become -inf * 0 at masked places (NaN scores land here too: they count as -inf).
constexpr float kFloorY = -2000.0f;

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

// 2^x; results below the smallest normal number are 0.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Stat {
    float c, s, t;
};

__device__ __forceinline__ Stat stat_none() { return Stat{neg_inf(), 0.f, 0.f}; }

// What the rounding of c log2e took.
__device__ __forceinline__ float stat_rest(float c) {
    return fabsf(c) < kFar ? fmaf(c, kLog2e, -__fmul_rn(c, kLog2e)) : 0.f;
}

// y of a score.
__device__ __forceinline__ float stat_y(float x, float c) {
    const float y = fabsf(c) < kFar ? fmaf(x, kLog2e, -(c * kLog2e)) : (x - c) * kLog2e;
    return fmaxf(y, kFloorY);
}

// Move statistics to a larger maximum.
__device__ __forceinline__ void stat_shift(Stat& a, float c) {
    if (a.s != 0.f) {
        // each maximum's sums lack what its own product's rounding took
        const float d = fmaxf(fmaf(a.c - c, kLog2e, stat_rest(c) - stat_rest(a.c)), kFloorY);
        const float f = ex2(d);
        a.t = f * fmaf(d, a.s, a.t);
        a.s *= f;
    }
    a.c = c;
}

__device__ __forceinline__ Stat stat_join(Stat a, Stat b) {
    const float c = fmaxf(a.c, b.c);
    stat_shift(a, c);
    stat_shift(b, c);
    return Stat{c, a.s + b.s, a.t + b.t};
}

// The same statistics with the sums in two halves, for long runs of scores.
struct Stat2 {
    float c;
    F2 s, t;
    __device__ __forceinline__ void clear() {
        c = neg_inf();
        s = t = f2(0.f, 0.f);
    }
    __device__ __forceinline__ Stat get() const {
        const float2 a = f2_get(s), b = f2_get(t);
        return Stat{c, a.x + a.y, b.x + b.y};
    }
    __device__ __forceinline__ void raise(float m) {  // a new maximum
        if (m > c) {
            Stat a = get();
            stat_shift(a, m);
            c = m;
            s = f2(a.s, 0.f);
            t = f2(a.t, 0.f);
        }
    }
    // Two scores; c is their maximum or more, not -inf.
    __device__ __forceinline__ void add(float x0, float x1) { add_y(stat_y(x0, c), stat_y(x1, c)); }
    // The same where |c| >= kFar.
    __device__ __forceinline__ void add_far(float x0, float x1) {
        add_y(fmaxf((x0 - c) * kLog2e, kFloorY), fmaxf((x1 - c) * kLog2e, kFloorY));
    }
    // Two scores of which none is -inf or NaN, where |c| < kFar: minus_cl = -c log2e twice.
    __device__ __forceinline__ void add_plain(float x0, float x1, F2 minus_cl) {
        const F2 y = f2_fma(f2(x0, x1), f2(kLog2e, kLog2e), minus_cl);
        const float2 v = f2_get(y);
        const F2 e = f2(ex2(v.x), ex2(v.y));
        s = f2_add(s, e);
        t = f2_fma(e, y, t);
    }
    __device__ __forceinline__ F2 minus_cl() const { return f2(-(c * kLog2e), -(c * kLog2e)); }

private:
    __device__ __forceinline__ void add_y(float y0, float y1) {
        const F2 y = f2(y0, y1), e = f2(ex2(y0), ex2(y1));
        s = f2_add(s, e);
        t = f2_fma(e, y, t);
    }
};

__device__ __forceinline__ Stat stat_warp(Stat a) {
    float c;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(c) : "f"(a.c));
    stat_shift(a, c);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, m);
        a.t += __shfl_xor_sync(0xFFFFFFFFu, a.t, m);
    }
    return a;
}

// A finished row.
struct RowStat {
    float c, log2_s, lse, entropy;  // log2_s: of the sum relative to c log2e itself, not to its rounding
};
__device__ __forceinline__ RowStat stat_finish(const Stat& a) {
    RowStat r;
    r.c = a.c;
    const float l = log2f(a.s);
    r.log2_s = l - stat_rest(a.c);
    if (a.c == neg_inf()) {  // nothing but -inf (or NaN)
        r.lse = neg_inf();
        r.entropy = 0.f;
    } else if (a.c == -neg_inf()) {
        r.lse = r.entropy = quiet_nan();
    } else {
        r.lse = fmaf(r.log2_s, kLn2, a.c);
        r.entropy = fmaxf((l - a.t / a.s) * kLn2, 0.f);
    }
    return r;
}
// Log probability of a score of the row.
__device__ __forceinline__ float stat_logprob(const RowStat& r, float x) {
    if (x != x || r.c == neg_inf()) return neg_inf();
    if (r.c == -neg_inf()) return quiet_nan();
    return fmaf(-r.log2_s, kLn2, x - r.c);
}

// ---------------------------------------------------------------------------
// The 32 largest keys a warp has seen, sorted: lane i holds the i-th largest
// (0 = none).  Keys are those of the argmax (score, then lower id), so the
// order is total and the result does not depend on the order of insertion.

__device__ __forceinline__ unsigned long long shfl_key(unsigned long long k, int mask) {
    return __shfl_xor_sync(0xFFFFFFFFu, k, mask);
}

// A bitonic sequence over the lanes -> descending.
__device__ __forceinline__ unsigned long long top_clean(unsigned long long k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        const unsigned long long o = shfl_key(k, m);
        const bool keep_max = (lane & m) == 0;
        k = ((o > k) == keep_max) ? o : k;
    }
    return k;
}

// Any 32 keys -> descending (bitonic sort).
__device__ __forceinline__ unsigned long long top_sort(unsigned long long k) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll 1
        for (int m = size >> 1; m >= 1; m >>= 1) {
            const unsigned long long o = shfl_key(k, m);
            const bool keep_max = ((lane & m) == 0) == ((lane & size) == 0);
            k = ((o > k) == keep_max) ? o : k;
        }
    }
    return k;
}

// Merge a sorted list into `top` (both descending).
__device__ __forceinline__ void top_merge(unsigned long long& top, unsigned long long sorted) {
    const unsigned long long r = __shfl_sync(0xFFFFFFFFu, sorted, 31 - (threadIdx.x & 31));
    top = top_clean(r > top ? r : top);
}

// Merge any 32 keys, given that only the n largest matter.
__device__ __forceinline__ void top_insert(unsigned long long& top, unsigned long long key, int n) {
    const unsigned long long floor = __shfl_sync(0xFFFFFFFFu, top, n - 1);
    if (__any_sync(0xFFFFFFFFu, key > floor)) top_merge(top, top_sort(key));
}

// ---------------------------------------------------------------------------
// The n <= kMaxTop largest elements of a row, from the maxima of the units it
// is cut into, by a CTA of kSelThreads threads.
//
// 64 groups of units give a bound: the n-th largest of their maxima, which n
// elements at least reach, and about 1.3 n units do.  Those units are listed,
// then their elements that reach the bound; an element's place is the number
// of listed keys above its own.  No step depends on a search, so the whole is
// a chain of a few loads and barriers.
//
// Where a list overflows many elements are equal to the bound (a row masked
// to fewer than n places, equal logits): then only the elements above it are
// listed, and the rest come, in the order of their ids, from the first units
// that reach it.  Where even those overflow (rows laid out against the
// groups) the CTA sorts: each warp keeps the 32 largest keys of its share,
// first of the maxima, then of the elements of the n best units, which hold
// the n largest elements since any element elsewhere is preceded by n others
// (equal maxima: the lower unit first, as a unit is a range of ids).

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelGroups = 64;
constexpr int kSelUnits = 256;  // listed units
constexpr int kSelElems = 512;  // listed elements: 31 units of 16, which a row of fewer units than n has at most

struct SelectSmem {
    uint32_t mine[kSelThreads];
    uint32_t group[kSelGroups];
    uint32_t unit[kSelUnits];
    unsigned long long elem[kSelElems];
    unsigned long long sorted[kSelWarps][32];
    uint32_t bound;
    int n_unit, n_elem;
};

// HELD: maxima a thread holds in registers; up to HELD * kSelThreads units are read once, more are read twice.
// Units: float max(int g), the maximum of unit g < units (NaN left out);
//   kLane: whether a unit is read by one lane (each its own) or by a warp together;
//   Item load(int g), this lane's elements of unit g;
//   float peak(const Item&), the largest of them (NaN left out);
//   void each(const Item&, int g, float b, f): f(key) with the argmax key of those that are not below b;
//   kBatches, key(int g, int i): by a warp, the lane's key in batch i < kBatches of the unit's elements, in the order of
//   their ids; 0 past the last.
// meanwhile(): called once, by the last warp, while the others read the listed units; emit() may use what it left in
//   shared memory.
// emit(i, key): key of the i-th largest element, i < n (0 = the row has fewer).
// floor: ord_f32 of a value that n elements are known to reach, 0 = none.
// All threads call it; nothing of sm need be set.
template <int HELD, typename Units, typename Meanwhile, typename Emit>
__device__ __forceinline__ void select_top(SelectSmem& sm, int units, int n, uint32_t floor, const Units& un,
                                           Meanwhile meanwhile, Emit emit) {
    constexpr int kAtOnce = 4;  // units a warp loads at once
    constexpr int kReaders = kSelWarps - 1;  // warps that read units
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float held[HELD];
    auto hold = [&](int base) {  // no branches between the loads
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i] = un.max(min(base + i * kSelThreads + tid, units - 1));
    };
    auto held_max = [&](int base, float m) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) m = fmaxf(m, base + i * kSelThreads + tid < units ? held[i] : neg_inf());
        return m;
    };
    hold(0);
    float m = held_max(0, neg_inf());
    for (int base = HELD * kSelThreads; base < units; base += HELD * kSelThreads) {
        hold(base);
        m = held_max(base, m);
    }
    const uint32_t mine = tid < units ? ord_f32(m) : 0u;
    sm.mine[tid] = mine;
    if (tid == 0) sm.n_unit = sm.n_elem = 0;
    __syncthreads();
    uint32_t me = 0u;
    if (tid < kSelGroups) {
#pragma unroll
        for (int i = 0; i < kSelThreads; i += kSelGroups) me = max(me, sm.mine[tid + i]);
        sm.group[tid] = me;
    }
    __syncthreads();
    if (tid < kSelGroups) {
        int above = 0;
#pragma unroll
        for (int j = 0; j < kSelGroups; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(sm.group + j);
            above += (o.x > me || (o.x == me && j < tid)) + (o.y > me || (o.y == me && j + 1 < tid)) +
                     (o.z > me || (o.z == me && j + 2 < tid)) + (o.w > me || (o.w == me && j + 3 < tid));
        }
        if (above == n - 1) sm.bound = max(me, floor);
    }
    __syncthreads();
    const uint32_t bound = sm.bound;
    const float least = unord_f32(bound);  // may be NaN, which nothing is below

    bool told = false;
    // Units and elements of ord_f32 `from` or more into the lists; false where a list overflows.
    auto list = [&](uint32_t from) {
        if (mine >= from && mine != 0u) {
            for (int base = 0; base < units; base += HELD * kSelThreads) {
                if (units > HELD * kSelThreads) hold(base);
#pragma unroll
                for (int i = 0; i < HELD; ++i) {
                    const int g = base + i * kSelThreads + tid;
                    if (!(held[i] < least) && g < units && ord_f32(held[i]) >= from) {
                        const int e = atomicAdd(&sm.n_unit, 1);
                        if (e < kSelUnits) sm.unit[e] = (uint32_t)g;
                    }
                }
            }
        }
        __syncthreads();
        const int n_unit = sm.n_unit;
        if (!told && warp == kReaders) meanwhile();
        told = true;
        if (n_unit > kSelUnits) return false;
        auto take = [&](unsigned long long k) {
            if ((uint32_t)(k >> 32) >= from) {
                const int e = atomicAdd(&sm.n_elem, 1);
                if (e < kSelElems) sm.elem[e] = k;
            }
        };
        if constexpr (Units::kLane) {
            if (tid < n_unit) {
                const int g = (int)sm.unit[tid];
                un.each(un.load(g), g, least, take);
            }
        } else {
            for (int i0 = warp; i0 < n_unit && warp < kReaders; i0 += kReaders * kAtOnce) {
                typename Units::Item it[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int i = i0 + u * kReaders;
                    if (i < n_unit) it[u] = un.load((int)sm.unit[i]);
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int i = i0 + u * kReaders;
                    if (i < n_unit && ord_f32(un.peak(it[u])) >= from) un.each(it[u], (int)sm.unit[i], least, take);
                }
            }
        }
        __syncthreads();
        return sm.n_elem <= kSelElems;
    };
    auto emit_listed = [&](int m2) {
        for (int e = tid; e < m2; e += kSelThreads) {
            const unsigned long long k = sm.elem[e];
            int above = 0;
#pragma unroll 8
            for (int j = 0; j < m2; ++j) above += sm.elem[j] > k;
            if (above < n) emit(above, k);
        }
    };

    if (list(bound)) {
        const int m2 = sm.n_elem;
        emit_listed(m2);
        if (tid >= m2 && tid < n) emit(tid, 0ull);  // fewer elements than n
        return;
    }
    __syncthreads();
    if (tid == 0) sm.n_unit = sm.n_elem = 0;
    __syncthreads();
    if (list(bound + 1u)) {
        const int m2 = sm.n_elem;
        emit_listed(m2);
        if (m2 >= n || warp != 0) return;
        int at = m2;
        for (int g0 = 0; g0 < units && at < n; g0 += 32) {
            uint32_t some = __ballot_sync(0xFFFFFFFFu, g0 + lane < units && ord_f32(un.max(min(g0 + lane, units - 1))) >= bound);
            for (; some != 0u && at < n; some &= some - 1u) {
                const int g = g0 + __ffs(some) - 1;
#pragma unroll 1
                for (int j = 0; j < Units::kBatches && at < n; ++j) {
                    const unsigned long long k = un.key(g, j);
                    const bool equal = k != 0ull && (uint32_t)(k >> 32) == bound;
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, equal);
                    const int i = at + __popc(who & ((1u << lane) - 1u));
                    if (equal && i < n) emit(i, k);
                    at += __popc(who);
                }
            }
        }
        for (int i = at + lane; i < n; i += 32) emit(i, 0ull);
        return;
    }
    __syncthreads();
    unsigned long long top = 0ull;
    for (int g = warp * 32; g < units; g += kSelThreads) {
        const int gg = g + lane;
        top_insert(top, gg < units ? make_key(un.max(gg), (uint32_t)gg) : 0ull, n);
    }
    sm.sorted[warp][lane] = top;
    __syncthreads();
    unsigned long long best = sm.sorted[0][lane];
#pragma unroll 1
    for (int w = 1; w < kSelWarps; ++w) top_merge(best, sm.sorted[w][lane]);
    __syncthreads();
    top = 0ull;
    for (int i = warp; i < n; i += kSelWarps) {
        const unsigned long long k = __shfl_sync(0xFFFFFFFFu, best, i);
        if (k == 0ull) break;
#pragma unroll 1
        for (int j = 0; j < Units::kBatches; ++j) top_insert(top, un.key((int)key_gid(k), j), n);
    }
    sm.sorted[warp][lane] = top;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll 1
    for (int w = 1; w < kSelWarps; ++w) top_merge(top, sm.sorted[w][lane]);
    if (lane < n) emit(lane, top);
}

}  // namespace vh
