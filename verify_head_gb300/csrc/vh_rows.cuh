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

__device__ __forceinline__ void rows_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void rows_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
    static_assert(VEC * sizeof(T) == 16, "one 16-byte vector");
    union {
        uint4 q;
        uint32_t u[4];
    };
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
    __device__ __forceinline__ void load(const T* p) { q = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = q; }
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
// Softmax statistics relative to a running maximum c: s = sum e^(x - c),
// t = sum e^(x - c) y with y = log2(e) (x - c) <= 0.  Then lse = c + ln s,
// log p = (x - c) - ln s and entropy = ln2 (log2 s - t / s): the entropy's
// terms are small where the row is peaked, so nothing cancels.  c = -inf:
// nothing summed yet (s = t = 0).  A +inf score leaves c = +inf and the row's
// statistics are NaN.  x - c is taken before the factor log2(e): the type's
// lowest value times that factor would be -inf, and a row that holds nothing
// else would be lost.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
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

// Move statistics to a larger shift.
__device__ __forceinline__ void stat_shift(Stat& a, float c) {
    if (a.s != 0.f) {
        const float d = fmaxf((a.c - c) * kLog2e, kFloorY);
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

__device__ __forceinline__ void stat_add(Stat& a, float x) {  // a.c >= x, not -inf
    const float y = fmaxf((x - a.c) * kLog2e, kFloorY);
    const float e = ex2(y);
    a.s += e;
    a.t = fmaf(e, y, a.t);
}

__device__ __forceinline__ Stat stat_warp(Stat a) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        Stat b;
        b.c = __shfl_xor_sync(0xFFFFFFFFu, a.c, m);
        b.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, m);
        b.t = __shfl_xor_sync(0xFFFFFFFFu, a.t, m);
        a = stat_join(a, b);
    }
    return a;
}

// A finished row.
struct RowStat {
    float c, log2_s, lse, entropy;
};
__device__ __forceinline__ RowStat stat_finish(const Stat& a) {
    RowStat r;
    r.c = a.c;
    r.log2_s = log2f(a.s);
    if (a.c == neg_inf()) {  // nothing but -inf (or NaN)
        r.lse = neg_inf();
        r.entropy = 0.f;
    } else if (a.c == -neg_inf()) {
        r.lse = r.entropy = quiet_nan();
    } else {
        r.lse = fmaf(r.log2_s, kLn2, a.c);
        r.entropy = fmaxf((r.log2_s - a.t / a.s) * kLn2, 0.f);
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
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
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

}  // namespace vh
