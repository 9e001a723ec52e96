// Root-mean-square norm with the residual's addition, with output in the
// input's type or in 8 bits with one scale per token, and its gradient.
//
//     h = x + r            u = h (w + offset)        rstd = 1 / sqrt(mean h^2 + eps)
//     y = u rstd           8 bits: code = round(u (Q (1 / max|u|))), scale = max|u| rstd / Q
//
// The scale of a token is a maximum over the same row that the norm divides
// by, so rstd cancels in the codes: they depend on h and w alone, not on the
// order in which the squares are summed.  Q is 127 (int8) or 448 (e4m3).
//
// Gradient, with n = h rstd, g = dy (w + offset):
//     dx = rstd (g - n mean(g n)) + dh        dw = sum over tokens of dy n
//
// Bound: memory.  The forward pass reads x, r and writes h, y once (the row
// stays in registers between the sum and the output); the gradient reads dy,
// h, dh and writes dx once.  Every sum is in 32 bits.
#include <cuda_fp8.h>

#include <algorithm>

#include "vh_ptx.cuh"
#include "vh_row_kernels.h"
#include "vh_rows.cuh"
#include "vh_window.h"

namespace vh {
namespace norm {

constexpr int kMaxThreads = 512;  // register-resident rows: up to 128 registers a thread
constexpr int kWideThreads = 512;
// Shares of dweight that eight warps per 32 columns sum (67 x 5120 bf16, 67 shares: 6.1 us a call against 7.0 with 32
// warps; 120 x 4096, 120 shares: 7.4 against 7.0).
constexpr int kFewParts = 80;
constexpr int kMaxRing = 4;                // tokens in flight per CTA of the gradient
constexpr size_t kRingBytes = 56 * 1024;   // of shared memory per CTA that a ring of over two tokens stays below
constexpr size_t kSmRingBytes = 220 * 1024;  // of shared memory per SM for rings
// The largest ring: two tokens' three rows of four vectors a thread, each begun in its granule.  A kernel's limit of
// shared memory is set to this whatever the call needs, so that it never falls between another thread's setting it and its launch.
constexpr size_t kMaxRingBytes = 2 * 3 * ((size_t)kMaxThreads * 4 * 16 + 16);

// Bounded wait for a barrier's phase: whether it completed.
__device__ __forceinline__ bool mbar_done(unsigned long long* bar, uint32_t parity) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > ptx::kTimeoutNs) return false;
    return true;
}

// 1-D copy global -> shared that completes on an mbarrier (both addresses and the size multiples of 16 bytes).
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, unsigned long long* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     ptx::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
                 : "memory");
}

// The larger value; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sums of two values over the threads of one row: wpr warps, of which this is number w; `row`: the row's wpr slots in
// shared memory.  MAX_SECOND: the second value is a maximum instead of a sum.  sync(): a barrier of all threads that
// call this together (not called where a row has one warp).  The lower half of a warp goes on with the first value and
// the upper half with the second, so both take one chain of shuffles.
template <bool MAX_SECOND, typename Sync>
__device__ __forceinline__ float2 reduce_row(float a, float b, float2* row, int w, int wpr, Sync sync) {
    const int lane = threadIdx.x & 31;
    const bool second = lane >= 16;
    auto join = [&](float v, float o) { return MAX_SECOND && second ? max_nan(v, o) : v + o; };
    const float other = __shfl_xor_sync(0xFFFFFFFFu, second ? a : b, 16);
    float v = join(second ? b : a, other);
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
    if (wpr == 1) return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
    if ((lane & 15) == 0) reinterpret_cast<float*>(row + w)[lane >> 4] = v;
    sync();
    float2 t = row[0];
#pragma unroll 4
    for (int i = 1; i < wpr; ++i) {
        const float2 o = row[i];
        t.x += o.x;
        t.y = MAX_SECOND ? max_nan(t.y, o.y) : t.y + o.y;
    }
    return t;
}

// The same for a CTA of one row per threadIdx.y.
template <bool MAX_SECOND>
__device__ __forceinline__ float2 reduce_row(float a, float b, float2* red) {
    const int wpr = blockDim.x >> 5;
    return reduce_row<MAX_SECOND>(a, b, red + threadIdx.y * wpr, threadIdx.x >> 5, wpr, [] { __syncthreads(); });
}

// 1 / sqrt(sum / H + eps).
__device__ __forceinline__ float row_rstd(float sum, float inv_h, float eps) { return rsqrtf(fmaf(sum, inv_h, eps)); }

template <typename T, int VEC>
__device__ __forceinline__ void load_weight(const void* w, int w32, size_t i, float off, float (&f)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = 1.0f + off;
    } else if (w32) {
        const float* p = static_cast<const float*>(w) + i;
        if constexpr (VEC == 1) {
            f[0] = *p + off;
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const float4 q = *reinterpret_cast<const float4*>(p + k);
                f[k] = q.x + off;
                f[k + 1] = q.y + off;
                f[k + 2] = q.z + off;
                f[k + 3] = q.w + off;
            }
        }
    } else {
        RawVec<T, VEC> v;
        v.load(static_cast<const T*>(w) + i);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = v.get(k) + off;
    }
}

// How a row's largest |u| becomes codes: u is multiplied by `pre` and then by
// `inv`.  pre is 1 unless the row is so small that Q / max|u| would overflow.
struct Quant {
    float pre, inv;
};
__device__ __forceinline__ Quant make_quant(float amax, float q) {
    Quant z;
    z.pre = amax < 1e-30f ? 18446744073709551616.0f : 1.0f;
    z.inv = amax > 0.0f ? q * (1.0f / (amax * z.pre)) : 0.0f;
    return z;
}

// A row's scale: NaN where the row, its sum of squares or a product with its weight is infinite or NaN, and 0 where all
// products are 0, whatever rstd is (infinite for a row of zeros without eps).
__device__ __forceinline__ float row_scale(float sum, float amax, float rstd, float q) {
    const float inf = -neg_inf();
    return !(sum < inf && amax < inf) ? quiet_nan() : amax > 0.f ? amax * rstd / q : 0.f;
}

// Codes of VEC elements.  |u inv| is at most Q up to a few roundings, so rounding cannot leave the codes' range.
// int8: added to 1.5 * 2^23 a float's low byte is the nearest integer (ties to even) in two's complement; the
// float-to-integer conversion runs at an eighth of that addition's rate.
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&u)[VEC], const Quant& z, int out) {
    constexpr float kRound = 12582912.0f;
    float v[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = __fmul_rn(u[k], z.inv);  // rounded before the addition below, not fused with it
    if (z.pre != 1.0f) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = __fmul_rn(u[k] * z.pre, z.inv);
    }
    if constexpr (VEC == 1) {
        p[0] = out == VH_NORM_INT8 ? (uint8_t)__float_as_uint(v[0] + kRound)
                                   : (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[VEC / 4];
        if (out == VH_NORM_INT8) {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const uint32_t lo = __byte_perm(__float_as_uint(v[k] + kRound), __float_as_uint(v[k + 1] + kRound), 0x0040);
                const uint32_t hi = __byte_perm(__float_as_uint(v[k + 2] + kRound), __float_as_uint(v[k + 3] + kRound), 0x0040);
                w[k / 4] = __byte_perm(lo, hi, 0x5410);
            }
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[k], v[k + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[k + 2], v[k + 3]), __NV_SATFINITE, __NV_E4M3);
                w[k / 4] = lo | (hi << 16);
            }
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// Rows of any alignment, as the aligned 16-byte slots that they touch: slot v holds elements [v VEC - shift, + VEC).
// The first and last slot of a row may hold elements of its neighbours, which other threads write: there the row's own
// elements are read and written one by one.
template <typename T, int VEC>
__device__ __forceinline__ void load_slot(RawVec<T, VEC>& r, const T* row, int e, int H) {
    if (e >= 0 && e + VEC <= H) {
        r.load(row + e);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) r.put(k, e + k >= 0 && e + k < H ? row[e + k] : from_f32<T>(0.f));
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_slot(T* row, int e, int H, const float (&f)[VEC], bool whole = true) {
    if (whole && e >= 0 && e + VEC <= H) {
        RawVec<T, VEC> o;
        pack_vec<T, VEC>(o, f);
        o.store(row + e);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (e + k >= 0 && e + k < H) row[e + k] = from_f32<T>(f[k]);
    }
}

// The weights of a slot (0 outside the row).  They lie across two aligned vectors, from which they are shifted; where
// those would reach past the weights, and for fp32 weights of 16-bit rows, they are read one by one.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight_slot(const void* w, int w32, int e, int H, float off, float (&f)[VEC]) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(w), at = base + (long long)e * (int)sizeof(T), lo = at & ~uintptr_t(15);
    if (w != nullptr && (sizeof(T) == 4 || !w32) && e >= 0 && lo >= base && lo + 32 <= base + (size_t)H * sizeof(T)) {
        RawVec<T, VEC> a, b, r;
        a.load(reinterpret_cast<const T*>(lo));
        b.load(reinterpret_cast<const T*>(lo + 16));
        const bool by8 = at & 8, by4 = at & 4;
        uint32_t t[6], q[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = by8 ? (i < 2 ? a.u[i + 2] : b.u[i - 2]) : (i < 4 ? a.u[i] : b.u[i - 4]);
#pragma unroll
        for (int i = 0; i < 5; ++i) q[i] = by4 ? t[i + 1] : t[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) r.u[i] = sizeof(T) == 4 ? q[i] : __funnelshift_r(q[i], q[i + 1], (uint32_t)(at & 2) * 8);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = r.get(k) + off;
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        float v = 0.f;
        if (e + k >= 0 && e + k < H) {
            v = 1.f;
            if (w != nullptr) v = w32 ? static_cast<const float*>(w)[e + k] : to_f32(static_cast<const T*>(w)[e + k]);
            v += off;
        }
        f[k] = v;
    }
}

// One row per threadIdx.y, NV vectors of VEC elements per thread, the row in registers.  SHIFT: by slots; all tensors'
// rows lie alike in them (codes in slots of VEC bytes).
template <typename T, int VEC, int NV, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) k_norm(const NormArgs a) {
    __shared__ float2 red[32];
    rows_wait();
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.T;
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride;
    const T* r = static_cast<const T*>(a.r) + (live ? row : 0) * a.r_stride;
    T* h = static_cast<T*>(a.h) + (live ? row : 0) * a.h_stride;
    const int shift = SHIFT ? (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)) : 0;
    const int nvec = SHIFT ? (a.H + shift + VEC - 1) / VEC : a.H / VEC;
    RawVec<T, VEC> xv[NV], rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (live && v < nvec) {
            if constexpr (SHIFT) {
                load_slot<T, VEC>(xv[j], x, v * VEC - shift, a.H);
                if (a.r != nullptr) load_slot<T, VEC>(rv[j], r, v * VEC - shift, a.H);
            } else {
                xv[j].load(x + (size_t)v * VEC);
                if (a.r != nullptr) rv[j].load(r + (size_t)v * VEC);
            }
        }
    }
    float u[NV][VEC];
    float ss = 0.f, amax = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (live && v < nvec) {
            float w[VEC];
            if constexpr (SHIFT)
                load_weight_slot<T, VEC>(a.w, a.w32, v * VEC - shift, a.H, a.w_offset, w);
            else
                load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) u[j][k] = xv[j].get(k) + (a.r != nullptr ? rv[j].get(k) : 0.f);
            if (a.h != nullptr) {
                if constexpr (SHIFT) {
                    store_slot<T, VEC>(h, v * VEC - shift, a.H, u[j]);
                } else {
                    RawVec<T, VEC> o;
                    pack_vec<T, VEC>(o, u[j]);
                    o.store(h + (size_t)v * VEC);
                }
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                ss = fmaf(u[j][k], u[j][k], ss);
                u[j][k] *= w[k];
                amax = max_nan(amax, fabsf(u[j][k]));
            }
        }
    }
    const float2 tot = reduce_row<true>(ss, amax, red);
    const float rstd = row_rstd(tot.x, a.inv_h, a.eps);
    if (!live) return;
    if (a.out == VH_NORM_SAME) {
        T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nvec) {
                float f[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[k] = u[j][k] * rstd;
                if constexpr (SHIFT) {
                    store_slot<T, VEC>(y, v * VEC - shift, a.H, f);
                } else {
                    RawVec<T, VEC> o;
                    pack_vec<T, VEC>(o, f);
                    o.store(y + (size_t)v * VEC);
                }
            }
        }
    } else {
        const float q = a.out == VH_NORM_INT8 ? 127.0f : 448.0f;
        const Quant z = make_quant(tot.y, q);
        uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * blockDim.x, e = v * VEC - shift;
            if (v < nvec) {
                if (!SHIFT || (e >= 0 && e + VEC <= a.H)) {
                    store_codes<VEC>(y + e, u[j], z, a.out);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        if (e + k >= 0 && e + k < a.H) {
                            const float one[1] = {u[j][k]};
                            store_codes<1>(y + e + k, one, z, a.out);
                        }
                }
            }
        }
        if (threadIdx.x == 0) a.scales[row] = row_scale(tot.x, tot.y, rstd, q);
    }
}

// Rows too wide for registers: one CTA per row, read twice.  Every thread
// reads an element for the last time just before it writes it, so the outputs
// may lie on the inputs as in the kernel above.
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(const NormArgs a) {
    __shared__ float2 red[32];
    rows_wait();
    const long long row = blockIdx.x;
    const int nvec = a.H / VEC;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = static_cast<const T*>(a.r) + row * a.r_stride;
    auto load = [&](int v, float (&hv)[VEC], float (&w)[VEC]) {
        RawVec<T, VEC> xv, rv;
        xv.load(x + (size_t)v * VEC);
        if (a.r != nullptr) rv.load(r + (size_t)v * VEC);
        load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) hv[k] = xv.get(k) + (a.r != nullptr ? rv.get(k) : 0.f);
    };
    float ss = 0.f, amax = 0.f;
    for (int v = threadIdx.x; v < nvec; v += kWideThreads) {
        float hv[VEC], w[VEC];
        load(v, hv, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            ss = fmaf(hv[k], hv[k], ss);
            amax = max_nan(amax, fabsf(hv[k] * w[k]));
        }
    }
    const float2 tot = reduce_row<true>(ss, amax, red);
    const float rstd = row_rstd(tot.x, a.inv_h, a.eps);
    const float q = a.out == VH_NORM_INT8 ? 127.0f : 448.0f;
    const Quant z = make_quant(tot.y, q);
    for (int v = threadIdx.x; v < nvec; v += kWideThreads) {
        float hv[VEC], w[VEC];
        load(v, hv, w);
        if (a.h != nullptr) {
            RawVec<T, VEC> o;
            pack_vec<T, VEC>(o, hv);
            o.store(static_cast<T*>(a.h) + row * a.h_stride + (size_t)v * VEC);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) hv[k] *= w[k];
        if (a.out == VH_NORM_SAME) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) hv[k] *= rstd;
            RawVec<T, VEC> o;
            pack_vec<T, VEC>(o, hv);
            o.store(static_cast<T*>(a.y) + row * a.y_stride + (size_t)v * VEC);
        } else {
            store_codes<VEC>(static_cast<uint8_t*>(a.y) + row * a.y_stride + (size_t)v * VEC, hv, z, a.out);
        }
    }
    if (a.out != VH_NORM_SAME && threadIdx.x == 0) a.scales[row] = row_scale(tot.x, tot.y, rstd, q);
}

// ---------------------------------------------------------------------------
// Gradient.  CTA c takes tokens c, c + grid, ...; a thread keeps its columns'
// share of dw in registers and leaves it in part[c][H]; a second kernel adds
// the shares in CTA order, so the sums do not change from call to call.

// The rows come by bulk copies into a ring of `depth` places in shared memory, so that loads are in flight whatever
// the registers hold.  A place holds ty tokens, so that narrow rows fill a CTA.  tx * ty threads sum, reduce (one
// barrier) and write a group of tokens; a further warp refills a place, a lane per row, when they are done with it.
//   8192 x 2048 bf16: 29.6 us, against 30.2 us with the next token's vectors in registers, where 64 registers a
//   thread left no room for a second token, and 42.1 us with a thread of the summing warps refilling.
//   16384 x 512: 18.9 us, against 46.0 us with one token at a time.
// Waits are for copies that the CTA has issued and for its own warps; should one expire (they are bounded) the results
// of that group and of the CTA's later ones are NaN, no further copies are made, and the refilling warp waits (again with
// a limit) for those in flight before it leaves.
//
// ROWS: whole aligned vectors of VEC elements; or rows that lie alike in their 16-byte slots (VEC as before); or rows of
// any alignment (VEC 1).  In the last two a token's place holds the 16-byte granules that its row touches.  What those
// hold beside the row is its neighbours' (or the gap between rows); granules that reach past the ends of the tensor are not
// copied, and the elements in them are stored one by one.
// Where rows lie alike, the start of a row in its slot repeats every `period` tokens, and a CTA takes tokens of one
// start only: so a thread's vectors hold the same columns of every token, as its weights and its share of dw need.
//   8191 x 2561 bf16: 98.9 us with loads of single elements, 63.1 us element by element out of the ring, 43 us by slots;
//   2047 x 8191: 61 and 41 us, 16383 x 257: 40 and 21 us, 4000 x 1025 fp16: 19 and 20 us.
// kAny is left with rows that lie differently in each tensor and fp32 rows too wide for slots; from 4,097 elements on, 16 a
// thread, it spills registers.
enum Rows { kWhole, kAlike, kAny };

// What a row at `p` holds outside [lo, hi), into its place.
template <typename T>
__device__ __forceinline__ void store_ends(uint8_t* to, const T* p, uint32_t bytes, uintptr_t lo, uintptr_t hi) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    T* at = reinterpret_cast<T*>(to + (b & 15));
    int head, tail;
    outside_window(b, bytes, (int)sizeof(T), lo, hi, head, tail);
    for (int i = 0; i < head; ++i) at[i] = p[i];
    for (int i = tail; i < (int)(bytes / sizeof(T)); ++i) at[i] = p[i];
}

template <typename T, int VEC, int NV, Rows ROWS>
__global__ void __launch_bounds__(kMaxThreads + 32)
    k_norm_grad(const NormGradArgs a, const int tx, const int ty, const int depth, const uint32_t pitch, const int period,
                const int stride /* CTAs of one start */, const bool dx_alike) {
    extern __shared__ __align__(128) uint8_t ring[];  // [depth][ty tokens][h, dy, dh][pitch]
    __shared__ float2 red[2][32];
    __shared__ unsigned long long full[kMaxRing], empty[kMaxRing];
    __shared__ volatile bool lost;  // a wait for a copy has expired
    const int workers = tx * ty;
    const int tid = threadIdx.x, lane = tid & 31;
    // this CTA's tokens are tok0, tok0 + period, ..: `mine` of them, in groups of ty
    const int tok0 = ROWS == kAlike ? (int)blockIdx.x % period : 0, cta = ROWS == kAlike ? (int)blockIdx.x / period : blockIdx.x;
    const int step = ROWS == kAlike ? period : 1;
    const int mine = (a.T - 1 - tok0) / step + 1;
    const int shift =
        ROWS == kAlike
            ? (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.h) + tok0 * a.h_stride) & 15) / sizeof(T))
            : 0;
    const int nvec = ROWS == kAlike ? (a.H + shift + VEC - 1) / VEC : a.H / VEC;
    const uint32_t place = (uint32_t)ty * 3 * pitch, row_bytes = (uint32_t)(a.H * sizeof(T));
    if (tid == 0) {
        for (int i = 0; i < depth; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], (uint32_t)workers / 32);
        }
        lost = false;
        ptx::fence_barrier_init();
    }
    __syncthreads();
    rows_wait();
    const int groups = (mine - 1) / ty + 1;
    const int n = groups > cta ? (groups - 1 - cta) / stride + 1 : 0;

    if (tid >= workers) {
        // a lane per row of a place: h, dy, dh of up to eight tokens
        rows_fence_async();
        const int q = lane / 3, which = lane - 3 * q;
        const T* rows = static_cast<const T*>(which == 0 ? a.h : which == 1 ? a.dy : a.dh);
        const long long pitch_of = which == 0 ? a.h_stride : which == 1 ? a.dy_stride : a.dh_stride;
        int i = 0;
        for (int s = 0, ph = 1; i < n; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_done(&empty[s], ph) && !lost)) break;
            const int i0 = (cta + i * stride) * ty;
            const bool on = rows != nullptr && q < min(ty, mine - i0);
            const long long t = tok0 + ((long long)i0 + q) * step;
            const T* p = rows + (on ? t : 0) * pitch_of;
            uint8_t* to = ring + (size_t)s * place + (size_t)lane * pitch;
            uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + row_bytes;
            if (ROWS != kWhole) {
                const uintptr_t b = lo, start = reinterpret_cast<uintptr_t>(rows);
                copy_window(b, row_bytes, start, start + (uintptr_t)((a.T - 1) * pitch_of) * sizeof(T) + row_bytes, lo, hi);
                if (on && (lo > b || hi < b + row_bytes)) {
                    store_ends(to, p, row_bytes, lo, hi);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later token's copy goes there
                }
                to += lo - (b & ~uintptr_t(15));
            }
            const uint32_t bytes = on ? (uint32_t)(hi - lo) : 0;
            const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, bytes);
            __syncwarp();  // lane 0 arrives for all: after every lane's stores of row ends
            if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], all);
            __syncwarp();
            if (bytes != 0) bulk_copy(to, reinterpret_cast<const void*>(lo), bytes, &full[s]);
            if (++s == depth) {
                s = 0;
                ph ^= 1;
            }
        }
        for (int j = max(0, i - depth); j < i; ++j) ptx::mbar_drain(&full[j % depth], (uint32_t)(j / depth) & 1u);
        return;
    }

    const int ry = tid / tx, rx = tid - ry * tx, wpr = tx >> 5;
    auto sync = [&] { asm volatile("bar.sync 1, %0;" ::"r"(workers) : "memory"); };
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = rx + j * tx;
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[j][k] = dw[j][k] = 0.f;
        if (v < nvec) {
            if constexpr (ROWS == kAlike)
                load_weight_slot<T, VEC>(a.w, a.w32, v * VEC - shift, a.H, a.w_offset, w[j]);
            else
                load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w[j]);
        }
    }
    bool there = true;
    for (int i = 0, s = 0, ph = 0; i < n; ++i) {
        const int i0 = (cta + i * stride) * ty;
        const bool live = ry < mine - i0;
        const long long token = tok0 + ((long long)i0 + ry) * step;
        const uint8_t* pl = ring + (size_t)s * place + (uint32_t)ry * 3 * pitch;
        auto at = [&](const uint8_t* p, const void* base, long long stride) {  // where a row lies in its place
            const uintptr_t b = ROWS != kAny ? 0 : reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + token * stride);
            return reinterpret_cast<const T*>(p + (b & 15));
        };
        const T* hs = at(pl, a.h, a.h_stride);
        const T* ys = at(pl + pitch, a.dy, a.dy_stride);
        const T* es = at(pl + 2 * pitch, a.dh, a.dh_stride);
        there = there && mbar_done(&full[s], ph);
        float ss = there ? 0.f : quiet_nan(), dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = rx + j * tx;
            if (live && v < nvec) {
                RawVec<T, VEC> hv, yv;
                hv.load(hs + v * VEC);
                yv.load(ys + v * VEC);
                if constexpr (ROWS == kAlike) {
                    const int e = v * VEC - shift;
                    if (e < 0 || e + VEC > a.H) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            if (e + k < 0 || e + k >= a.H) {
                                hv.put(k, from_f32<T>(0.f));
                                yv.put(k, from_f32<T>(0.f));
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float f = hv.get(k);
                    ss = fmaf(f, f, ss);
                    dot = fmaf(yv.get(k) * w[j][k], f, dot);
                }
            }
        }
        const float2 tot = reduce_row<false>(ss, dot, red[i & 1] + ry * wpr, rx >> 5, wpr, sync);
        const float rstd = row_rstd(tot.x, a.inv_h, a.eps);
        const float back = -tot.y * rstd * rstd * rstd * a.inv_h;  // dx = rstd g + back h + dh
        T* dx = static_cast<T*>(a.dx) + token * a.dx_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = rx + j * tx;
            if (live && v < nvec) {
                RawVec<T, VEC> hv, yv, ev;
                hv.load(hs + v * VEC);
                yv.load(ys + v * VEC);
                if (a.dh != nullptr) ev.load(es + v * VEC);
                float o[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float f = hv.get(k), d = yv.get(k) * rstd;
                    dw[j][k] = fmaf(d, f, dw[j][k]);
                    o[k] = fmaf(d, w[j][k], fmaf(back, f, a.dh != nullptr ? ev.get(k) : 0.f));
                }
                if constexpr (ROWS == kAlike) {
                    store_slot<T, VEC>(dx, v * VEC - shift, a.H, o, dx_alike);
                } else {
                    RawVec<T, VEC> p;
                    pack_vec<T, VEC>(p, o);
                    p.store(dx + (size_t)v * VEC);
                }
            }
        }
        if (!there) lost = true;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[s]);
        if (++s == depth) {
            s = 0;
            ph ^= 1;
        }
    }
    if (a.part == nullptr) return;
    // Only where the summing kernel follows.  The grid is one resident wave: CTAs of the next kernel that came before this
    // one's end would take places that the wave after needs (8192 x 2048 bf16: 39.7 us a call with the signal at the start).
    if (a.summed) rows_launch_dependents();
    // A share lies as its vectors do, so that they are stored whole (27 x 8192 bf16: 5.7 us, against 8.4 us with stores of
    // single elements 32 bytes apart): by slots it begins `shift` places before its first column (300 x 4097: 7.9 against
    // 10.4 us).  Shares that are first added in shared memory leave it column by column anyway, and begin with the first
    // (1000 x 1025: 8.2 against 9.9 us).
    const bool slots = ROWS == kAlike && a.part_pitch != a.H;
    float* p = a.part + (size_t)blockIdx.x * a.part_pitch;
    float* to = ty > 1 ? reinterpret_cast<float*>(ring) + (size_t)ry * a.H : p;  // [ty][H]
    const bool whole = VEC > 1 && (ROWS == kWhole || slots) && (reinterpret_cast<uintptr_t>(to) & 15) == 0;
    if (ty > 1) sync();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = rx + j * tx;
        if (v >= nvec) continue;
        if constexpr (VEC > 1) {
            if (whole) {
#pragma unroll
                for (int k = 0; k < VEC; k += 4)
                    *reinterpret_cast<float4*>(to + v * VEC + k) = make_float4(dw[j][k], dw[j][k + 1], dw[j][k + 2], dw[j][k + 3]);
                continue;
            }
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int c = v * VEC - shift + k;
            if (ROWS != kAlike || (c >= 0 && c < a.H)) to[c] = dw[j][k];
        }
    }
    if (ty == 1) return;
    sync();
    for (int c = tid; c < a.H; c += workers) {
        float t = 0.f;
        for (int q = 0; q < ty; ++q) t += reinterpret_cast<const float*>(ring)[(size_t)q * a.H + c];
        p[c] = t;
    }
}

// Rows too wide for registers: read twice; the CTA's share of dw lives in its
// part[c] row, each element touched by one thread only.
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_grad_wide(const NormGradArgs a) {
    __shared__ float2 red[2][32];
    if (a.summed) rows_launch_dependents();
    rows_wait();
    const int nvec = a.H / VEC;
    float* p = a.part == nullptr ? nullptr : a.part + (size_t)blockIdx.x * a.H;
    int slot = 0;
    bool first = true;
    for (long long row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1, first = false) {
        const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* dh = static_cast<const T*>(a.dh) + row * a.dh_stride;
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
        float ss = 0.f, dot = 0.f;
        for (int v = threadIdx.x; v < nvec; v += kWideThreads) {
            RawVec<T, VEC> hv, yv;
            float w[VEC];
            hv.load(h + (size_t)v * VEC);
            yv.load(dy + (size_t)v * VEC);
            load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float f = hv.get(k);
                ss = fmaf(f, f, ss);
                dot = fmaf(yv.get(k) * w[k], f, dot);
            }
        }
        const float2 tot = reduce_row<false>(ss, dot, red[slot]);
        const float rstd = row_rstd(tot.x, a.inv_h, a.eps);
        const float mean = tot.y * rstd * a.inv_h;
        for (int v = threadIdx.x; v < nvec; v += kWideThreads) {
            RawVec<T, VEC> hv, yv, ev;
            float w[VEC], f[VEC];
            hv.load(h + (size_t)v * VEC);
            yv.load(dy + (size_t)v * VEC);
            if (a.dh != nullptr) ev.load(dh + (size_t)v * VEC);
            load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float n = hv.get(k) * rstd, d = yv.get(k);
                if (p != nullptr) {
                    float* q = p + (size_t)v * VEC + k;
                    *q = fmaf(d, n, first ? 0.f : *q);
                }
                f[k] = fmaf(rstd, fmaf(-n, mean, d * w[k]), a.dh != nullptr ? ev.get(k) : 0.f);
            }
            RawVec<T, VEC> o;
            pack_vec<T, VEC>(o, f);
            o.store(dx + (size_t)v * VEC);
        }
    }
}

// The tokens' shares of dweight: n of them, `pitch` floats apart; column c of share r lies (base + r step) & mask places on.
struct Parts {
    const float* at;
    int n, pitch;
    uint32_t base, step, mask;
};

// dweight[c] = sum of the shares' columns c, in order: 32 columns x GROUPS row groups per CTA, loads in batches.
template <int GROUPS, bool SLOTS>
__global__ void __launch_bounds__(32 * GROUPS) k_sum_parts(const Parts p, const int H, float* out) {
    const float* part = p.at;
    const int n = p.n;
    constexpr int kBatch = 10;
    __shared__ float s[GROUPS][33];
    rows_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < H)
        for (int r0 = threadIdx.y; r0 < n; r0 += GROUPS * kBatch) {
            float x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * GROUPS;
                if constexpr (SLOTS)
                    x[i] = r < n ? part[(size_t)r * p.pitch + c + ((p.base + (uint32_t)r * p.step) & p.mask)] : 0.f;
                else
                    x[i] = r < n ? part[(size_t)r * H + c] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v += x[i];
        }
    s[threadIdx.y][threadIdx.x] = v;
    rows_launch_dependents();
    __syncthreads();
    if (threadIdx.y == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) t += s[g][threadIdx.x];
        out[c] = t;
    }
}

template <typename... P, typename... A>
static cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

static inline bool mult16(const void* p, long long stride_elems, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride_elems * size) % 16 == 0;
}

// Threads per row (a multiple of 32) for nvec vectors, nv per thread.
static inline int row_threads(int nvec, int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; }

template <typename T, int VEC, bool SHIFT>
static cudaError_t norm_vec(const NormArgs& a, cudaStream_t s) {
    const int nvec = SHIFT ? (a.H + 2 * (VEC - 1)) / VEC : a.H / VEC;  // SHIFT: of the least favourable row
    auto go = [&](auto kernel, int nv) {
        const int tx = row_threads(nvec, nv);
        const int ty = std::max(1, 128 / tx);
        return launch(kernel, dim3((unsigned)((a.T - 1) / ty + 1)), dim3(tx, ty), 0, s, a);
    };
    // Two vectors a thread: 16384 x 2048 bf16 36.8 us to int8, 40.4 us to bf16 (36.4 / 40.8 since the kernel lets no other
    // start early), against 42.4 / 41.2 us with one, 37.2 /
    // 41.1 us with four and 41.3 / 43.5 us with eight (a warp per row).  One where that leaves less than two warps.
    if (nvec <= 64) return go(k_norm<T, VEC, 1, SHIFT>, 1);
    if (nvec <= kMaxThreads * 2) return go(k_norm<T, VEC, 2, SHIFT>, 2);
    if (nvec <= kMaxThreads * 4) return go(k_norm<T, VEC, 4, SHIFT>, 4);
    if constexpr (VEC == 1) {
        if (nvec <= kMaxThreads * 8) return go(k_norm<T, 1, 8, false>, 8);
    }
    if constexpr (SHIFT)
        return launch(k_norm_wide<T, 1>, dim3((unsigned)a.T), dim3(kWideThreads), 0, s, a);
    else
        return launch(k_norm_wide<T, VEC>, dim3((unsigned)a.T), dim3(kWideThreads), 0, s, a);
}

template <typename T>
static cudaError_t norm_type(const NormArgs& a, cudaStream_t s) {
    constexpr int V = kVecOf<T>;
    const int size = (int)sizeof(T);
    const bool q8 = a.out != VH_NORM_SAME;
    const bool vec = a.H % V == 0 && mult16(a.x, a.x_stride, size) && (!a.r || mult16(a.r, a.r_stride, size)) &&
                     (!a.h || mult16(a.h, a.h_stride, size)) && (!a.w || mult16(a.w, 0, size)) &&
                     (q8 ? (reinterpret_cast<uintptr_t>(a.y) % V == 0 && a.y_stride % V == 0)
                         : mult16(a.y, a.y_stride, size));
    if (vec) return norm_vec<T, V, false>(a, s);
    // Rows that lie alike in their slots, whatever their alignment: 8191 x 2561 bf16 38.0 us by slots, 66 us by elements;
    // fp32 50.2 us by slots.
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x);
    auto alike = [&](const void* p, long long stride, int bytes) {
        return reinterpret_cast<uintptr_t>(p) / bytes % V == at / size % V && (stride - a.x_stride) % V == 0;
    };
    const bool slots = (!a.r || alike(a.r, a.r_stride, size)) && (!a.h || alike(a.h, a.h_stride, size)) &&
                       alike(a.y, a.y_stride, q8 ? 1 : size);
    return slots ? norm_vec<T, V, true>(a, s) : norm_vec<T, 1, false>(a, s);
}

// sum: the shares that are left to add up (in: at most n); one is dweight itself.
template <typename T>
static cudaError_t grad_type(NormGradArgs a, Parts& sum, float* dweight, cudaStream_t s) {
    constexpr int V = kVecOf<T>;
    const int size = (int)sizeof(T);
    const bool vec = a.H % V == 0 && mult16(a.h, a.h_stride, size) && mult16(a.dy, a.dy_stride, size) &&
                     (!a.dh || mult16(a.dh, a.dh_stride, size)) && mult16(a.dx, a.dx_stride, size) &&
                     (!a.w || mult16(a.w, 0, size));
    auto alike = [&](const void* p, long long stride) {
        return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(a.h)) & 15) == 0 && (stride - a.h_stride) % V == 0;
    };
    const bool dx_alike = alike(a.dx, a.dx_stride);
    // n vectors (or elements) a row, nv a thread; `period`: the tokens after which a row's start in its slot repeats
    auto go = [&](auto kernel, int n, int nv, size_t pitch, int period, bool by_slots) -> cudaError_t {
        const int tx = row_threads(n, nv);
        const int ty = std::max(1, std::min(256 / tx, (int)(kRingBytes / kMaxRing / (3 * pitch))));  // keeps the ring deep
        const size_t place = (size_t)ty * 3 * pitch;
        const int depth = std::max(2, std::min(kMaxRing, (int)(kRingBytes / place)));
        // One resident wave; from half a wave on, three groups a CTA before more CTAs, since each leaves a share of dw that
        // is written and read again (585 x 2048 bf16: 8.6 us against 12.0 us with a CTA per token, 393 x 8192: 14.0
        // against 20.5 us).  All of it for each start of a row.
        const int per_sm = std::min(4, (int)(kSmRingBytes / (depth * place)));
        const int groups = (a.T - 1) / period / ty + 1;
        const int each = std::max(1, std::min({sum.n / period, groups, 152 * per_sm / period,
                                               std::max(76 * per_sm / period, groups / 3)}));
        sum.n = std::min(sum.n, each * period);
        a.part_pitch = a.H;
        a.summed = a.part != nullptr && sum.n > 1;
        if (sum.n == 1) {
            a.part = dweight;  // the only share: no second launch (1 x 256: 2.6 against 4.6 us)
        } else if (by_slots && ty == 1 && a.H % V != 0) {  // the workspace has room for slots in rows of such widths
            sum.pitch = a.part_pitch = (a.H + 2 * (V - 1)) / V * V;
            sum.base = (uint32_t)((reinterpret_cast<uintptr_t>(a.h) & 15) / size);
            sum.step = (uint32_t)(a.h_stride % V);
            sum.mask = V - 1;
        }
        if (depth * place > kMaxRingBytes) return cudaErrorInvalidValue;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxRingBytes);
        if (e != cudaSuccess) return e;
        return launch(kernel, dim3((unsigned)sum.n), dim3(tx * ty + 32), depth * place, s, a, tx, ty, depth, (uint32_t)pitch,
                      period, each, dx_alike);
    };
    if (vec) {
        // Two vectors a thread halve what a thread spends on each token's reduction (8192 x 2048 bf16: 28.8 against
        // 30.6 us with one).
        const int n = a.H / V;
        const size_t pitch = (size_t)a.H * size;
        if (n <= 64) return go(k_norm_grad<T, V, 1, kWhole>, n, 1, pitch, 1, false);
        if (n <= kMaxThreads * 2) return go(k_norm_grad<T, V, 2, kWhole>, n, 2, pitch, 1, false);
        if (n <= kMaxThreads * 4) return go(k_norm_grad<T, V, 4, kWhole>, n, 4, pitch, 1, false);
        a.summed = a.part != nullptr && sum.n > 1;
        if (sum.n == 1) a.part = dweight;
        return launch(k_norm_grad_wide<T, V>, dim3((unsigned)sum.n), dim3(kWideThreads), 0, s, a);
    }
    const size_t pitch = ((size_t)a.H * size + 30) / 16 * 16;  // a row may start 15 bytes into its first granule
    // Where dx lies differently it is written by elements, so that its place does not change its bits.
    if (alike(a.dy, a.dy_stride) && (!a.dh || alike(a.dh, a.dh_stride))) {
        int period = 1;
        while (a.h_stride * period % V != 0) period *= 2;  // V is a power of two
        const int n = (a.H + 2 * (V - 1)) / V;             // slots of the least favourable row
        if (n <= 64) return go(k_norm_grad<T, V, 1, kAlike>, n, 1, pitch, period, true);
        if (n <= kMaxThreads * 2) return go(k_norm_grad<T, V, 2, kAlike>, n, 2, pitch, period, true);
        if (n <= kMaxThreads * 4) return go(k_norm_grad<T, V, 4, kAlike>, n, 4, pitch, period, true);
    }
    if (a.H <= kMaxThreads * 8) return go(k_norm_grad<T, 1, 8, kAny>, a.H, 8, pitch, 1, false);
    if (a.H <= kMaxThreads * 16) return go(k_norm_grad<T, 1, 16, kAny>, a.H, 16, pitch, 1, false);
    a.summed = a.part != nullptr && sum.n > 1;
    if (sum.n == 1) a.part = dweight;
    return launch(k_norm_grad_wide<T, 1>, dim3((unsigned)sum.n), dim3(kWideThreads), 0, s, a);
}

}  // namespace norm

int norm_grad_parts(int T) { return std::min(T, kNormGradParts); }

cudaError_t launch_add_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s) {
    if (dtype == VH_BF16) return norm::norm_type<__nv_bfloat16>(a, s);
    if (dtype == VH_F16) return norm::norm_type<__half>(a, s);
    return norm::norm_type<float>(a, s);
}

cudaError_t launch_add_rmsnorm_grad(const NormGradArgs& a, int dtype, float* dweight, cudaStream_t s) {
    norm::Parts sum = {a.part, norm_grad_parts(a.T), a.H, 0, 0, 0};
    cudaError_t e = dtype == VH_BF16  ? norm::grad_type<__nv_bfloat16>(a, sum, dweight, s)
                    : dtype == VH_F16 ? norm::grad_type<__half>(a, sum, dweight, s)
                                      : norm::grad_type<float>(a, sum, dweight, s);
    if (e != cudaSuccess || dweight == nullptr || sum.n == 1) return e;
    auto add = [&](auto kernel, int groups) {
        return norm::launch(kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(32, groups), 0, s, sum, a.H, dweight);
    };
    if (sum.n <= norm::kFewParts)
        return sum.mask ? add(norm::k_sum_parts<8, true>, 8) : add(norm::k_sum_parts<8, false>, 8);
    return sum.mask ? add(norm::k_sum_parts<32, true>, 32) : add(norm::k_sum_parts<32, false>, 32);
}

}  // namespace vh
