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

#include "vh_kernels.h"
#include "vh_ptx.cuh"
#include "vh_rows.cuh"

namespace vh {
namespace norm {

constexpr int kMaxThreads = 512;  // register-resident rows: up to 128 registers a thread
constexpr int kWideThreads = 512;
constexpr int kMaxRing = 4;                // tokens in flight per CTA of the gradient
constexpr size_t kRingBytes = 56 * 1024;   // of shared memory per CTA that a ring of over two tokens stays below
constexpr size_t kSmRingBytes = 220 * 1024;  // of shared memory per SM for rings

// Sums of two values over the threads of one row (threadIdx.y) of the CTA.
// MAX_SECOND: the second value is a maximum instead of a sum.  All threads of
// the CTA call it; `slot` alternates between calls.  The lower half of a warp
// goes on with the first value and the upper half with the second, so both
// take one chain of shuffles.
template <bool MAX_SECOND>
__device__ __forceinline__ float2 reduce_row(float a, float b, float2 (*red)[32], int slot) {
    const int lane = threadIdx.x & 31;
    const bool second = lane >= 16;
    auto join = [&](float v, float o) { return MAX_SECOND && second ? fmaxf(v, o) : v + o; };
    const float other = __shfl_xor_sync(0xFFFFFFFFu, second ? a : b, 16);
    float v = join(second ? b : a, other);
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
    float2* row = red[slot] + threadIdx.y * wpr;
    if ((lane & 15) == 0) reinterpret_cast<float*>(row + (threadIdx.x >> 5))[lane >> 4] = v;
    __syncthreads();
    float2 t = row[0];
#pragma unroll 4
    for (int w = 1; w < wpr; ++w) {
        const float2 o = row[w];
        t.x += o.x;
        t.y = MAX_SECOND ? fmaxf(t.y, o.y) : t.y + o.y;
    }
    return t;
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

// One row per threadIdx.y, NV vectors of VEC elements per thread, the row in registers.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) k_norm(const NormArgs a) {
    __shared__ float2 red[1][32];
    rows_launch_dependents();
    rows_wait();
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.T;
    const int nvec = a.H / VEC;
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride;
    const T* r = static_cast<const T*>(a.r) + (live ? row : 0) * a.r_stride;
    T* h = static_cast<T*>(a.h) + (live ? row : 0) * a.h_stride;
    RawVec<T, VEC> xv[NV], rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (live && v < nvec) {
            xv[j].load(x + (size_t)v * VEC);
            if (a.r != nullptr) rv[j].load(r + (size_t)v * VEC);
        }
    }
    float u[NV][VEC];
    float ss = 0.f, amax = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (live && v < nvec) {
            float w[VEC];
            load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) u[j][k] = xv[j].get(k) + (a.r != nullptr ? rv[j].get(k) : 0.f);
            if (a.h != nullptr) {
                RawVec<T, VEC> o;
                pack_vec<T, VEC>(o, u[j]);
                o.store(h + (size_t)v * VEC);
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                ss = fmaf(u[j][k], u[j][k], ss);
                u[j][k] *= w[k];
                amax = fmaxf(amax, fabsf(u[j][k]));
            }
        }
    }
    const float2 tot = reduce_row<true>(ss, amax, red, 0);
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
                RawVec<T, VEC> o;
                pack_vec<T, VEC>(o, f);
                o.store(y + (size_t)v * VEC);
            }
        }
    } else {
        const float q = a.out == VH_NORM_INT8 ? 127.0f : 448.0f;
        const Quant z = make_quant(tot.y, q);
        uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nvec) store_codes<VEC>(y + (size_t)v * VEC, u[j], z, a.out);
        }
        if (threadIdx.x == 0) a.scales[row] = tot.y * rstd / q;
    }
}

// Rows too wide for registers: one CTA per row, read twice.  Every thread
// reads an element for the last time just before it writes it, so the outputs
// may lie on the inputs as in the kernel above.
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(const NormArgs a) {
    __shared__ float2 red[1][32];
    rows_launch_dependents();
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
            amax = fmaxf(amax, fabsf(hv[k] * w[k]));
        }
    }
    const float2 tot = reduce_row<true>(ss, amax, red, 0);
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
    if (a.out != VH_NORM_SAME && threadIdx.x == 0) a.scales[row] = tot.y * rstd / q;
}

// ---------------------------------------------------------------------------
// Gradient.  CTA c takes tokens c, c + grid, ...; a thread keeps its columns'
// share of dw in registers and leaves it in part[c][H]; a second kernel adds
// the shares in CTA order, so the sums do not change from call to call.

// Whole 16-byte vectors: the rows come by bulk copies into a ring of `depth` tokens in shared memory, so that loads
// are in flight whatever the registers hold (8192 x 2048 bf16: 28.7 against 30.2 us with the next token's vectors in
// registers, where 64 registers a thread left no room for a second token).  Token i is summed, reduced (one barrier)
// and written; behind that barrier every thread is done with token i - 1, whose place is refilled.
// A wait is for copies that the CTA itself has issued; should it expire (it is bounded) the token's results are NaN.
template <typename T, int NV>
__global__ void __launch_bounds__(kMaxThreads) k_norm_grad_ring(const NormGradArgs a, const int depth) {
    constexpr int VEC = kVecOf<T>;
    extern __shared__ __align__(128) uint8_t ring[];  // [depth][h, dy, dh][H]
    __shared__ float2 red[2][32];
    __shared__ unsigned long long full[kMaxRing];
    const int nvec = a.H / VEC;
    const uint32_t row_bytes = (uint32_t)(a.H * sizeof(T));
    const int streams = a.dh != nullptr ? 3 : 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < depth; ++i) ptx::mbar_init(&full[i], 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    rows_launch_dependents();
    rows_wait();
    const long long step = gridDim.x;
    const int n = (int)((a.T - blockIdx.x + step - 1) / step);  // tokens of this CTA
    auto fill = [&](int i) {                                    // by thread 0
        const long long row = blockIdx.x + i * step;
        const int s = i % depth;
        uint8_t* to = ring + (size_t)s * 3 * row_bytes;
        ptx::mbar_arrive_expect_tx(&full[s], streams * row_bytes);
        ptx::bulk_copy(to, static_cast<const T*>(a.h) + row * a.h_stride, row_bytes, &full[s]);
        ptx::bulk_copy(to + row_bytes, static_cast<const T*>(a.dy) + row * a.dy_stride, row_bytes, &full[s]);
        if (a.dh != nullptr)
            ptx::bulk_copy(to + 2 * row_bytes, static_cast<const T*>(a.dh) + row * a.dh_stride, row_bytes, &full[s]);
    };
    if (threadIdx.x == 0) {
        rows_fence_async();
        for (int i = 0; i < min(depth, n); ++i) fill(i);
    }
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < nvec) load_weight<T, VEC>(a.w, a.w32, (size_t)v * VEC, a.w_offset, w[j]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) dw[j][k] = 0.f;
    }
    T* dx = static_cast<T*>(a.dx) + blockIdx.x * a.dx_stride;
    for (int i = 0; i < n; ++i, dx += step * a.dx_stride) {
        const int s = i % depth;
        const T* hs = reinterpret_cast<const T*>(ring + (size_t)s * 3 * row_bytes);
        const T* ys = reinterpret_cast<const T*>(ring + ((size_t)s * 3 + 1) * row_bytes);
        const T* es = reinterpret_cast<const T*>(ring + ((size_t)s * 3 + 2) * row_bytes);
        const bool there = ptx::mbar_drain(&full[s], (i / depth) & 1u);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nvec) {
                RawVec<T, VEC> hv, yv;
                hv.load(hs + v * VEC);
                yv.load(ys + v * VEC);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float f = hv.get(k);
                    ss = fmaf(f, f, ss);
                    dot = fmaf(yv.get(k) * w[j][k], f, dot);
                }
            }
        }
        const float2 tot = reduce_row<false>(ss, dot, red, i & 1);
        if (threadIdx.x == 0 && i > 0 && i - 1 + depth < n) fill(i - 1 + depth);
        const float rstd = there ? row_rstd(tot.x, a.inv_h, a.eps) : quiet_nan();
        const float back = -tot.y * rstd * rstd * rstd * a.inv_h;  // dx = rstd g + back h + dh
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nvec) {
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
                RawVec<T, VEC> p;
                pack_vec<T, VEC>(p, o);
                p.store(dx + (size_t)v * VEC);
            }
        }
    }
    if (a.part == nullptr) return;
    float* p = a.part + (size_t)blockIdx.x * a.H;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < nvec)
#pragma unroll
            for (int k = 0; k < VEC; k += 4)
                *reinterpret_cast<float4*>(p + (size_t)v * VEC + k) =
                    make_float4(dw[j][k], dw[j][k + 1], dw[j][k + 2], dw[j][k + 3]);
    }
}

// Any other alignment or width: NE elements a thread, the next token's in registers while one is reduced and written.
template <typename T, int NE>
__global__ void __launch_bounds__(kMaxThreads) k_norm_grad(const NormGradArgs a) {
    __shared__ float2 red[2][32];
    rows_launch_dependents();
    rows_wait();
    T hn[NE], yn[NE], en[NE];
    auto request = [&](long long row) {
        const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* dh = static_cast<const T*>(a.dh) + row * a.dh_stride;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < a.H) {
                hn[j] = h[c];
                yn[j] = dy[c];
                if (a.dh != nullptr) en[j] = dh[c];
            }
        }
    };
    if (blockIdx.x < a.T) request(blockIdx.x);
    float w[NE], dw[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        float f[1] = {0.f};
        if (c < a.H) load_weight<T, 1>(a.w, a.w32, c, a.w_offset, f);
        w[j] = f[0];
        dw[j] = 0.f;
    }
    int slot = 0;
    for (long long row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        T hv[NE], yv[NE], ev[NE];
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            hv[j] = hn[j];
            yv[j] = yn[j];
            ev[j] = en[j];
        }
        if (row + gridDim.x < a.T) request(row + gridDim.x);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NE; ++j)
            if (threadIdx.x + j * blockDim.x < a.H) {
                const float f = to_f32(hv[j]);
                ss = fmaf(f, f, ss);
                dot = fmaf(to_f32(yv[j]) * w[j], f, dot);
            }
        const float2 tot = reduce_row<false>(ss, dot, red, slot);
        const float rstd = row_rstd(tot.x, a.inv_h, a.eps);
        const float mean = tot.y * rstd * a.inv_h;  // mean(g n)
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < a.H) {
                const float n = to_f32(hv[j]) * rstd, d = to_f32(yv[j]);
                dw[j] = fmaf(d, n, dw[j]);
                dx[c] = from_f32<T>(fmaf(rstd, fmaf(-n, mean, d * w[j]), a.dh != nullptr ? to_f32(ev[j]) : 0.f));
            }
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < a.H) a.part[(size_t)blockIdx.x * a.H + c] = dw[j];
    }
}

// Rows too wide for registers: read twice; the CTA's share of dw lives in its
// part[c] row, each element touched by one thread only.
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) k_norm_grad_wide(const NormGradArgs a) {
    __shared__ float2 red[2][32];
    rows_launch_dependents();
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
        const float2 tot = reduce_row<false>(ss, dot, red, slot);
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

// dweight[c] = sum of part[0..n)[c], in order: 32 columns x 32 row groups per CTA, loads in batches.
constexpr int kSumGroups = 32;
__global__ void __launch_bounds__(32 * kSumGroups) k_sum_parts(const float* part, int n, int H, float* out) {
    constexpr int kBatch = 10;
    __shared__ float s[kSumGroups][33];
    rows_launch_dependents();
    rows_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < H)
        for (int r0 = threadIdx.y; r0 < n; r0 += kSumGroups * kBatch) {
            float x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * kSumGroups;
                x[i] = r < n ? part[(size_t)r * H + c] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v += x[i];
        }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < kSumGroups; ++g) t += s[g][threadIdx.x];
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

template <typename T, int VEC>
static cudaError_t norm_vec(const NormArgs& a, cudaStream_t s) {
    const int nvec = a.H / VEC;
    auto go = [&](auto kernel, int nv) {
        const int tx = row_threads(nvec, nv);
        const int ty = std::max(1, 128 / tx);
        return launch(kernel, dim3((unsigned)((a.T + ty - 1) / ty)), dim3(tx, ty), 0, s, a);
    };
    // Two vectors a thread: 16384 x 2048 bf16 36.8 us to int8, 40.4 us to bf16, against 42.4 / 41.2 us with one, 37.2 /
    // 41.1 us with four and 41.3 / 43.5 us with eight (a warp per row).  One where that leaves less than two warps.
    if (nvec <= 64) return go(k_norm<T, VEC, 1>, 1);
    if (nvec <= kMaxThreads * 2) return go(k_norm<T, VEC, 2>, 2);
    if (nvec <= kMaxThreads * 4) return go(k_norm<T, VEC, 4>, 4);
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
    return vec ? norm_vec<T, V>(a, s) : norm_vec<T, 1>(a, s);
}

// `parts`: the CTAs that share the tokens (in: at most).
template <typename T>
static cudaError_t grad_type(const NormGradArgs& a, int& parts, cudaStream_t s) {
    constexpr int V = kVecOf<T>;
    const int size = (int)sizeof(T);
    const bool vec = a.H % V == 0 && mult16(a.h, a.h_stride, size) && mult16(a.dy, a.dy_stride, size) &&
                     (!a.dh || mult16(a.dh, a.dh_stride, size)) && mult16(a.dx, a.dx_stride, size) &&
                     (!a.w || mult16(a.w, 0, size));
    dim3 grid((unsigned)parts);
    if (!vec) {
        if (a.H <= kMaxThreads) return launch(k_norm_grad<T, 1>, grid, dim3(row_threads(a.H, 1)), 0, s, a);
        if (a.H <= kMaxThreads * 4) return launch(k_norm_grad<T, 4>, grid, dim3(row_threads(a.H, 4)), 0, s, a);
        if (a.H <= kMaxThreads * 8) return launch(k_norm_grad<T, 8>, grid, dim3(row_threads(a.H, 8)), 0, s, a);
        return launch(k_norm_grad_wide<T, 1>, grid, dim3(kWideThreads), 0, s, a);
    }
    const int nvec = a.H / V;
    if (nvec > kMaxThreads * 2) return launch(k_norm_grad_wide<T, V>, grid, dim3(kWideThreads), 0, s, a);
    const size_t token = 3 * (size_t)a.H * size;
    const int depth = std::max(2, std::min(kMaxRing, (int)(kRingBytes / token)));
    parts = std::min(parts, 152 * std::min(4, (int)(kSmRingBytes / (depth * token))));  // one resident wave
    grid.x = (unsigned)parts;
    auto go = [&](auto kernel, int nv) -> cudaError_t {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(depth * token));
        if (e != cudaSuccess) return e;
        return launch(kernel, grid, dim3(row_threads(nvec, nv)), depth * token, s, a, depth);
    };
    // two vectors a thread halve what a thread spends on each token's reduction (8192 x 2048 bf16: 28.8 against 30.6 us)
    return nvec <= 64 ? go(k_norm_grad_ring<T, 1>, 1) : go(k_norm_grad_ring<T, 2>, 2);
}

}  // namespace norm

int norm_grad_parts(int T) { return std::min(T, kNormGradParts); }

cudaError_t launch_add_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s) {
    if (dtype == VH_BF16) return norm::norm_type<__nv_bfloat16>(a, s);
    if (dtype == VH_F16) return norm::norm_type<__half>(a, s);
    return norm::norm_type<float>(a, s);
}

cudaError_t launch_add_rmsnorm_grad(const NormGradArgs& a, int dtype, float* dweight, cudaStream_t s) {
    int parts = norm_grad_parts(a.T);
    cudaError_t e = dtype == VH_BF16  ? norm::grad_type<__nv_bfloat16>(a, parts, s)
                    : dtype == VH_F16 ? norm::grad_type<__half>(a, parts, s)
                                      : norm::grad_type<float>(a, parts, s);
    if (e != cudaSuccess || dweight == nullptr) return e;
    return norm::launch(norm::k_sum_parts, dim3((unsigned)((a.H + 31) / 32)), dim3(32, norm::kSumGroups), 0, s,
                        (const float*)a.part, parts, a.H, dweight);
}

}  // namespace vh
