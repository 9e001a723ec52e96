// Rows to block-scaled 4 bits and back (the NVFP4 format of the 4-bit heads),
// and the tiled layout that the product of two 4-bit matrices reads.
//
//     g = given, or fp32(max|row| / (6 * 448)) for each row
//     s = e4m3(max|block| / (6 g)),  c = e2m1(x / (s g)),  both to the nearest, ties to even
//     value = c s g
//
// Codes are those of the exact quotient.  fp32 gives a quotient to a few units
// in the last place; only where that lies next to a border between two codes
// can it be on the wrong side.  Every border has at most two (e2m1) or four
// (e4m3) fraction bits, so "next to a border" is a test of the low mantissa
// bits, and the border is then compared exactly: border * s has at most seven
// bits, and fma(border * s, -g, |x|) rounds once, so its sign is that of the
// exact difference.  A block without such an element takes one multiply and
// one test per element.  g is brought near one first, so that nothing of this
// underflows.
//
// A thread has blocks of 16 elements in registers (32 bytes of 16-bit types),
// so a row is read once, whatever finds its scale: a row's threads are one
// warp or several of a CTA.  Bound: memory.
#include <algorithm>

#include "vh_nvfp4_tiles.h"
#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace q4 {

constexpr float kTop = 2688.0f;  // 6 * 448
constexpr uint32_t kNanScale = 0x7Fu;

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_code(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
    return __half2float(__ushort_as_half((unsigned short)h));
}
// Four bytes of codes (eight elements) as f16 pairs.
__device__ __forceinline__ void e2m1_values(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---------------------------------------------------------------------------
// A block of 16 elements as loaded.

template <typename T>
struct Block {
    static constexpr int N = 16 * (int)sizeof(T) / 4;
    uint32_t u[N];
    // wide: the address is a multiple of 32 bytes; else element by element
    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < N; i += 8)
                asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3]), "=r"(u[i + 4]),
                               "=r"(u[i + 5]), "=r"(u[i + 6]), "=r"(u[i + 7])
                             : "l"(reinterpret_cast<const uint32_t*>(p) + i));
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = __float_as_uint(p[i]);
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = (uint32_t)q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = 0u;
    }
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
    // The bits of max|x| as fp32: ordered as unsigned numbers, infinities and NaN on top.
    __device__ __forceinline__ uint32_t amax_bits() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < N; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
            return m;
        } else {
            using P = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
            uint32_t a[N];
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = u[i] & 0x7FFF7FFFu;
#pragma unroll
            for (int s = N / 2; s > 0; s >>= 1)
#pragma unroll
                for (int i = 0; i < s; ++i) {
                    const P r = __hmax2_nan(*reinterpret_cast<const P*>(&a[i]), *reinterpret_cast<const P*>(&a[i + s]));
                    a[i] = *reinterpret_cast<const uint32_t*>(&r);
                }
            Block b;
            b.u[0] = a[0];
            return max(__float_as_uint(b.get(0)), __float_as_uint(b.get(1))) & 0x7FFFFFFFu;
        }
    }
};

// Row or tensor scale, with a power of two that brings it near one.
struct Scale {
    float g, up;  // g * up lies within 2^-85 and 2^64
    __device__ __forceinline__ explicit Scale(float g_) {
        up = g_ < 5.42101086e-20f ? 18446744073709551616.0f : g_ > 18446744073709551616.0f ? 5.42101086e-20f : 1.0f;  // 2^+-64
        g = g_ * up;
    }
};

// The code of a block's scale for its largest magnitude (a finite number).
__device__ __forceinline__ uint32_t block_scale(float amax, const Scale& sc) {
    if (!(sc.g > 0.0f)) return 0u;
    const float a = amax * sc.up;
    const float q = a * rcp_approx(6.0f * sc.g);  // within 8 units in the last place
    uint32_t b = __float_as_uint(q);
    if (((b + 8u) & 0x7FFFFu) <= 16u && q < 1e30f) {
        b = (b + 8u) & 0xFFF80000u;
        const float off = __fmaf_rn(-6.0f * __uint_as_float(b), sc.g, a);
        b = off > 0.0f ? b + 64u : off < 0.0f ? b - 64u : b;
    }
    return e4m3_code(__uint_as_float(b));
}

// Codes of a block of finite numbers, eight to a word.
template <typename T>
__device__ __forceinline__ uint2 block_codes(const Block<T>& x, uint32_t scale_code, const Scale& sc) {
    if (scale_code == 0u) return make_uint2(0u, 0u);
    const float s = e4m3_value(scale_code);
    const float inv = rcp_approx(s * sc.g);
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x.get(i) * inv;  // within 8 units in the last place
    if (sc.up != 1.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] *= sc.up;
    }
    uint32_t near = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 16; ++i) near = min(near, __float_as_uint(y[i]) * 2048u + (8u << 11));
    if (near <= (16u << 11)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t u = __float_as_uint(y[i]);
            if ((u * 2048u + (8u << 11)) <= (16u << 11)) {
                uint32_t b = ((u & 0x7FFFFFFFu) + 8u) & 0xFFE00000u;
                const float off = __fmaf_rn(-(__uint_as_float(b) * s), sc.g, fabsf(x.get(i)) * sc.up);
                b = off > 0.0f ? b + 64u : off < 0.0f ? b - 64u : b;
                // far above the largest border the product above may be infinite: the code is 6 all the same
                y[i] = fabsf(y[i]) < 16.0f ? __uint_as_float(b | (u & 0x80000000u)) : y[i];
            }
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float* p = y + 8 * h;
        const uint32_t c = e2m1x2(p[0], p[1]) | e2m1x2(p[2], p[3]) << 8 | e2m1x2(p[4], p[5]) << 16 | e2m1x2(p[6], p[7]) << 24;
        const uint32_t some = (c | c >> 1 | c >> 2) & 0x11111111u;  // a zero has no sign
        w[h] = c & (some << 3 | 0x77777777u);
    }
    return make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------------------

// Where a block's codes and scale go.
struct Place {
    uint8_t* codes;   // or the tiles
    uint8_t* scales;  // null: tiles
    int blocks;       // per row
    int tiles;        // per row of tiles
    __device__ __forceinline__ void put(int row, int k, uint2 c, uint32_t s) const {
        if (scales != nullptr) {
            const size_t at = (size_t)row * blocks + k;
            reinterpret_cast<uint2*>(codes)[at] = c;
            scales[at] = (uint8_t)s;
        } else {
            uint8_t* p = codes + ((size_t)(row >> 7) * tiles + (k >> 4)) * kTileBytes;
            *reinterpret_cast<uint2*>(p + tile_code_at(row & 127, k & 15)) = c;
            p[tile_scale_at(row & 127, k & 15)] = (uint8_t)s;
        }
    }
};

struct QuantArgs {
    const void* x;
    long long stride;
    int T;
    int blocks;        // of 16 elements per row
    int padded;        // blocks written per row
    int warps;         // per row
    float g;           // tensor scale, when row_scales is null
    float* row_scales;
    Place to;
};

constexpr int kMaxThreads = 1024;

// ITEMS blocks per thread in registers (0: a row is read twice).
template <typename T, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads) k_quantize(const QuantArgs a, bool wide) {
    __shared__ uint32_t s_max[32];
    rows_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_cta = warp / a.warps;                     // row of the CTA
    const int at = (warp - in_cta * a.warps) * 32 + lane;  // thread of the row
    const int step = a.warps * 32;
    const int row = blockIdx.x * ((int)(blockDim.x >> 5) / a.warps) + in_cta;
    const bool live = row < a.T;
    const T* x = static_cast<const T*>(a.x) + (size_t)(live ? row : 0) * a.stride;
    constexpr int HELD = ITEMS > 0 ? ITEMS : 1;
    Block<T> b[HELD];
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int k = at + i * step;
            if (live && k < a.blocks)
                b[i].load(x + (size_t)k * 16, wide);
            else
                b[i].zero();
        }
    }
    float g = a.g;
    bool bad_row = false;
    if (a.row_scales != nullptr) {
        uint32_t m = 0u;
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) m = max(m, b[i].amax_bits());
        } else {
            for (int k = at; live && k < a.blocks; k += step) {
                b[0].load(x + (size_t)k * 16, wide);
                m = max(m, b[0].amax_bits());
            }
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (a.warps > 1) {
            if (lane == 0) s_max[warp] = m;
            __syncthreads();
            m = __reduce_max_sync(0xFFFFFFFFu, lane < a.warps ? s_max[in_cta * a.warps + lane] : 0u);
        }
        bad_row = m >= 0x7F800000u;
        g = bad_row ? 0.0f : __fdiv_rn(__uint_as_float(m), kTop);
        if (live && at == 0) a.row_scales[row] = bad_row ? __uint_as_float(0x7FC00000u) : g;
    }
    if (!live) return;
    const Scale sc(g);
    auto one = [&](const Block<T>& x, int k) {
        const uint32_t m = x.amax_bits();
        uint32_t s = 0u;
        uint2 c = make_uint2(0u, 0u);
        if (m < 0x7F800000u) {
            s = block_scale(__uint_as_float(m), sc);
            c = block_codes(x, s, sc);
        } else if (!bad_row) {
            s = kNanScale;
        }
        a.to.put(row, k, c, s);
    };
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int k = at + i * step;
            if (k < a.padded) one(b[i], k);
        }
    } else {
        for (int k = at; k < a.padded; k += step) {
            if (k < a.blocks)
                b[0].load(x + (size_t)k * 16, wide);
            else
                b[0].zero();
            one(b[0], k);
        }
    }
}

// ---------------------------------------------------------------------------

struct DequantArgs {
    const uint8_t* codes;  // or the tiles
    const uint8_t* scales; // null: tiles
    int T, blocks, tiles;
    float g;
    const float* row_scales;  // null: g
    void* y;
    long long stride;
};

template <typename T>
__global__ void __launch_bounds__(256) k_dequantize(const DequantArgs a, bool wide) {
    rows_wait();
    const int k = blockIdx.y * 32 + (threadIdx.x & 31);
    if (k >= a.blocks) return;
    for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.T; row += (long long)gridDim.x * 8) {
        uint2 c;
        uint32_t s;
        if (a.scales != nullptr) {
            const size_t at = (size_t)row * a.blocks + k;
            c = reinterpret_cast<const uint2*>(a.codes)[at];
            s = a.scales[at];
        } else {
            const uint8_t* p = a.codes + ((size_t)(row >> 7) * a.tiles + (k >> 4)) * kTileBytes;
            c = *reinterpret_cast<const uint2*>(p + tile_code_at((int)row & 127, k & 15));
            s = p[tile_scale_at((int)row & 127, k & 15)];
        }
        const float g = a.row_scales != nullptr ? a.row_scales[row] : a.g;
        const __half2 sh = __float2half2_rn(e4m3_value(s));
        T* y = static_cast<T*>(a.y) + (size_t)row * a.stride + (size_t)k * 16;
        float v[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t f[4];
            e2m1_values(h ? c.y : c.x, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // code * scale has at most six bits: exact in f16
                const float2 q = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&f[i]), sh));
                v[8 * h + 2 * i] = q.x * g;
                v[8 * h + 2 * i + 1] = q.y * g;
            }
        }
        if (wide) {
            constexpr int VEC = kVecOf<T>;
#pragma unroll
            for (int i = 0; i < 16; i += VEC) {
                RawVec<T, VEC> r;
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) r.u[j] = __float_as_uint(v[i + j]);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) r.set2(j, v[i + 2 * j], v[i + 2 * j + 1]);
                }
                r.store(y + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = from_f32<T>(v[i]);
        }
    }
}

// Row-major 4-bit matrix to tiles: a thread has 32 elements (16 bytes of codes, two scales).
__global__ void __launch_bounds__(256) k_tile(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int V,
                                              int blocks, int tiles, uint8_t* __restrict__ out) {
    rows_wait();
    const int lane = threadIdx.x & 31;
    const int rows = (V + 127) / 128 * 128;
    const int k = (blockIdx.y * 32 + lane) * 2;
    if (k >= tiles * 16) return;
    for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += (long long)gridDim.x * 8) {
        uint2 c0 = make_uint2(0u, 0u), c1 = c0;
        uint32_t s0 = 0u, s1 = 0u;
        const size_t at = (size_t)row * blocks + k;
        if (row < V && k < blocks) {
            c0 = reinterpret_cast<const uint2*>(codes)[at];
            s0 = scales[at];
        }
        if (row < V && k + 1 < blocks) {
            c1 = reinterpret_cast<const uint2*>(codes)[at + 1];
            s1 = scales[at + 1];
        }
        uint8_t* p = out + ((size_t)(row >> 7) * tiles + (k >> 4)) * kTileBytes;
        *reinterpret_cast<uint4*>(p + tile_code_at((int)row & 127, k & 15)) = make_uint4(c0.x, c0.y, c1.x, c1.y);
        *reinterpret_cast<uint16_t*>(p + tile_scale_at((int)row & 127, k & 15)) = (uint16_t)(s0 | s1 << 8);
    }
}

// ---------------------------------------------------------------------------

template <typename K, typename... A>
static cudaError_t launch(K kernel, dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
static cudaError_t quantize(const Nvfp4QuantArgs& q, cudaStream_t s) {
    QuantArgs a{};
    a.x = q.x;
    a.stride = q.x_stride;
    a.T = q.T;
    a.blocks = q.H / 16;
    a.g = q.tensor_scale;
    a.row_scales = q.row_scales;
    a.to.codes = q.codes;
    a.to.scales = q.scales;
    a.to.blocks = a.blocks;
    a.to.tiles = tiles_per_row(q.H);
    a.padded = q.scales != nullptr ? a.blocks : a.to.tiles * 16;
    const bool wide = reinterpret_cast<uintptr_t>(q.x) % 32 == 0 && (q.T == 1 || q.x_stride * sizeof(T) % 32 == 0);
    constexpr int kHeld = sizeof(T) == 4 ? 2 : 4;  // blocks per thread of a wide launch: 32 registers
    const int items = a.padded <= kHeld * kMaxThreads ? kHeld : 0;
    const int per = items > 0 ? 32 * items : 32 * kHeld;
    a.warps = std::min((a.padded + per - 1) / per, kMaxThreads / 32);
    const int rows = std::max(1, 8 / a.warps);
    const dim3 grid((unsigned)((q.T + (long long)rows - 1) / rows));
    const int threads = rows * a.warps * 32;
    return items > 0 ? launch(k_quantize<T, kHeld>, grid, threads, s, a, wide) : launch(k_quantize<T, 0>, grid, threads, s, a, wide);
}

template <typename T>
static cudaError_t dequantize(const Nvfp4DequantArgs& q, cudaStream_t s) {
    DequantArgs a{};
    a.codes = q.codes;
    a.scales = q.scales;
    a.T = q.T;
    a.blocks = q.H / 16;
    a.tiles = tiles_per_row(q.H);
    a.g = q.tensor_scale;
    a.row_scales = q.row_scales;
    a.y = q.y;
    a.stride = q.y_stride;
    const bool wide = reinterpret_cast<uintptr_t>(q.y) % 16 == 0 && (q.T == 1 || q.y_stride * sizeof(T) % 16 == 0);
    const int across = (a.blocks + 31) / 32;
    const int down = (int)std::min<long long>(((long long)q.T + 7) / 8, std::max(1, 152 * 64 / across));
    return launch(k_dequantize<T>, dim3((unsigned)down, (unsigned)across), 256, s, a, wide);
}

}  // namespace q4

cudaError_t launch_nvfp4_quantize(const Nvfp4QuantArgs& a, int dtype, cudaStream_t s) {
    return dtype == VH_F32    ? q4::quantize<float>(a, s)
           : dtype == VH_BF16 ? q4::quantize<__nv_bfloat16>(a, s)
                              : q4::quantize<__half>(a, s);
}

cudaError_t launch_nvfp4_dequantize(const Nvfp4DequantArgs& a, int dtype, cudaStream_t s) {
    return dtype == VH_F32    ? q4::dequantize<float>(a, s)
           : dtype == VH_BF16 ? q4::dequantize<__nv_bfloat16>(a, s)
                              : q4::dequantize<__half>(a, s);
}

cudaError_t launch_nvfp4_tile(const uint8_t* codes, const uint8_t* scales, int V, int H, uint8_t* tiles, cudaStream_t s) {
    const int per_row = tiles_per_row(H), across = (per_row * 8 + 31) / 32;
    const int down = (int)std::min<long long>(((long long)V + 127) / 128 * 16, std::max(1, 152 * 64 / across));
    return q4::launch(q4::k_tile, dim3((unsigned)down, (unsigned)across), 256, s, codes, scales, V, H / 16, per_row, tiles);
}

}  // namespace vh
