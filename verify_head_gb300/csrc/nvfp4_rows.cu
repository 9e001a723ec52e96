// Rows to block-scaled 4 bits and back (the NVFP4 format of the 4-bit heads),
// and the tiled layout that the product of two 4-bit matrices reads.
//
//     g = given, or fp32(max|row| / (6 * 448)) for each row
//     s = e4m3(max|block| / (6 g)),  c = e2m1(x / (s g)),  both to the nearest, ties to even
//     value = c s g
//
// Codes are those of the exact quotient.  fp32 gives a quotient to a few units
// in the last place; only where that lies next to a border between two codes
// can it be on the wrong side.  So elements are converted twice, from products
// a little below and a little above the quotient: where both give one code it
// is the exact one's.  Else x is compared with the border exactly: border * s
// has at most seven bits, and fma(border * s, -g, |x|) rounds once, so its
// sign is that of the exact difference.  (In rows of 16-bit types whose
// largest element makes the scale, the quotients are ratios of small whole
// numbers and one in 250 lies at a border, so that most warps have one: a
// path that looked at all 16 elements again took 34 us for 16384 x 2048.)
// g is brought near one first, so that nothing of this underflows.
//
// A thread has blocks of 16 elements in registers (32 bytes of 16-bit types),
// so a row is read once, whatever finds its scale: a row's threads are one
// warp or several of a CTA.  16384 x 2048 bf16: 20.1 us to 4 bits (86 MB:
// 0.64 of the copy rate; no unit at its limit: 69% of the issue slots, 15
// instructions per element, with 40% of the warps that an SM holds) and 14.7
// us back (0.88), 15.4 from tiles.  Rows that lie off 32 bytes (a pitch of 2049)
// go element by element: 40 us, and 182 back.  Row-major to tiles: 248320 x
// 2048 in 106 us (572 MB: 0.81).
#include <algorithm>

#include "vh_nvfp4_tiles.h"
#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace q4 {

constexpr int kRowsPerThread = 4;  // of values, where there are enough

constexpr float kTop = 2688.0f;  // 6 * 448
constexpr uint32_t kNanScale = 0x7Fu;

// Codes of eight numbers, the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_codes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
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
                asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
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
            for (int i = 0; i < N; ++i) {
                const P r = __habs2(*reinterpret_cast<const P*>(&u[i]));
                a[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
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
    float g, up;   // g * up lies within 2^-85 and 2^64
    float sixth;   // 1 / (6 g)
    __device__ __forceinline__ explicit Scale(float g_) {
        up = g_ < 5.42101086e-20f ? 18446744073709551616.0f : g_ > 18446744073709551616.0f ? 5.42101086e-20f : 1.0f;  // 2^+-64
        g = g_ * up;
        sixth = rcp_approx(6.0f * g);
    }
};

// The code of a block's scale for its largest magnitude (a finite number).
__device__ __forceinline__ uint32_t block_scale(float amax, const Scale& sc) {
    if (!(sc.g > 0.0f)) return 0u;
    const float a = amax * sc.up;
    const float q = a * sc.sixth;  // within 8 units in the last place, 2^-20
    const uint32_t both = e4m3_codes(q * (1.0f - 0x1p-20f), q * (1.0f + 0x1p-20f));
    uint32_t lo = both & 0xFFu;
    const uint32_t hi = both >> 8;
    if (lo != hi) {  // neighbours, with the border between them
        const float off = __fmaf_rn(-3.0f * (e4m3_value(lo) + e4m3_value(hi)), sc.g, a);
        lo = off > 0.0f ? hi : off < 0.0f ? lo : (lo & 1u) ? hi : lo;
    }
    return lo;
}

__device__ __forceinline__ void mul2(float& a, float& b, float x, float y, float f) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(x), "f"(y), "f"(f));
}

// The code of a number whose magnitude lies between two neighbouring codes, or at the border between them.
__device__ __forceinline__ uint32_t between(uint32_t lo, uint32_t hi, float x, float s, const Scale& sc) {
    // twice the border: the sum of the two values
    const uint32_t pair = lo | hi << 4;
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(h) : "r"(pair));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const float off = __fmaf_rn(-(0.5f * (v.x + v.y) * s), sc.g, fabsf(x) * sc.up);
    return off > 0.0f ? hi : off < 0.0f ? lo : (lo & 1u) ? hi : lo;
}

// Codes of a block of finite numbers at p, eight to a word.
template <typename T>
__device__ __forceinline__ uint2 block_codes(const Block<T>& x, const T* p, uint32_t scale_code, const Scale& sc) {
    if (scale_code == 0u) return make_uint2(0u, 0u);
    const float s = e4m3_value(scale_code);
    const float inv = rcp_approx(s * sc.g);  // the quotient within 8 units in the last place, 2^-20
    const float below = inv * (1.0f - 0x1p-20f), above = inv * (1.0f + 0x1p-20f);
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            mul2(y[i], y[i + 1], x.get(8 * h + i), x.get(8 * h + i + 1), below);
            mul2(z[i], z[i + 1], x.get(8 * h + i), x.get(8 * h + i + 1), above);
        }
        if (sc.up != 1.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] *= sc.up;
                z[i] *= sc.up;
            }
        }
        lo[h] = e2m1x8(y);
        hi[h] = e2m1x8(z);
    }
    uint32_t differ[2] = {lo[0] ^ hi[0], lo[1] ^ hi[1]};
    while ((differ[0] | differ[1]) != 0u) {
        const bool second = differ[0] == 0u;
        const uint32_t d = second ? differ[1] : differ[0], l = second ? lo[1] : lo[0], h = second ? hi[1] : hi[0];
        const int at = (__ffs((int)d) - 1) & ~3;  // of the four bits
        const uint32_t c = between((l >> at) & 7u, (h >> at) & 7u, to_f32(p[(second ? 8 : 0) + (at >> 2)]), s, sc);
        const uint32_t word = (l & ~(7u << at)) | c << at, rest = d & ~(15u << at);
        lo[0] = second ? lo[0] : word;
        lo[1] = second ? word : lo[1];
        differ[0] = second ? 0u : rest;
        differ[1] = second ? rest : differ[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t some = (lo[h] | lo[h] >> 1 | lo[h] >> 2) & 0x11111111u;  // a zero has no sign
        lo[h] &= some << 3 | 0x77777777u;
    }
    return make_uint2(lo[0], lo[1]);
}

// ---------------------------------------------------------------------------

// Where a row's codes and scales go.  A thread's blocks are whole warps apart, so in the tiled layout its place within a record
// is the same for all of them.
struct Place {
    uint8_t* codes;   // or the tiles
    uint8_t* scales;  // null: tiles
    int blocks;       // per row
    int tiles;        // per row of tiles
};
struct RowPlace {
    uint8_t *codes, *scales;  // of the thread's first block
    int code_step, scale_step;  // bytes per 32 blocks
    __device__ __forceinline__ RowPlace(const Place& p, int row, int k) {
        if (p.scales != nullptr) {
            const size_t at = (size_t)row * p.blocks + k;
            codes = p.codes + at * 8;
            scales = p.scales + at;
            code_step = 256;
            scale_step = 32;
        } else {
            uint8_t* t = p.codes + ((size_t)(row >> 7) * p.tiles + (k >> 4)) * kTileBytes;
            codes = t + tile_code_at(row & 127, k & 15);
            scales = t + tile_scale_at(row & 127, k & 15);
            code_step = scale_step = 2 * kTileBytes;
        }
    }
    // the block 32 n places on
    __device__ __forceinline__ void put(int n, uint2 c, uint32_t s) const {
        *reinterpret_cast<uint2*>(codes + (long long)n * code_step) = c;
        scales[(long long)n * scale_step] = (uint8_t)s;
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
template <typename T, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS) k_quantize(const QuantArgs a, bool wide) {
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
    const RowPlace to(a.to, row, at);
    auto one = [&](const Block<T>& v, int k, int n) {
        const uint32_t m = v.amax_bits();
        uint32_t s = 0u;
        uint2 c = make_uint2(0u, 0u);
        if (m < 0x7F800000u) {
            s = block_scale(__uint_as_float(m), sc);
            c = block_codes(v, x + (size_t)k * 16, s, sc);
        } else if (!bad_row) {
            s = kNanScale;
        }
        to.put(n, c, s);
    };
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int k = at + i * step;
            if (k < a.padded) one(b[i], k, i * a.warps);
        }
    } else {
        for (int k = at, n = 0; k < a.padded; k += step, n += a.warps) {
            if (k < a.blocks)
                b[0].load(x + (size_t)k * 16, wide);
            else
                b[0].zero();
            one(b[0], k, n);
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
__device__ __forceinline__ void dequantize_block(uint2 c, uint32_t scale, float g, T* y, bool wide) {
    const __half2 sh = __float2half2_rn(e4m3_value(scale));
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t f[4];
        e2m1_values(h ? c.y : c.x, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // code * scale has at most six bits: exact in f16
            const float2 q = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&f[i]), sh));
            mul2(v[8 * h + 2 * i], v[8 * h + 2 * i + 1], q.x, q.y, g);
        }
    }
    if (wide) {  // 32 bytes at a time
        constexpr int E = 32 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < 16; i += E) {
            RawVec<T, E> r;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (sizeof(T) == 4)
                    r.u[j] = __float_as_uint(v[i + j]);
                else
                    r.set2(j, v[i + 2 * j], v[i + 2 * j + 1]);
            }
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(y + i), "r"(r.u[0]), "r"(r.u[1]), "r"(r.u[2]),
                         "r"(r.u[3]), "r"(r.u[4]), "r"(r.u[5]), "r"(r.u[6]), "r"(r.u[7])
                         : "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = from_f32<T>(v[i]);
    }
}

// A thread has block k of the rows row, row + step, ..., two of them in flight.
template <typename T, bool TILES>
__global__ void __launch_bounds__(256) k_dequantize(const DequantArgs a, bool wide) {
    rows_wait();
    const int k = blockIdx.y * 32 + (threadIdx.x & 31);
    if (k >= a.blocks) return;
    const long long step = (long long)gridDim.x * 8;
    long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    auto codes_of = [&](long long r) {
        if constexpr (TILES)
            return a.codes + ((size_t)(r >> 7) * a.tiles + (k >> 4)) * kTileBytes + tile_code_at((int)r & 127, k & 15);
        else
            return a.codes + ((size_t)r * a.blocks + k) * 8;
    };
    auto scale_of = [&](long long r) {
        if constexpr (TILES)
            return a.codes + ((size_t)(r >> 7) * a.tiles + (k >> 4)) * kTileBytes + tile_scale_at((int)r & 127, k & 15);
        else
            return a.scales + (size_t)r * a.blocks + k;
    };
    const uint8_t *cp = codes_of(row), *sp = scale_of(row);
    const long long cs = step * a.blocks * 8, ss = step * a.blocks;
    T* y = static_cast<T*>(a.y) + row * a.stride + (size_t)k * 16;
    const long long ys = step * a.stride;
    auto fetch = [&](uint2& c, uint32_t& s, float& g) {
        if (row >= a.T) return;
        if constexpr (TILES) {
            cp = codes_of(row);
            sp = scale_of(row);
        }
        c = __ldcg(reinterpret_cast<const uint2*>(cp));
        s = __ldcg(sp);
        g = a.row_scales != nullptr ? a.row_scales[row] : a.g;
        cp += cs;
        sp += ss;
        row += step;
    };
    uint2 c0, c1;
    uint32_t s0, s1;
    float g0, g1;
    long long left = row < a.T ? (a.T - 1 - row) / step + 1 : 0;
    fetch(c0, s0, g0);
    fetch(c1, s1, g1);
    while (left > 0) {
        dequantize_block(c0, s0, g0, y, wide);
        fetch(c0, s0, g0);
        y += ys;
        if (--left == 0) break;
        dequantize_block(c1, s1, g1, y, wide);
        fetch(c1, s1, g1);
        y += ys;
        --left;
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
    // Blocks per thread: four where that leaves a few waves of warps (16384 x 2048 bf16 21.2 us, 22.6 with two), else two (256 x
    // 8192 3.1 us, 3.8 with four).
    constexpr int kMany = sizeof(T) == 4 ? 2 : 4, kHeld = 2;
    auto go = [&](auto kernel, int items, int most) {
        const int per = 32 * std::max(items, 1);
        a.warps = std::min((a.padded + per - 1) / per, most / 32);
        const int rows = std::max(1, 8 / a.warps);
        return launch(kernel, dim3((unsigned)((q.T + (long long)rows - 1) / rows)), rows * a.warps * 32, s, a, wide);
    };
    if (a.padded <= kMany * 256 && (long long)q.T * a.padded >= 152ll * 32 * 32 * kMany) return go(k_quantize<T, kMany, 256>, kMany, 256);
    if (a.padded <= kHeld * 256) return go(k_quantize<T, kHeld, 256>, kHeld, 256);
    if (a.padded <= kHeld * kMaxThreads) return go(k_quantize<T, kHeld, kMaxThreads>, kHeld, kMaxThreads);
    return go(k_quantize<T, 0, kMaxThreads>, 0, kMaxThreads);
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
    const bool wide = reinterpret_cast<uintptr_t>(q.y) % 32 == 0 && (q.T == 1 || q.y_stride * sizeof(T) % 32 == 0);
    const int across = (a.blocks + 31) / 32;
    // some rows a thread where that leaves a few waves of CTAs
    const int down = (int)std::min<long long>(((long long)q.T + 7) / 8, std::max<long long>(((long long)q.T + 8 * kRowsPerThread - 1) / (8 * kRowsPerThread), 152 * 8 / across));
    const dim3 grid((unsigned)down, (unsigned)across);
    return q.scales != nullptr ? launch(k_dequantize<T, false>, grid, 256, s, a, wide) : launch(k_dequantize<T, true>, grid, 256, s, a, wide);
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
