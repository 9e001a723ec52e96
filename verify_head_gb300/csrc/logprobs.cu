// Log probabilities of given tokens from logits, with the entropy of each row
// and its largest alternatives, and the gradient.
//
//     lse = log sum_v e^x_v      logprob = x_token - lse      entropy = lse - sum_v p_v x_v
//     dx_v = g_lp ([v = token] - p_v) - g_ent p_v (log p_v + entropy)
//
// Forward: one pass over the logits.  A row is cut into slots of 16 aligned
// bytes and segments of 32 slots (one warp load).  Each thread keeps a running
// maximum and the two sums of Stat; where alternatives are wanted the warp
// also writes each segment's maximum, and the row's last CTA picks the
// alternatives from the segments with the largest maxima (select_top), reading
// about n segments of 512 bytes again.
//
// A row is split over several CTAs when there are few rows; their statistics
// meet in the workspace and the last CTA of a row (a ticket per row, left
// zero again) finishes it.
//
// Bound: memory (the logits once; the gradient also writes them once).
#include <algorithm>

#include "vh_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace lp {

constexpr int kThreadsL = kSelThreads;
constexpr int kWarpsL = kThreadsL / 32;
constexpr int kUnroll = 4;            // segments in flight per warp
constexpr int kTargetCtas = 608;      // CTAs wanted on the GPU at once (four per SM)
constexpr int kMinSegs = 2 * kWarpsL;  // segments per CTA below which a row is not cut further

// A row as aligned 16-byte slots: slot v holds elements [v * VEC - shift, +VEC).
template <typename T>
struct Row {
    const uint8_t* base;  // row address rounded down to 16 bytes
    int shift;            // elements before the row's first one in slot 0
    int V;
    __device__ __forceinline__ Row(const T* p, int V_) : V(V_) {
        const uintptr_t u = reinterpret_cast<uintptr_t>(p);
        base = reinterpret_cast<const uint8_t*>(u & ~uintptr_t(15));
        shift = (int)((u & 15) / sizeof(T));
    }
    __device__ __forceinline__ int slots() const { return (int)(((long long)V + shift + kVecOf<T> - 1) / kVecOf<T>); }
    __device__ __forceinline__ long long first(int slot) const { return (long long)slot * kVecOf<T> - shift; }
    // Elements of a slot; places outside the row (and whole slots past the end) read as -inf.
    __device__ __forceinline__ void load(int slot, float (&f)[kVecOf<T>]) const {
        constexpr int VEC = kVecOf<T>;
        const long long e0 = first(slot);
        if (e0 >= 0 && e0 + VEC <= V) {
            RawVec<T, VEC> r;
            r.load(reinterpret_cast<const T*>(base + (size_t)slot * 16));
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = r.get(i);
        } else {
            const T* p = reinterpret_cast<const T*>(base) + (long long)slot * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = (e0 + i >= 0 && e0 + i < V) ? to_f32(p[i]) : neg_inf();
        }
    }
};

// A row's segments for select_top.
template <typename T>
struct Segments {
    struct Item {
        float f[kVecOf<T>];
    };
    const Row<T>& x;
    const float* maxima;
    __device__ __forceinline__ float max(int g) const { return __ldcg(maxima + g); }
    __device__ __forceinline__ Item load(int g) const {
        Item it;
        x.load(g * 32 + (threadIdx.x & 31), it.f);
        return it;
    }
    template <typename F>
    __device__ __forceinline__ void each(const Item& it, int g, F take) const {
        const long long e0 = x.first(g * 32 + (threadIdx.x & 31));
#pragma unroll
        for (int j = 0; j < kVecOf<T>; ++j)
            take(e0 + j >= 0 && e0 + j < x.V ? make_key(it.f[j], (uint32_t)(e0 + j)) : 0ull);
    }
};

// Upper bound of the segments of a row of V elements of `size` bytes, whatever its alignment.
__host__ __device__ inline int max_segs(int V, int size) {
    const long long per = 512 / size;
    return (int)(((long long)V + 16 / size - 1 + per - 1) / per);
}

struct Ws {
    unsigned int* ticket;  // [kTargetCtas]: rows that are split
    float4* part;          // [R][splits]: c, s, t
    float* seg_max;        // [R][segs]
};
struct Plan {
    int segs, splits;
};
inline Plan plan(int R, int V, int size) {
    Plan p;
    p.segs = max_segs(V, size);
    const int by_rows = std::max(1, (kTargetCtas + R - 1) / R);
    p.splits = std::max(1, std::min(by_rows, p.segs / kMinSegs));
    return p;
}
// Only calls of fewer than kTargetCtas rows split rows, so the tickets take a fixed place and a
// workspace serves calls of any size up to its own.
constexpr size_t kTicketEnd = kWsHeaderBytes + (size_t)kTargetCtas * 4;

template <typename T>
__global__ void __launch_bounds__(kThreadsL, 4) k_logprobs(const LogprobArgs a, const Ws ws, const Plan pl) {
    constexpr int VEC = kVecOf<T>;
    __shared__ float4 s_part[kWarpsL];
    __shared__ SelectSmem s_sel;
    __shared__ RowStat s_rs;
    __shared__ int s_last;
    rows_launch_dependents();
    rows_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.y;
    const Row<T> x(static_cast<const T*>(a.logits) + (long long)row * a.stride, a.V);
    const int segs = (x.slots() + 31) / 32;
    const int g0 = (int)((long long)segs * blockIdx.x / gridDim.x), g1 = (int)((long long)segs * (blockIdx.x + 1) / gridDim.x);
    float* seg_max = ws.seg_max + (size_t)row * pl.segs;

    // Segments [in0, in1) hold whole slots only.
    const int in0 = x.shift != 0 ? 1 : 0;
    const int in1 = (int)(((long long)a.V + x.shift) / (32 * VEC));
    Stat2 run;
    run.clear();
    auto add = [&](const RawVec<T, VEC>& r) {
        const F2 mc = f2(-run.c, -run.c);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) run.add(r.get(i), r.get(i + 1), mc);
    };
    auto keep_max = [&](int g, float m) {
        if (a.top_n > 0) {
            float w;
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(w) : "f"(m));
            if (lane == 0) seg_max[g] = w;
        }
    };
    for (int g = g0 + warp; g < g1; g += kWarpsL * kUnroll) {
        const int last = g + (kUnroll - 1) * kWarpsL;
        if (g >= in0 && last < min(g1, in1)) {
            RawVec<T, VEC> r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                r[u].load(reinterpret_cast<const T*>(x.base + ((size_t)(g + u * kWarpsL) * 32 + lane) * 16));
            float m = neg_inf();
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const float mu = r[u].max();
                m = fmaxf(m, mu);
                keep_max(g + u * kWarpsL, mu);
            }
            run.raise(m);
            if (run.c != neg_inf()) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) add(r[u]);
            }
        } else {  // a row's ends
            for (int gg = g; gg < g1 && gg <= last; gg += kWarpsL) {
                float f[VEC];
                x.load(gg * 32 + lane, f);
                float m = neg_inf();
#pragma unroll
                for (int i = 0; i < VEC; ++i) m = fmaxf(m, f[i]);
                keep_max(gg, m);
                run.raise(m);
                if (run.c != neg_inf()) {
                    const F2 mc = f2(-run.c, -run.c);
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) run.add(f[i], f[i + 1], mc);
                }
            }
        }
    }
    Stat st = run.get();
    st = stat_warp(st);
    if (lane == 0) s_part[warp] = make_float4(st.c, st.s, st.t, 0.f);
    __syncthreads();
    if (warp == 0) {
        st = stat_none();
        if (lane < kWarpsL) st = Stat{s_part[lane].x, s_part[lane].y, s_part[lane].z};
        st = stat_warp(st);
    }
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) ws.part[(size_t)row * pl.splits + blockIdx.x] = make_float4(st.c, st.s, st.t, 0.f);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(ws.ticket + row, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        if (threadIdx.x == 0) atomicExch(ws.ticket + row, 0u);
        if (warp == 0) {
            st = stat_none();
            for (int i = lane; i < (int)gridDim.x; i += 32) {
                const float4 p = __ldcg(ws.part + (size_t)row * pl.splits + i);
                st = stat_join(st, Stat{p.x, p.y, p.z});
            }
            st = stat_warp(st);
        }
    }
    RowStat rs{};
    if (warp == 0) {
        rs = stat_finish(st);
        if (lane == 0) {
            if (a.logprob != nullptr) {
                const int tok = a.tokens != nullptr ? a.tokens[row] : -1;
                const T* p = static_cast<const T*>(a.logits) + (long long)row * a.stride;
                a.logprob[row] = (tok >= 0 && tok < a.V) ? stat_logprob(rs, to_f32(p[tok])) : 0.f;
            }
            if (a.entropy != nullptr) a.entropy[row] = rs.entropy;
            if (a.lse != nullptr) a.lse[row] = rs.lse;
        }
    }
    if (a.top_n == 0) return;
    if (threadIdx.x == 0) s_rs = rs;  // select_top has barriers before it emits
    select_top(
        s_sel, segs, a.top_n, 0u, Segments<T>{x, seg_max}, [] {},
        [&](int i, unsigned long long k) {
            const size_t o = (size_t)row * a.top_n + i;
            a.top_ids[o] = k != 0ull ? (int32_t)key_gid(k) : -1;
            a.top_logprobs[o] = k != 0ull ? stat_logprob(s_rs, key_score(k)) : neg_inf();
        });
}

// ---------------------------------------------------------------------------
// Gradient: every thread takes kGradUnroll vectors of its row.

constexpr int kGradUnroll = 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreadsL) k_logprobs_grad(const LogprobGradArgs a, int chunks) {
    rows_launch_dependents();
    rows_wait();
    const int row = (int)(blockIdx.x / chunks);
    const int chunk = (int)(blockIdx.x % chunks);
    const T* x = static_cast<const T*>(a.logits) + (long long)row * a.stride;
    T* d = static_cast<T*>(a.dlogits) + (long long)row * a.d_stride;
    const long long nvec = a.V / VEC;
    const float lse = a.lse[row];
    const int tok = a.tokens != nullptr ? a.tokens[row] : -1;
    const bool given = tok >= 0 && tok < a.V;
    float gl = (given && a.g_logprob != nullptr) ? a.g_logprob[row] : 0.f;
    float ge = a.g_entropy != nullptr ? a.g_entropy[row] : 0.f;
    const float ent = a.g_entropy != nullptr ? a.entropy[row] : 0.f;
    const bool empty = lse == neg_inf();
    // dx = p (k0 - ge2 y) with y = log2 p: -g_lp p - g_ent p (ln2 y + entropy)
    const float k0 = empty ? 0.f : (lse != lse ? quiet_nan() : -gl - ge * ent);
    const float ge2 = empty ? 0.f : ge * kLn2;
    if (empty) gl = 0.f;
    const long long v0 = (long long)chunk * kThreadsL * kGradUnroll + threadIdx.x;
    RawVec<T, VEC> r[kGradUnroll];
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
        const long long v = v0 + u * kThreadsL;
        if (v < nvec) r[u].load(x + v * VEC);
    }
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
        const long long v = v0 + u * kThreadsL;
        if (v < nvec) {
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float y = fmaxf((r[u].get(i) - lse) * kLog2e, kFloorY);
                const float p = empty ? 0.f : ex2(y);
                f[i] = p * fmaf(-ge2, y, k0);
            }
            const long long at = (long long)tok - v * VEC;
            if (given && at >= 0 && at < VEC) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] += i == at ? gl : 0.f;
            }
            RawVec<T, VEC> o;
            pack_vec<T, VEC>(o, f);
            o.store(d + v * VEC);
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
    const Plan pl = plan(a.R, a.V, (int)sizeof(T));
    Ws ws;
    uint8_t* p = static_cast<uint8_t*>(a.ws);
    ws.ticket = reinterpret_cast<unsigned int*>(p + kWsHeaderBytes);
    ws.part = reinterpret_cast<float4*>(p + kTicketEnd);
    ws.seg_max = reinterpret_cast<float*>(ws.part + (size_t)a.R * pl.splits);
    for (int r0 = 0; r0 < a.R; r0 += 65535) {  // the grid's second dimension holds 65,535 rows
        LogprobArgs b = a;
        Ws w = ws;
        const int nr = std::min(65535, a.R - r0);
        b.logits = static_cast<const T*>(a.logits) + (long long)r0 * a.stride;
        b.tokens = a.tokens ? a.tokens + r0 : nullptr;
        b.logprob = a.logprob ? a.logprob + r0 : nullptr;
        b.entropy = a.entropy ? a.entropy + r0 : nullptr;
        b.lse = a.lse ? a.lse + r0 : nullptr;
        if (a.top_n > 0) {
            b.top_ids += (size_t)r0 * a.top_n;
            b.top_logprobs += (size_t)r0 * a.top_n;
        }
        w.part += (size_t)r0 * pl.splits;
        w.seg_max += (size_t)r0 * pl.segs;
        cudaError_t e = launch(k_logprobs<T>, dim3((unsigned)pl.splits, (unsigned)nr), dim3(kThreadsL), s, b, w, pl);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int VEC>
static cudaError_t grad_vec(const LogprobGradArgs& a, cudaStream_t s) {
    const long long per = (long long)kThreadsL * kGradUnroll * VEC;
    const long long chunks = (a.V + per - 1) / per;
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
    const bool vec = a.V % V == 0 && a.stride % V == 0 && a.d_stride % V == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) & 15) == 0;
    return vec ? grad_vec<T, V>(a, s) : grad_vec<T, 1>(a, s);
}

}  // namespace lp

size_t logits_logprobs_ws_bytes(int R, int V, int top_n) {
    const lp::Plan p = lp::plan(R, V, 4);  // 32-bit logits have the most segments
    const lp::Plan q = lp::plan(R, V, 2);
    const size_t part = (size_t)R * std::max(p.splits, q.splits) * 16;
    return lp::kTicketEnd + part + (top_n > 0 ? round16((size_t)R * p.segs * 4) : 0);
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
