// Processing of logits before a token is picked, and its gradient.
//
//     z = x + bias;  seen: z = z > 0 ? z / rep : z rep;  z -= freq m + pres [m > 0];  out = z / temp, or -inf
//     dx = dout / temp, seen: / rep (z > 0) or * rep, or 0
//
// Almost every token of the vocabulary is neither biased nor in the history:
// its place is one product with 1 / temperature (two units in the last place
// of fp32 at most, instead of a division's half).  So a CTA takes the rows of
// one sequence over a chunk of the vocabulary, counts the history's tokens of
// its chunk in shared memory once for all of the sequence's rows (whole
// numbers: the order of the atomics does not matter), and marks them, with
// the biased and drafted ones, in a bitmap.  Then the rows stream through by
// slots of 16 aligned bytes: a slot without a marked place is converted and
// scaled, one with no allowed place is not read at all, and marked places are
// done one by one, where the drafts before the row are counted too.
//
// Every CTA reads the whole history, so the chunk grows with its length.
// Bound: memory (the logits once in and once out).
#include <algorithm>

#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace proc {

constexpr int kThreadsP = 256;
constexpr uint32_t kInPrompt = 0x80000000u;
constexpr int kMaxChunk = 32768;  // places of a chunk (a multiple of 128) at most
constexpr int kGroupRows = 8;  // rows of a sequence per CTA

struct Args {
    const void *in, *logits;
    void* out;
    long long in_stride, logits_stride, out_stride;
    int V, per_seq, chunk;
    int chunks, groups;  // of the vocabulary, and of a sequence's rows
    vh_logits_rules r;
};

// Shared memory of a chunk: counts, marks, the last bias entry of each place.
struct Chunk {
    uint32_t* count;   // [chunk]: occurrences in output, kInPrompt
    uint32_t* marked;  // [chunk / 32], and a word that bits_at reads past them
    uint16_t* entry;   // [chunk]: bias entry + 1 (null: no biases)
    __device__ __forceinline__ void mark(int at) const { atomicOr(marked + (at >> 5), 1u << (at & 31)); }
};
__host__ __device__ constexpr size_t smem_bytes(int chunk, bool biased) {
    return (size_t)chunk * (biased ? 6 : 4) + (size_t)(chunk / 32 + 4) * 4;  // a multiple of 16
}

// n <= 32 bits of a bitmap from bit `at` on, of which words beyond `last` are not read.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, long long at, int n, long long last) {
    const long long w = at >> 5;
    const uint32_t lo = words[w], hi = w < last ? words[w + 1] : 0u;
    const uint32_t b = __funnelshift_r(lo, hi, (uint32_t)at & 31u);
    return n < 32 ? b & ((1u << n) - 1u) : b;
}

// What one sequence's rows share.
struct Rules {
    float rep, freq, pres, inv_temp;
    const float* bias;
    const int32_t* draft;
};

// The rules at a marked place; `z` the logit, `v` the value that is changed (the logit itself, or the gradient).
template <bool GRAD>
__device__ __forceinline__ float apply(const Rules& u, const Chunk& c, int at, int token, int j0, int j, float z, float g) {
    if (c.entry != nullptr) {
        const uint32_t e = c.entry[at];
        if (e != 0u) z += u.bias[e - 1];
    }
    const uint32_t count = c.count[at];
    uint32_t n = count & ~kInPrompt;
    if (u.draft != nullptr)
        for (int i = j0; i < j; ++i) n += u.draft[i] == token;
    const bool seen = n > 0u || (count & kInPrompt) != 0u;
    if constexpr (GRAD) {
        if (seen) g = z > 0.0f ? __fdiv_rn(g, u.rep) : g * u.rep;
        return g * u.inv_temp;
    } else {
        if (seen) z = z > 0.0f ? __fdiv_rn(z, u.rep) : z * u.rep;
        if (n > 0u) z = __fsub_rn(__fsub_rn(z, __fmul_rn(u.freq, (float)n)), u.pres);
        return z * u.inv_temp;
    }
}

template <typename T, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThreadsP) k_process(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    constexpr int VEC = kVecOf<T>;
    constexpr int UNROLL = 4;
    rows_wait();
    const unsigned int part = blockIdx.x / a.chunks;
    const int seq = part / a.groups;
    const int j0 = (int)(part % a.groups) * kGroupRows, j1 = min(j0 + kGroupRows, a.per_seq);
    const long long c0 = (long long)(blockIdx.x % a.chunks) * a.chunk;
    const int n = (int)min((long long)a.chunk, a.V - c0);
    Chunk c;
    c.count = s_words;
    c.marked = s_words + a.chunk;
    c.entry = a.r.bias_ids != nullptr ? reinterpret_cast<uint16_t*>(c.marked + a.chunk / 32 + 4) : nullptr;
    const int tid = threadIdx.x;

    for (int i = tid; i < (int)(smem_bytes(a.chunk, c.entry != nullptr) / 16); i += kThreadsP)
        reinterpret_cast<uint4*>(s_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    if (a.r.history != nullptr) {
        const int32_t* h = a.r.history + (size_t)seq * a.r.history_stride;
        const int len = a.r.history_len != nullptr ? min(a.r.history_len[seq], a.r.history_width) : a.r.history_width;
        const int prompt = a.r.prompt_len != nullptr ? a.r.prompt_len[seq] : 0;
#pragma unroll 4
        for (int i = tid; i < len; i += kThreadsP) {
            const long long at = (long long)h[i] - c0;
            if (at >= 0 && at < n) {
                if (i < prompt)
                    atomicOr(c.count + at, kInPrompt);
                else
                    atomicAdd(c.count + at, 1u);
                c.mark((int)at);
            }
        }
    }
    Rules u;
    u.rep = a.r.repetition != nullptr ? a.r.repetition[seq] : 1.0f;
    u.freq = a.r.frequency != nullptr ? a.r.frequency[seq] : 0.0f;
    u.pres = a.r.presence != nullptr ? a.r.presence[seq] : 0.0f;
    const float temp = a.r.temperature != nullptr ? a.r.temperature[seq] : 1.0f;
    u.inv_temp = temp > 0.0f ? __fdiv_rn(1.0f, temp) : 1.0f;
    u.bias = nullptr;
    u.draft = a.r.draft_ids != nullptr && a.per_seq > 1 ? a.r.draft_ids + (size_t)seq * (a.per_seq - 1) : nullptr;
    if (u.draft != nullptr)
        for (int i = tid; i < j1 - 1; i += kThreadsP) {
            const long long at = (long long)u.draft[i] - c0;
            if (at >= 0 && at < n) {
                if (i < j0) atomicAdd(c.count + at, 1u);  // before all of the CTA's rows
                c.mark((int)at);
            }
        }
    if (c.entry != nullptr) {
        u.bias = a.r.bias + (size_t)seq * a.r.n_bias;
        const int32_t* ids = a.r.bias_ids + (size_t)seq * a.r.n_bias;
        for (int i = tid; i < a.r.n_bias; i += kThreadsP) {
            const long long at = (long long)ids[i] - c0;
            if (at >= 0 && at < n) {
                // the last entry of an id: the larger of the two halves of a word, by whole words
                uint32_t* w = reinterpret_cast<uint32_t*>(c.entry) + (at >> 1);
                const int sh = (int)(at & 1) * 16;
                uint32_t old = *w;
                while (((old >> sh) & 0xFFFFu) < (uint32_t)(i + 1)) {
                    const uint32_t was = atomicCAS(w, old, (old & ~(0xFFFFu << sh)) | (uint32_t)(i + 1) << sh);
                    if (was == old) break;
                    old = was;
                }
                c.mark((int)at);
            }
        }
    }
    __syncthreads();

    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    for (int j = j0; j < j1; ++j) {
        const long long row = (long long)seq * a.per_seq + j;
        const T* x = static_cast<const T*>(a.in) + row * a.in_stride;
        const T* lg = static_cast<const T*>(a.logits) + row * a.logits_stride;
        TO* y = static_cast<TO*>(a.out) + row * a.out_stride;
        const uint32_t* ok = a.r.allowed != nullptr ? reinterpret_cast<const uint32_t*>(a.r.allowed) + row * a.r.allowed_stride : nullptr;
        // slot i: elements [i * VEC - shift, +VEC) of the chunk
        const int shift = (int)((reinterpret_cast<uintptr_t>(x + c0) & 15) / sizeof(T));
        const int slots = (n + shift + VEC - 1) / VEC;
        const bool vec_out = (reinterpret_cast<uintptr_t>(y + c0 - shift) & 15) == 0;
        for (int base = 0; base < slots; base += kThreadsP * UNROLL) {
            RawVec<T, VEC> in[UNROLL];
            uint32_t allow[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int slot = base + k * kThreadsP + tid;
                const int e0 = slot * VEC - shift;
                allow[k] = (1u << VEC) - 1u;
                if (slot >= slots) continue;
                if (e0 >= 0 && e0 + VEC <= n) {
                    if (ok != nullptr) allow[k] = bits_at(ok, c0 + e0, VEC, last_word);
                    if (allow[k] != 0u) in[k].load(x + c0 + e0);
                }
            }
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int slot = base + k * kThreadsP + tid;
                const int e0 = slot * VEC - shift;
                if (slot >= slots) break;
                if (e0 >= 0 && e0 + VEC <= n) {
                    uint32_t m = bits_at(c.marked, e0, VEC, a.chunk / 32) & allow[k];
                    float v[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = (allow[k] >> i) & 1u ? in[k].get(i) * u.inv_temp : GRAD ? 0.0f : neg_inf();
                    if (m != 0u) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            if ((m >> i) & 1u) {
                                const float z = GRAD ? to_f32(lg[c0 + e0 + i]) : in[k].get(i);
                                v[i] = apply<GRAD>(u, c, e0 + i, (int)(c0 + e0 + i), j0, j, z, in[k].get(i));
                            }
                    }
                    TO* p = y + c0 + e0;
                    if (vec_out) {
                        constexpr int VO = kVecOf<TO>;
#pragma unroll
                        for (int i = 0; i < VEC; i += VO) {
                            RawVec<TO, VO> o;
                            if constexpr (sizeof(TO) == 4) {
#pragma unroll
                                for (int q = 0; q < VO; ++q) o.u[q] = __float_as_uint(v[i + q]);
                            } else {
#pragma unroll
                                for (int q = 0; q < VO / 2; ++q) o.set2(q, v[i + 2 * q], v[i + 2 * q + 1]);
                            }
                            o.store(p + i);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) p[i] = from_f32<TO>(v[i]);
                    }
                } else {  // a slot that the chunk has a part of
                    for (int i = 0; i < VEC; ++i) {
                        const int e = e0 + i;
                        if (e < 0 || e >= n) continue;
                        float v = GRAD ? 0.0f : neg_inf();
                        if (ok == nullptr || ((ok[(c0 + e) >> 5] >> ((c0 + e) & 31)) & 1u) != 0u) {
                            const float xv = to_f32(x[c0 + e]);
                            v = ((c.marked[e >> 5] >> (e & 31)) & 1u) != 0u
                                    ? apply<GRAD>(u, c, e, (int)(c0 + e), j0, j, GRAD ? to_f32(lg[c0 + e]) : xv, xv)
                                    : xv * u.inv_temp;
                        }
                        y[c0 + e] = from_f32<TO>(v);
                    }
                }
            }
        }
    }
}

template <typename T, typename TO, bool GRAD>
static cudaError_t run(const ProcessArgs& p, cudaStream_t s) {
    Args a{};
    a.in = p.in;
    a.logits = p.logits;
    a.out = p.out;
    a.in_stride = p.in_stride;
    a.logits_stride = p.logits_stride;
    a.out_stride = p.out_stride;
    a.V = p.V;
    a.per_seq = p.per_seq;
    a.r = p.rules;
    if (a.r.n_bias == 0) a.r.bias_ids = nullptr;
    if (a.r.history_width == 0) a.r.history = nullptr;
    const int S = p.R / p.per_seq;
    a.chunk = 8192;
    a.chunks = (int)(((long long)p.V + a.chunk - 1) / a.chunk);
    a.groups = (p.per_seq + kGroupRows - 1) / kGroupRows;
    const long long ctas = (long long)S * a.groups * a.chunks;
    if (ctas > 2147483647ll) return cudaErrorInvalidValue;
    auto kernel = k_process<T, TO, GRAD>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kMaxChunk, true));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = smem_bytes(a.chunk, a.r.bias_ids != nullptr);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace proc

cudaError_t launch_logits_process(const ProcessArgs& a, int dtype, int out_dtype, cudaStream_t s) {
    if (dtype == VH_F32) return proc::run<float, float, false>(a, s);
    if (dtype == VH_BF16)
        return out_dtype == VH_F32 ? proc::run<__nv_bfloat16, float, false>(a, s)
                                   : proc::run<__nv_bfloat16, __nv_bfloat16, false>(a, s);
    return out_dtype == VH_F32 ? proc::run<__half, float, false>(a, s) : proc::run<__half, __half, false>(a, s);
}

cudaError_t launch_logits_process_grad(const ProcessArgs& a, int dtype, cudaStream_t s) {
    return dtype == VH_F32    ? proc::run<float, float, true>(a, s)
           : dtype == VH_BF16 ? proc::run<__nv_bfloat16, __nv_bfloat16, true>(a, s)
                              : proc::run<__half, __half, true>(a, s);
}

}  // namespace vh
