// Processing of logits before a token is picked, and its gradient.
//
//     z = x + bias;  seen: z = z > 0 ? z / rep : z rep;  z -= freq m + pres [m > 0];  out = z / temp, or -inf
//     dx = dout / temp, seen: / rep (z > 0) or * rep, or 0
//
// Almost every token of the vocabulary is neither biased nor in the history:
// its place is one product with 1 / temperature (two units in the last place
// of fp32 at most, instead of a division's half).  The others are marked
// places.  There are CTAs of two kinds:
//
// - Dense: some rows of one sequence over a chunk of the vocabulary stream
//   through by slots of 16 aligned bytes; a slot with no allowed place is not
//   read.
// - Sparse: the marked places of the same rows.  A table in shared memory
//   counts each token (whole numbers: the order of the atomics does not
//   matter), then each place of the table is read, changed and written.  It is
//   a hash table with room for all tokens that may come; for histories past its
//   size several CTAs have a range of the vocabulary each, with a place for
//   every token.
//
// Usually the dense CTAs write every place, and the sparse ones, a kernel that
// builds its tables while the dense one ends, write theirs over it.  Where the
// output is the input, what they read must not have been written: the dense
// CTAs then look through the history too and leave the marked places of their
// chunk, a bitmap, out of their stores, so that no place is written by two
// threads or read after another wrote it, in whatever order they run.  Calls of
// few rows, where a launch counts, go that way too; for all calls it would cost
// more, since the bitmap's slots are stored element by element (gradient of
// 2048 x 65536 bf16 with histories of 512: 158 us, 111 in two kernels).
//
// Bound: memory (the logits once in and once out).  256 x 248320 bf16: 43 us
// without a history (255 MB: 0.89 of the copy rate), 48 with 512 tokens, 58 with
// 4096; the gradient of 2048 x 65536: 89 (0.90) and, with 512 tokens, 111.
#include <algorithm>

#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace proc {

constexpr int kThreadsP = 256;
// Threads of the sparse CTAs where they are a launch of their own: few tokens and many sequences (256; 2048 sequences of 512
// tokens: 111 us, 121 with 512 threads), up to kShort tokens (512; 64 sequences of 2900 tokens: 61 us, 134 with 256), more.
constexpr int kThreadsFew = 256, kThreadsShort = 512, kThreadsLong = 1024;
constexpr int kFew = 768;
constexpr int kManyCtas = 304;
// CTAs with every place up to which both kinds are one launch although the output is another one (4 x 248320 fp32, 244 CTAs:
// 6.1 us, 8.3 in two launches; 129 x 40001, 645 CTAs: 14.6 and 16.6; 16 x 248320, 976 CTAs: 10.0 and 9.4).
constexpr int kOneLaunch = 800;
constexpr uint32_t kInPrompt = 0x80000000u;
constexpr uint32_t kDrafted = 0x40000000u;
// 16-byte slots, four per thread, where every place is written: 256 x 248320 bf16 42.6 us; 32-byte ones 45.4 to 46.3.
constexpr int kSlotBytes = 16;
constexpr int kUnroll = 4;
constexpr int kMaxChunk = 32768;       // places of a dense CTA (a multiple of 128) at most
// A hash table is at most 3/4 full and has 12 bytes per place: token, count, bias entry, list; a table by tokens has 8.
constexpr int kShort = 3072;           // tokens up to which sparse CTAs are small: tables of 48 KiB
constexpr int kHashed = 12288;         // tokens of the largest hash table
constexpr int kRange = 24576;          // places of a table by tokens
constexpr int kHashBytes = 12, kRangeBytes = 8;
constexpr size_t kMostShort = (size_t)kShort / 3 * 4 * kHashBytes;
constexpr size_t kMostLong = (size_t)kRange * kRangeBytes;
static_assert(kMostLong >= (size_t)kHashed / 3 * 4 * kHashBytes && kMostShort >= (size_t)(kMaxChunk / 32 + 4) * 4, "one limit each");

struct Args {
    const void *in, *logits;
    void* out;
    long long in_stride, logits_stride, out_stride;
    int V, per_seq;
    int rows, groups;    // rows of a sequence per CTA, and CTAs for them
    int chunk, chunks;   // dense: places per CTA, and CTAs for the vocabulary
    int table;           // sparse: places of the table (0: no place is marked)
    bool hashed;         // a hash table, of a power of two
    int range, parts;    // sparse: tokens of a table by tokens; CTAs that share a sequence's marked places
    unsigned int sparse; // CTAs of the sparse kind, the first ones of the launch
    vh_logits_rules r;
};

// n <= 32 bits of a bitmap from bit `at` on, of which words beyond `last` are not read.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, long long at, int n, long long last) {
    const long long w = at >> 5;
    const uint32_t lo = words[w], hi = w < last ? words[w + 1] : 0u;
    const uint32_t b = __funnelshift_r(lo, hi, (uint32_t)at & 31u);
    return n < 32 ? b & ((1u << n) - 1u) : b;
}
__device__ __forceinline__ bool bit_at(const uint32_t* words, long long at) { return ((words[at >> 5] >> (at & 31)) & 1u) != 0u; }

// The rows of a sequence that a CTA has, and what they share.
struct Unit {
    int seq, j0, j1;
    float inv_temp;
    const int32_t* draft;  // null: none
    __device__ __forceinline__ Unit(const Args& a, unsigned int group) {
        seq = (int)(group / a.groups);
        j0 = (int)(group % a.groups) * a.rows;
        j1 = min(j0 + a.rows, a.per_seq);
        const float temp = a.r.temperature != nullptr ? __ldcg(a.r.temperature + seq) : 1.0f;
        inv_temp = temp > 0.0f ? __fdiv_rn(1.0f, temp) : 1.0f;
        draft = a.r.draft_ids != nullptr && a.per_seq > 1 ? a.r.draft_ids + (size_t)seq * (a.per_seq - 1) : nullptr;
    }
    // f(token, whether it is the prompt's) for every token of the history, over the CTA's threads.  The first tokens are asked
    // for together with the lengths.
    template <int THREADS, typename F>
    __device__ __forceinline__ void history(const Args& a, F f) const {
        if (a.r.history == nullptr) return;
        const int32_t* h = a.r.history + (size_t)seq * a.r.history_stride;
        constexpr int BATCH = 8;
        int t[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = (int)threadIdx.x + k * THREADS;
            t[k] = i < a.r.history_width ? __ldcg(h + i) : -1;
        }
        const int len = a.r.history_len != nullptr ? min(__ldcg(a.r.history_len + seq), a.r.history_width) : a.r.history_width;
        const int prompt = a.r.prompt_len != nullptr ? __ldcg(a.r.prompt_len + seq) : 0;
        for (int base = threadIdx.x; base < len; base += THREADS * BATCH) {
            if (base != (int)threadIdx.x) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) t[k] = base + k * THREADS < len ? __ldcg(h + base + k * THREADS) : -1;
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (base + k * THREADS < len) f(t[k], base + k * THREADS < prompt);
        }
    }
    // f(token, entry) for every bias; `first`: the thread's first one (see first_bias).
    template <int THREADS, typename F>
    __device__ __forceinline__ void biases(const Args& a, int first, F f) const {
        if (a.r.bias_ids == nullptr) return;
        for (int i = threadIdx.x; i < a.r.n_bias; i += THREADS)
            f(i == (int)threadIdx.x ? first : __ldcg(a.r.bias_ids + (size_t)seq * a.r.n_bias + i), i);
    }
    __device__ __forceinline__ int first_bias(const Args& a) const {
        return a.r.bias_ids != nullptr && (int)threadIdx.x < a.r.n_bias ? __ldcg(a.r.bias_ids + (size_t)seq * a.r.n_bias + threadIdx.x) : -1;
    }
};

// ---------------------------------------------------------------------------

// A row from place c0 on; slot i: elements [i * VEC - shift, +VEC).
template <typename T, typename TO>
struct Row {
    static constexpr int VEC = kSlotBytes / (int)sizeof(T);
    const T* x;
    TO* y;
    const uint32_t* ok;  // of the whole row
    int shift;
    __device__ __forceinline__ Row(const Args& a, long long row, long long c0) {
        x = static_cast<const T*>(a.in) + row * a.in_stride + c0;
        y = static_cast<TO*>(a.out) + row * a.out_stride + c0;
        ok = a.r.allowed != nullptr ? reinterpret_cast<const uint32_t*>(a.r.allowed) + row * a.r.allowed_stride : nullptr;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & (kSlotBytes - 1)) / sizeof(T));
    }
};

// The slot at element e0 (counted from the Row's c0) of a row that has elements [lo, n).
template <typename T, typename TO, bool GRAD>
struct Slot {
    static constexpr int VEC = Row<T, TO>::VEC;
    RawVec<T, VEC> in;
    uint32_t allow;
    __device__ __forceinline__ void load(const Row<T, TO>& r, int e0, int lo, int n, long long c0, long long last_word) {
        allow = (1u << VEC) - 1u;
        if (e0 >= lo && e0 + VEC <= n) {
            if (r.ok != nullptr) allow = bits_at(r.ok, c0 + e0, VEC, last_word);
            if (allow != 0u) in.load(r.x + e0);
        }
    }
    // marked: places that are left out (null: none), of so many words and one more.
    __device__ __forceinline__ void store(const Row<T, TO>& r, int e0, int lo, int n, long long c0, float scale,
                                          const uint32_t* marked, int words) const {
        constexpr int VO = kVecOf<TO>;
        const float masked = GRAD ? 0.0f : neg_inf();
        if (e0 >= n) return;
        if (e0 >= lo && e0 + VEC <= n) {
            const uint32_t skip = marked != nullptr ? bits_at(marked, e0, VEC, words) : 0u;
            auto value = [&](int i) { return (allow >> i) & 1u ? in.get(i) * scale : masked; };
            if (skip == 0u && (reinterpret_cast<uintptr_t>(r.y + e0) & 15) == 0) {
#pragma unroll
                for (int i = 0; i < VEC; i += VO) {
                    RawVec<TO, VO> o;
                    if constexpr (sizeof(TO) == 4) {
#pragma unroll
                        for (int q = 0; q < VO; ++q) o.u[q] = __float_as_uint(value(i + q));
                    } else {
#pragma unroll
                        for (int q = 0; q < VO / 2; ++q) o.set2(q, value(i + 2 * q), value(i + 2 * q + 1));
                    }
                    o.store(r.y + e0 + i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (!((skip >> i) & 1u)) r.y[e0 + i] = from_f32<TO>(value(i));
            }
        } else {  // the ends
#pragma unroll 1
            for (int e = max(e0, lo); e < min(e0 + VEC, n); ++e)
                if (marked == nullptr || !bit_at(marked, e))
                    r.y[e] = from_f32<TO>(r.ok == nullptr || bit_at(r.ok, c0 + e) ? to_f32(r.x[e]) * scale : masked);
        }
    }
};

// Some rows of a sequence over a chunk, marked places left out.
template <typename T, typename TO, bool GRAD>
__device__ __forceinline__ void dense_but_marked(const Args& a, unsigned int block, uint32_t* marked) {
    const Unit u(a, block / a.chunks);
    const long long c0 = (long long)(block % a.chunks) * a.chunk;
    const int n = (int)min((long long)a.chunk, a.V - c0);
    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    const int tid = threadIdx.x;
    const int words = a.chunk / 32;
    constexpr int VEC = Row<T, TO>::VEC;
    constexpr int kStep = kThreadsP * VEC;
    Slot<T, TO, GRAD> s[2];  // one on its way while the other is stored
    Row<T, TO> r(a, (long long)u.seq * a.per_seq + u.j0, c0);
    s[0].load(r, tid * VEC - r.shift, 0, n, c0, last_word);
    const int first = u.first_bias(a);
    for (int i = tid; i <= words; i += kThreadsP) marked[i] = 0u;
    __syncthreads();
    auto mark = [&](int token) {
        const long long at = (long long)token - c0;
        if (at >= 0 && at < n) atomicOr(marked + (at >> 5), 1u << (at & 31));
    };
    u.history<kThreadsP>(a, [&](int token, bool) { mark(token); });
    u.biases<kThreadsP>(a, first, [&](int token, int) { mark(token); });
    if (u.draft != nullptr)
        for (int i = tid; i < u.j1 - 1; i += kThreadsP) mark(__ldcg(u.draft + i));
    __syncthreads();
    for (int j = u.j0; j < u.j1; ++j) {
        int e = tid * VEC - r.shift;
        if (j > u.j0) {
            r = Row<T, TO>(a, (long long)u.seq * a.per_seq + j, c0);
            e = tid * VEC - r.shift;
            s[0].load(r, e, 0, n, c0, last_word);
        }
        for (; e < n; e += 2 * kStep) {
            s[1].load(r, e + kStep, 0, n, c0, last_word);
            s[0].store(r, e, 0, n, c0, u.inv_temp, marked, words);
            s[0].load(r, e + 2 * kStep, 0, n, c0, last_word);
            s[1].store(r, e + kStep, 0, n, c0, u.inv_temp, marked, words);
        }
    }
}

// ---------------------------------------------------------------------------

struct Table {
    uint32_t* count;  // occurrences in output, kInPrompt, kDrafted
    uint16_t* entry;  // bias entry + 1
    uint16_t* list;   // the places that are taken
    uint32_t* key;    // token + 1, 0: none; null: the place is the token's
    uint32_t mask;
    int shift;
    __device__ __forceinline__ Table(uint32_t* base, int n, bool hashed)
        : count(base), entry(reinterpret_cast<uint16_t*>(base + n)), list(entry + n), key(hashed ? base + 2 * n : nullptr),
          mask((uint32_t)n - 1u) {
        shift = __clz(n) + 1;
    }
    // The place of a token (counted from the CTA's first one).
    __device__ __forceinline__ uint32_t place(uint32_t token) const {
        if (key == nullptr) return token;
        uint32_t p = (token * 2654435769u) >> shift;  // 2^32 / golden ratio: neighbours lie far apart
        while (true) {
            const uint32_t was = atomicCAS(key + p, 0u, token + 1u);
            if (was == 0u || was == token + 1u) return p;
            p = (p + 1u) & mask;
        }
    }
    __device__ __forceinline__ bool taken(int p) const { return key != nullptr ? key[p] != 0u : (count[p] != 0u || entry[p] != 0u); }
};

// LATE: what is read up to the logits is read past the first-level cache, before the previous kernel (the dense one, which has
// waited for its predecessors before it let this one start) has ended.
template <typename T, typename TO, bool GRAD, int THREADS, bool LATE>
__device__ __forceinline__ void sparse(const Args& a, unsigned int block, uint32_t* smem) {
    __shared__ int s_taken;
    const float masked = GRAD ? 0.0f : neg_inf();
    const Unit u(a, block / a.parts);
    const uint32_t part = block % a.parts;
    const long long v0 = a.hashed ? 0 : (long long)part * a.range;
    const long long range = a.hashed ? a.V : min((long long)a.range, a.V - v0);
    const Table t(smem, a.table, a.hashed);
    const int tid = threadIdx.x;
    const float rep = a.r.repetition != nullptr ? __ldcg(a.r.repetition + u.seq) : 1.0f;
    const float freq = a.r.frequency != nullptr ? __ldcg(a.r.frequency + u.seq) : 0.0f;
    const float pres = a.r.presence != nullptr ? __ldcg(a.r.presence + u.seq) : 0.0f;
    const int first = u.first_bias(a);
    for (int i = tid; i < a.table * (a.hashed ? kHashBytes : kRangeBytes) / 16; i += THREADS)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_taken = 0;
    __syncthreads();
    // f(place) if the token is this CTA's: of its range, or by its hash
    auto at = [&](int token, auto f) {
        const long long v = (long long)token - v0;
        if (v < 0 || v >= range) return;
        if (a.hashed && a.parts > 1 && __umulhi((uint32_t)v * 2246822519u, (uint32_t)a.parts) != part) return;  // an odd number's product
        f(t.place((uint32_t)v));
    };
    u.history<THREADS>(a, [&](int token, bool prompt) {
        at(token, [&](uint32_t p) {
            if (prompt)
                atomicOr(t.count + p, kInPrompt);
            else
                atomicAdd(t.count + p, 1u);
        });
    });
    if (u.draft != nullptr)
        for (int i = tid; i < u.j1 - 1; i += THREADS)
            at(__ldcg(u.draft + i), [&](uint32_t p) {
                if (i < u.j0)
                    atomicAdd(t.count + p, 1u);  // before all of the CTA's rows
                else
                    atomicOr(t.count + p, kDrafted);
            });
    u.biases<THREADS>(a, first, [&](int token, int i) {
        at(token, [&](uint32_t p) {
            // the last entry of an id: the larger one, in its half of a word
            uint32_t* w = reinterpret_cast<uint32_t*>(t.entry) + (p >> 1);
            const int sh = (int)(p & 1u) * 16;
            uint32_t old = *w;
            while (((old >> sh) & 0xFFFFu) < (uint32_t)(i + 1)) {
                const uint32_t was = atomicCAS(w, old, (old & ~(0xFFFFu << sh)) | (uint32_t)(i + 1) << sh);
                if (was == old) break;
                old = was;
            }
        });
    });
    __syncthreads();
    for (int p0 = tid - (tid & 31); p0 < a.table; p0 += THREADS) {  // tables are of whole warps
        const bool taken = t.taken(p0 + (tid & 31));
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, taken);
        int first = 0;
        if ((tid & 31) == 0 && all != 0u) first = atomicAdd(&s_taken, __popc(all));
        first = __shfl_sync(0xFFFFFFFFu, first, 0);
        if (taken) t.list[first + __popc(all & ((1u << (tid & 31)) - 1u))] = (uint16_t)(p0 + (tid & 31));
    }
    __syncthreads();
    if constexpr (LATE) rows_wait();
    constexpr int UNROLL = 4;  // places with their reads in flight
    for (int i0 = tid; i0 < s_taken; i0 += THREADS * UNROLL) {
        int token[UNROLL];
        uint32_t count[UNROLL], entry[UNROLL];
        float bias[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            token[k] = -1;
            if (i0 + k * THREADS < s_taken) {
                const int p = t.list[i0 + k * THREADS];
                token[k] = a.hashed ? (int)t.key[p] - 1 : (int)(v0 + p);
                count[k] = t.count[p];
                entry[k] = t.entry[p];
                bias[k] = entry[k] != 0u ? a.r.bias[(size_t)u.seq * a.r.n_bias + entry[k] - 1u] : 0.0f;
            }
        }
        for (int j = u.j0; j < u.j1; ++j) {
            const long long row = (long long)u.seq * a.per_seq + j;
            const T* x = static_cast<const T*>(a.in) + row * a.in_stride;
            const T* lg = static_cast<const T*>(a.logits) + row * a.logits_stride;
            TO* y = static_cast<TO*>(a.out) + row * a.out_stride;
            const uint32_t* ok = a.r.allowed != nullptr ? reinterpret_cast<const uint32_t*>(a.r.allowed) + row * a.r.allowed_stride : nullptr;
            T in[UNROLL], lo[UNROLL];
            bool off[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k)
                if (token[k] >= 0) {
                    in[k] = x[token[k]];
                    if constexpr (GRAD) lo[k] = lg[token[k]];
                    off[k] = ok != nullptr && !bit_at(ok, token[k]);
                }
            const int drafted = j > u.j0 && u.draft != nullptr ? u.draft[j - 1] : -1;
#pragma unroll
            for (int k = 0; k < UNROLL; ++k)
                if (token[k] >= 0) {
                    if (token[k] == drafted) ++count[k];
                    const uint32_t m = count[k] & ~(kInPrompt | kDrafted);
                    const bool seen = m > 0u || (count[k] & kInPrompt) != 0u;
                    float z = to_f32(GRAD ? lo[k] : in[k]);
                    if (entry[k] != 0u) z += bias[k];
                    float r = GRAD ? to_f32(in[k]) : z;
                    if (seen) r = z > 0.0f ? __fdiv_rn(r, rep) : r * rep;
                    if (!GRAD && m > 0u) r = __fsub_rn(__fsub_rn(r, __fmul_rn(freq, (float)m)), pres);
                    y[token[k]] = from_f32<TO>(off[k] ? masked : r * u.inv_temp);
                }
        }
    }
}

// Every place of a row, a few slots per thread, all asked for before anything else; the sparse kernel follows where there
// are marked ones.
template <typename T, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThreadsP) k_process(const Args a, int chunks) {
    constexpr int VEC = Row<T, TO>::VEC;
    constexpr int kStep = kThreadsP * VEC;
    rows_wait();
    if (a.table > 0) rows_launch_dependents();
    const long long row = blockIdx.x / chunks;
    const long long c0 = (long long)(blockIdx.x % chunks) * (kStep * kUnroll);  // the slots begin `shift` before it
    const Row<T, TO> r(a, row, c0);
    const int lo = c0 > 0 ? -r.shift : 0, n = (int)min(a.V - c0, (long long)kStep * kUnroll);
    const int e0 = (int)threadIdx.x * VEC - r.shift;
    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    Slot<T, TO, GRAD> s[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) s[k].load(r, e0 + k * kStep, lo, n, c0, last_word);
    const float temp = a.r.temperature != nullptr ? a.r.temperature[row / a.per_seq] : 1.0f;
    const float inv_temp = temp > 0.0f ? __fdiv_rn(1.0f, temp) : 1.0f;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) s[k].store(r, e0 + k * kStep, lo, n, c0, inv_temp, nullptr, 0);
}
template <typename T, typename TO, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS) k_process_marked(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    sparse<T, TO, GRAD, THREADS, true>(a, blockIdx.x, s_words);
}

// Both kinds in one launch, marked places left to the sparse ones.
template <typename T, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThreadsP) k_process_apart(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    rows_wait();
    if (blockIdx.x < a.sparse)
        sparse<T, TO, GRAD, kThreadsP, false>(a, blockIdx.x, s_words);
    else
        dense_but_marked<T, TO, GRAD>(a, blockIdx.x - a.sparse, s_words);
}
template <typename T, bool GRAD>
__global__ void __launch_bounds__(kThreadsLong) k_process_marked_first(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    rows_wait();
    sparse<T, T, GRAD, kThreadsLong, false>(a, blockIdx.x, s_words);
}

static int cut(long long n, long long by) { return (int)((n + by - 1) / by); }

// How the work is cut.
struct Plan {
    int chunks;       // per row, where every place is written
    long long whole;  // CTAs then
    long long dense;  // CTAs that leave marked places out
    long long sparse;
    long long marks;  // places, at most
    bool small;       // the sparse ones
    size_t bitmap, table;
    // size: of a logit
    Plan(Args& a, int S, int size) {
        const long long per = (long long)kThreadsP * kUnroll * (kSlotBytes / size);
        chunks = cut((long long)a.V + kSlotBytes / size - 1, per);  // up to a slot less one begins before the row
        whole = (long long)S * a.per_seq * chunks;
        constexpr int kResident = 152 * 4;
        // rows of a sequence share a table as long as the machine is filled
        a.rows = std::min(a.per_seq, 8);
        while (a.rows > 1 && (long long)S * cut(a.per_seq, a.rows) * cut(a.V, 4096) < kResident) a.rows = (a.rows + 1) / 2;
        a.groups = cut(a.per_seq, a.rows);
        // chunks of even size: some waves of CTAs, or one
        const long long units = (long long)S * a.groups;
        const long long wanted = std::max<long long>(1, std::min<long long>(cut(a.V, 8192) * units >= 4 * kResident ? 4 * kResident / units : kResident / units, cut(a.V, 1024)));
        a.chunks = (int)std::max<long long>(cut(a.V, kMaxChunk), wanted);
        a.chunk = cut(cut(a.V, a.chunks), 128) * 128;
        a.chunks = cut(a.V, a.chunk);
        dense = units * a.chunks;
        marks = (a.r.history != nullptr ? a.r.history_width : 0) + (a.r.bias_ids != nullptr ? a.r.n_bias : 0) +
                                (a.r.draft_ids != nullptr ? a.per_seq - 1ll : 0);
        const long long most = std::min<long long>(marks, a.V);
        sparse = 0;
        small = most <= kShort;
        bitmap = (size_t)(a.chunk / 32 + 4) * 4;
        table = 0;
        a.table = 0;
        if (most > 0) {
            a.hashed = most <= kHashed;
            a.table = a.hashed ? 128 : kRange;
            while (a.hashed && a.table * 3ll < most * 4) a.table *= 2;
            a.range = kRange;
            // a few hundred places per CTA while there are SMs left
            a.parts = a.hashed ? (int)std::max<long long>(1, std::min<long long>({most / 256, 152 / units, 8})) : cut(a.V, kRange);
            sparse = units * a.parts;
            table = (size_t)a.table * (a.hashed ? kHashBytes : kRangeBytes);
        }
    }
};

template <typename... P, typename... A>
static cudaError_t launch(void (*kernel)(P...), long long ctas, int threads, size_t smem, size_t most, cudaStream_t s, A... args) {
    if (most > 0) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
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
    if (a.per_seq == 1) a.r.draft_ids = nullptr;
    const Plan plan(a, p.R / p.per_seq, (int)sizeof(T));
    if (std::max(plan.whole, plan.dense + plan.sparse) > 2147483647ll) return cudaErrorInvalidValue;
    cudaError_t e;
    const bool in_place = p.out == p.in;
    if (a.table == 0) return launch(k_process<T, TO, GRAD>, plan.whole, kThreadsP, 0, 0, s, a, plan.chunks);
    if (plan.small && (in_place || plan.whole <= kOneLaunch)) {
        a.sparse = (unsigned int)plan.sparse;
        return launch(k_process_apart<T, TO, GRAD>, plan.sparse + plan.dense, kThreadsP, std::max(plan.bitmap, plan.table), kMostShort,
                      s, a);
    }
    if (!in_place) {
        e = launch(k_process<T, TO, GRAD>, plan.whole, kThreadsP, 0, 0, s, a, plan.chunks);
        if (e != cudaSuccess) return e;
        return plan.marks <= kFew && plan.sparse > kManyCtas
                   ? launch(k_process_marked<T, TO, GRAD, kThreadsFew>, plan.sparse, kThreadsFew, plan.table, kMostShort, s, a)
               : plan.small
                   ? launch(k_process_marked<T, TO, GRAD, kThreadsShort>, plan.sparse, kThreadsShort, plan.table, kMostShort, s, a)
                   : launch(k_process_marked<T, TO, GRAD, kThreadsLong>, plan.sparse, kThreadsLong, plan.table, kMostLong, s, a);
    }
    if constexpr (std::is_same<T, TO>::value) {
        e = launch(k_process_marked_first<T, GRAD>, plan.sparse, kThreadsLong, plan.table, kMostLong, s, a);
        if (e != cudaSuccess) return e;
        return launch(k_process_apart<T, T, GRAD>, plan.dense, kThreadsP, plan.bitmap, kMostShort, s, a);
    }
    return cudaErrorInvalidValue;
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
