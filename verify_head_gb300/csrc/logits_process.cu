// Processing of logits before a token is picked, and its gradient.
//
//     z = x + bias;  seen: z = z > 0 ? z / rep : z rep;  z -= freq m + pres [m > 0];  out = z / temp, or -inf
//     dx = dout / temp, seen: / rep (z > 0) or * rep, or 0
//
// Almost every token of the vocabulary is neither biased nor in the history:
// its place is one product with 1 / temperature (two units in the last place
// of fp32 at most, instead of a division's half).  The others are marked
// places.  Rows stream through by slots of 16 aligned bytes; a slot with no
// allowed place is not read.
//
// Large calls: one kernel streams every place (k_process_stream), and a second
// one (k_process_marked), which builds its tables while the first ends, writes
// the marked places over it.  A table in shared memory counts each token of
// the history, drafted and biased ones among them (whole numbers: the order of
// the atomics does not matter), then each place of the table is read, changed
// and written.  It is a hash table with room for all tokens that may come; for
// histories past its size several CTAs have a range of the vocabulary each,
// with a place for every token.
//
// Small calls, where a launch counts: one kernel (k_process_small).  A CTA has
// some rows of one sequence over a chunk of the vocabulary.  It looks through
// the history, the slots of a row of logits already on their way, counts the
// tokens of its chunk in 16 bits each and lists the marked places.  It writes
// all of a row's places, and after a barrier the listed ones again, shared out
// over its threads.
//
// Outputs that are the inputs, whose marked places would be lost that way, and
// long histories of small calls or of most of the vocabulary: one kernel
// (k_process) that counts like this and changes a marked place in its slot's
// registers, so that every slot is read and written once, by one thread.  Most
// warps have a marked place in some lane and wait for it.  With long histories
// its CTAs have 1,024 threads and chunks to match, so that fewer of them look
// through the same one.
//
//     us                                        small    in registers    two kernels
//     4 x 248320 fp32, history 1500               5.1             5.5            8.3
//     129 x 40001 fp16 to fp32, masked, 700      11.7            13.3           16.6
//     4 x 248320 fp32, history 8000              11.9             7.4
//     201 x 65536 fp16, masked, 9951                             35             59
//     256 x 248320 bf16, histories of 4096       69.4            94             58
//     256 x 248320 bf16, histories of 512                        69             45
//     2048 x 65536 bf16, histories of 512                       152            105
//     gradient of 2048 x 65536, 512                             179            110
//
// (The second column of the last three is what these calls take in place.)
//
// Bound: memory (the logits once in and once out).  256 x 248320 bf16: 43 us
// without a history (255 MB: 0.89 of the copy rate), 45 with 512 tokens, 58 with
// 4096: of each marked place the logit is read again and the output's sector
// filled and written again, long after the stream has left L2.  The gradient of
// 2048 x 65536: 89 us (0.90) and, with 512 tokens, 110.
#include <algorithm>
#include <type_traits>

#include "vh_row_kernels.h"
#include "vh_rows.cuh"

namespace vh {
namespace proc {

constexpr int kThreadsP = 256;
constexpr int kSlotBytes = 16;   // of logits per thread and load (256 x 248320 bf16 42.6 us; 32 bytes 45.4)
constexpr int kStreamSlots = 4;  // slots per thread, all asked for at once; in k_process
constexpr int kUnroll = 2;       // (four: as fast or slower)
constexpr int kMaxRows = 8;      // of a sequence per CTA
// Calls of up to so many CTAs of k_process_stream are small (129 x 40001, 645: above; 16 x 248320, 976: 10.0 us in registers, 9.4 in
// two kernels), and histories of up to kFewTokens are short (4 x 248320 with 3000: 6.4 us listed, 6.1 in registers; 129 x 40001 with
// 1500: 12.9 and 14.6).  In registers they want 256 threads (in place 64 sequences of 4 rows of 248320, 512 tokens: 69 us, 77 with
// 1,024; 2048 x 65536: 158 and 183), longer ones 1,024 (4 x 248320 with 8000: 9.7 and 7.4; 33 x 40001 with 20000: 21 and 12).
constexpr int kOneLaunch = 800;
constexpr int kFewTokens = 2048;
// Larger calls with one or two rows per sequence and more than kLongTokens, more than 1 / kDense of the vocabulary, are changed in
// registers too (135 sequences of 2 x 248320, 14815 tokens: 126 us, 152 in two kernels; 45 x 178281, 24762: 30 and 43; but 619 x 2 x
// 29595, 3232: 97 and 80; 270 x 248320, 7000: 147 and 135; 64 x 4 x 248320, 16000: 129 and 111).
constexpr int kLongTokens = 4096, kDense = 20;
// CTAs of k_process_small per SM (four: 129 x 40001 12.6 us, in more than one wave; 4 x 248320 5.0).  That is 48 registers a thread,
// for which the instances spill up to 48 bytes.
constexpr int kPerSmSmall = 5;
constexpr int kChunkPerThread = 32;  // places of a CTA of k_process at most, for each of its threads
constexpr int kBefore = 128;    // places of k_process_small's table before its chunk (a slot's at least, whole words of 16 bytes)
constexpr int kMostNarrow = 32767;  // tokens that 16-bit counts hold, beside the prompt's bit
constexpr uint32_t kInPrompt = 0x80000000u;
constexpr uint32_t kDrafted = 0x40000000u;
// Threads of k_process_marked: few tokens and many sequences (256; 2048 sequences of 512 tokens: 111 us, 121 with 512 threads), up
// to kShort tokens (512; 64 sequences of 2900 tokens: 61 us, 134 with 256), more.
constexpr int kThreadsFew = 256, kThreadsShort = 512, kThreadsLong = 1024;
constexpr int kFew = 768;
constexpr int kManyCtas = 304;
// A hash table is at most 3/4 full and has 12 bytes per place: token, count, bias entry, list; a table by tokens has 8.
constexpr int kShort = 4096 / 4 * 3;  // tokens up to which several CTAs with a table fit an SM (48 KiB)
constexpr int kHashed = 12288;   // tokens of the largest hash table
constexpr int kRange = 24576;    // places of a table by tokens
constexpr int kHashBytes = 12, kRangeBytes = 8;
constexpr size_t kMostShort = (size_t)kShort / 3 * 4 * kHashBytes;
constexpr size_t kMostLong = (size_t)kRange * kRangeBytes;
static_assert(kMostLong >= (size_t)kHashed / 3 * 4 * kHashBytes, "one limit for both kinds of table");

struct Args {
    const void *in, *logits;
    void* out;
    long long in_stride, logits_stride, out_stride;
    int V, per_seq;
    int rows, groups;   // rows of a sequence per CTA, and CTAs for them
    int chunk, chunks;  // k_process: places per CTA, and CTAs for the vocabulary
    int table;          // k_process_marked: places of the table
    bool hashed;        // a hash table, of a power of two
    int range, parts;   // tokens of a table by tokens; CTAs that share a sequence's marked places
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

// Of a temperature; a finite number also where that is below 2^-128, since 0 times it has to be 0.  The product with it is off by two
// roundings of 2^-24, where a quotient would be by one.
__device__ __forceinline__ float inverse(float temp) {
    return temp > 0.0f ? fminf(__fdiv_rn(1.0f, temp), 3.40282347e38f) : 1.0f;
}

// A row from place c0 on; its slots begin `shift` elements before an aligned place.
template <typename T, typename TO>
struct Row {
    static constexpr int VEC = kSlotBytes / (int)sizeof(T);
    const T* x;
    TO* y;
    const T* logits;
    const uint32_t* ok;  // of the whole row
    int shift;
    __device__ __forceinline__ Row(const Args& a, long long row, long long c0) {
        x = static_cast<const T*>(a.in) + row * a.in_stride + c0;
        y = static_cast<TO*>(a.out) + row * a.out_stride + c0;
        logits = static_cast<const T*>(a.logits) + row * a.logits_stride + c0;
        ok = a.r.allowed != nullptr ? reinterpret_cast<const uint32_t*>(a.r.allowed) + row * a.r.allowed_stride : nullptr;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & (kSlotBytes - 1)) / sizeof(T));
    }
};

// What a CTA knows of its chunk's tokens.  WIDE: counts of 32 bits, else of 16, two to a word; the highest bit is the prompt's.
template <bool WIDE>
struct Marks {
    uint32_t* count;
    uint32_t* bits;    // [chunk / 32], and a word that bits_at reads past them
    uint16_t* entry;   // bias entry + 1 (null: no biases)
    int words;
    __host__ __device__ static constexpr size_t bytes(int chunk, bool biased) {
        return (size_t)chunk * ((WIDE ? 4 : 2) + (biased ? 2 : 0)) + (size_t)(chunk / 32 + 4) * 4;  // a multiple of 16
    }
    __device__ __forceinline__ Marks(uint32_t* base, int chunk, bool biased) {
        count = base;
        bits = base + (WIDE ? chunk : chunk / 2);
        words = chunk / 32;
        entry = biased ? reinterpret_cast<uint16_t*>(bits + words + 4) : nullptr;
    }
    // Whether the place had not been marked.
    __device__ __forceinline__ bool mark(int at) const {
        const uint32_t bit = 1u << (at & 31);
        return (atomicOr(bits + (at >> 5), bit) & bit) == 0u;
    }
    __device__ __forceinline__ void add(int at, bool prompt) const {
        uint32_t* w = count + (WIDE ? at : at >> 1);
        const int sh = WIDE ? 0 : (at & 1) * 16;
        if (prompt)
            atomicOr(w, (WIDE ? 0x80000000u : 0x8000u) << sh);
        else
            atomicAdd(w, 1u << sh);
    }
    // The last entry of an id counts: the larger one, in its half of a word.
    __device__ __forceinline__ void bias(int at, int i) const {
        uint32_t* w = reinterpret_cast<uint32_t*>(entry) + (at >> 1);
        const int sh = (at & 1) * 16;
        uint32_t old = *w;
        while (((old >> sh) & 0xFFFFu) < (uint32_t)(i + 1)) {
            const uint32_t was = atomicCAS(w, old, (old & ~(0xFFFFu << sh)) | (uint32_t)(i + 1) << sh);
            if (was == old) break;
            old = was;
        }
    }
    // Occurrences in output, and whether the prompt has the token.
    __device__ __forceinline__ uint32_t get(int at, bool& prompt) const {
        const uint32_t c = WIDE ? count[at] : (count[at >> 1] >> ((at & 1) * 16)) & 0xFFFFu;
        prompt = (c & (WIDE ? 0x80000000u : 0x8000u)) != 0u;
        return c & (WIDE ? 0x7FFFFFFFu : 0x7FFFu);
    }
};

// What one sequence's rows share.
struct Rules {
    float rep, freq, pres, inv_temp;
    const float* bias;
    const int* draft;  // of the CTA's rows (shared memory), null: none
};

// A marked place of row j (of the CTA's), `v` its logit, or its gradient with `z` the logit.
template <bool GRAD, bool WIDE>
__device__ __forceinline__ float apply(const Rules& u, const Marks<WIDE>& c, int at, long long token, int j, float z, float v) {
    const uint32_t e = c.entry != nullptr ? c.entry[at] : 0u;
    if (e != 0u) z += u.bias[e - 1u];
    bool seen;
    uint32_t m = c.get(at, seen);
    if (u.draft != nullptr)
        for (int i = 0; i < j; ++i) m += u.draft[i] == token;
    seen = seen || m > 0u;
    float r = GRAD ? v : z;
    if (seen) r = z > 0.0f ? __fdiv_rn(r, u.rep) : r * u.rep;
    if (!GRAD && m > 0u) r = __fsub_rn(__fsub_rn(r, __fmul_rn(u.freq, (float)m)), u.pres);
    return r * u.inv_temp;
}

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
    __device__ __forceinline__ float pick(int i) const {  // element i, by selects
        const uint32_t u0 = in.u[0], u1 = in.u[1], u2 = in.u[2], u3 = in.u[3];
        const int k = sizeof(T) == 4 ? i : i >> 1;
        const uint32_t lo = (k & 1) ? u1 : u0, hi = (k & 1) ? u3 : u2, w = (k & 2) ? hi : lo;
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w);
        } else {
            const unsigned short h = (unsigned short)(w >> ((i & 1) * 16));
            return to_f32(*reinterpret_cast<const T*>(&h));
        }
    }
    // marked(first element, number) -> bits; change(element, logit of the row or gradient) -> value.
    template <typename M, typename C>
    __device__ __forceinline__ void store(const Row<T, TO>& r, int e0, int lo, int n, long long c0, float scale, M marked,
                                          C change) const {
        constexpr int VO = kVecOf<TO>;
        const float masked = GRAD ? 0.0f : neg_inf();
        if (e0 >= n) return;
        if (e0 >= lo && e0 + VEC <= n) {
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = (allow >> i) & 1u ? in.get(i) * scale : masked;
            uint32_t todo = marked(e0, VEC) & allow;
            while (todo != 0u) {
                const int i = __ffs((int)todo) - 1;
                todo &= todo - 1u;
                const float c = change(e0 + i, pick(i));
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = k == i ? c : v[k];
            }
            if ((reinterpret_cast<uintptr_t>(r.y + e0) & 15) == 0) {
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
                    o.store(r.y + e0 + i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) r.y[e0 + i] = from_f32<TO>(v[i]);
            }
        } else {  // the ends
#pragma unroll 1
            for (int e = max(e0, lo); e < min(e0 + VEC, n); ++e) {
                float v = masked;
                if (r.ok == nullptr || bit_at(r.ok, c0 + e)) {
                    v = to_f32(r.x[e]);
                    v = marked(e, 1) != 0u ? change(e, v) : v * scale;
                }
                r.y[e] = from_f32<TO>(v);
            }
        }
    }
};

// Every place, a few slots per thread, all asked for before anything else; k_process_marked follows where places are marked.
template <typename T, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThreadsP) k_process_stream(const Args a, int chunks, bool more) {
    constexpr int VEC = Row<T, TO>::VEC;
    constexpr int kStep = kThreadsP * VEC;
    rows_wait();
    if (more) rows_launch_dependents();
    const long long row = blockIdx.x / chunks;
    const long long c0 = (long long)(blockIdx.x % chunks) * (kStep * kStreamSlots);  // the slots begin `shift` before it
    const Row<T, TO> r(a, row, c0);
    const int lo = c0 > 0 ? -r.shift : 0, n = (int)min(a.V - c0, (long long)kStep * kStreamSlots);
    const int e0 = (int)threadIdx.x * VEC - r.shift;
    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    Slot<T, TO, GRAD> s[kStreamSlots];
#pragma unroll
    for (int k = 0; k < kStreamSlots; ++k) s[k].load(r, e0 + k * kStep, lo, n, c0, last_word);
    const float temp = a.r.temperature != nullptr ? a.r.temperature[row / a.per_seq] : 1.0f;
    const float inv_temp = inverse(temp);
#pragma unroll
    for (int k = 0; k < kStreamSlots; ++k)
        s[k].store(r, e0 + k * kStep, lo, n, c0, inv_temp, [](int, int) { return 0u; }, [](int, float v) { return v; });
}

template <typename T, typename TO, bool GRAD, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_process(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    __shared__ int s_draft[kMaxRows];
    constexpr int VEC = Row<T, TO>::VEC;
    constexpr int kStep = THREADS * VEC;
    rows_wait();
    const unsigned int part = blockIdx.x / a.chunks;
    const int seq = (int)(part / a.groups);
    const int j0 = (int)(part % a.groups) * a.rows, j1 = min(j0 + a.rows, a.per_seq);
    const long long c0 = (long long)(blockIdx.x % a.chunks) * a.chunk;
    const int n = (int)min((long long)a.chunk, a.V - c0);
    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    const int tid = threadIdx.x;
    const bool biased = a.r.bias_ids != nullptr;
    const Marks<WIDE> c(s_words, a.chunk, biased);

    // The first slots, and everything that one look needs, are asked for before the rest begins.
    Row<T, TO> r(a, (long long)seq * a.per_seq + j0, c0);
    Slot<T, TO, GRAD> s[kUnroll];
    int e = tid * VEC - r.shift;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) s[k].load(r, e + k * kStep, 0, n, c0, last_word);
    constexpr int BATCH = 4;
    const int32_t* h = a.r.history != nullptr ? a.r.history + (size_t)seq * a.r.history_stride : nullptr;
    int t[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) t[k] = h != nullptr && tid + k * THREADS < a.r.history_width ? h[tid + k * THREADS] : -1;
    const int len = h == nullptr ? 0 : a.r.history_len != nullptr ? min(a.r.history_len[seq], a.r.history_width) : a.r.history_width;
    const int prompt = h != nullptr && a.r.prompt_len != nullptr ? a.r.prompt_len[seq] : 0;
    const int32_t* bias_ids = biased ? a.r.bias_ids + (size_t)seq * a.r.n_bias : nullptr;
    const int first_bias = biased && tid < a.r.n_bias ? bias_ids[tid] : -1;
    const int32_t* draft = a.r.draft_ids != nullptr && a.per_seq > 1 ? a.r.draft_ids + (size_t)seq * (a.per_seq - 1) : nullptr;

    for (int i = tid; i < (int)(Marks<WIDE>::bytes(a.chunk, biased) / 16); i += THREADS)
        reinterpret_cast<uint4*>(s_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (draft != nullptr && tid < j1 - 1 - j0) s_draft[tid] = draft[j0 + tid];
    __syncthreads();
    // The place of a token in the chunk, or -1.
    auto place = [&](int token) {
        const long long at = (long long)token - c0;
        return at >= 0 && at < n ? (int)at : -1;
    };
    for (int base = tid; base < len; base += THREADS * BATCH) {
        int next[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = base + (k + BATCH) * THREADS;
            next[k] = i < len ? h[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = base + k * THREADS, at = place(t[k]);
            if (i < len && at >= 0) {
                c.add(at, i < prompt);
                c.mark(at);
            }
            t[k] = next[k];
        }
    }
    if (biased)
        for (int i = tid; i < a.r.n_bias; i += THREADS) {
            const int at = place(i == tid ? first_bias : bias_ids[i]);
            if (at < 0) continue;
            c.bias(at, i);
            c.mark(at);
        }
    if (draft != nullptr)
        for (int i = tid; i < j1 - 1; i += THREADS) {
            const int at = place(draft[i]);
            if (at < 0) continue;
            if (i < j0) c.add(at, false);  // before all of the CTA's rows
            c.mark(at);
        }
    Rules u;
    u.rep = a.r.repetition != nullptr ? a.r.repetition[seq] : 1.0f;
    u.freq = a.r.frequency != nullptr ? a.r.frequency[seq] : 0.0f;
    u.pres = a.r.presence != nullptr ? a.r.presence[seq] : 0.0f;
    const float temp = a.r.temperature != nullptr ? a.r.temperature[seq] : 1.0f;
    u.inv_temp = inverse(temp);
    u.bias = biased ? a.r.bias + (size_t)seq * a.r.n_bias : nullptr;
    u.draft = draft != nullptr ? s_draft : nullptr;
    __syncthreads();

    int j = j0;
    while (true) {
        auto store = [&](const Slot<T, TO, GRAD>& slot, int at_e) {
            slot.store(r, at_e, 0, n, c0, u.inv_temp, [&](int at, int count) { return bits_at(c.bits, at, count, c.words); },
                       [&](int at, float v) {
                           const float z = GRAD ? to_f32(r.logits[at]) : v;
                           return apply<GRAD, WIDE>(u, c, at, c0 + at, j - j0, z, v);
                       });
        };
        store(s[0], e);
        store(s[1], e + kStep);
        static_assert(kUnroll == 2, "as written out here");
        e += kUnroll * kStep;
        if (e - tid * VEC >= n) {  // the row's last slots: the same for all threads
            if (++j == j1) break;
            r = Row<T, TO>(a, (long long)seq * a.per_seq + j, c0);
            e = tid * VEC - r.shift;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) s[k].load(r, e + k * kStep, 0, n, c0, last_word);
    }
}

// Every place of some rows of a sequence, then the marked ones again.  A chunk has as many places as the CTA's threads have slots;
// as the slots begin `shift` places before it, so does the table.  The slots of the next row are on their way while a row's
// marked places are written.
template <typename T, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThreadsP, kPerSmSmall) k_process_small(const Args a) {
    extern __shared__ __align__(16) uint32_t s_words[];
    __shared__ int s_draft[kMaxRows];
    __shared__ int s_marks;
    constexpr int VEC = Row<T, TO>::VEC;
    constexpr int kStep = kThreadsP * VEC;
    constexpr int kPlaces = kStep * kStreamSlots;
    rows_wait();
    const unsigned int part = blockIdx.x / a.chunks;
    const int seq = (int)(part / a.groups);
    const int j0 = (int)(part % a.groups) * a.rows, j1 = min(j0 + a.rows, a.per_seq);
    const long long c0 = (long long)(blockIdx.x % a.chunks) * kPlaces;
    const long long last_word = ((long long)a.V + 31) / 32 - 1;
    const int tid = threadIdx.x;
    const bool biased = a.r.bias_ids != nullptr;
    const Marks<false> c(s_words, kPlaces + kBefore, biased);
    uint16_t* list = reinterpret_cast<uint16_t*>(s_words + Marks<false>::bytes(kPlaces + kBefore, biased) / 4);
    const int lo = c0 > 0 ? -VEC : 0, n = (int)min(a.V - c0, (long long)kPlaces);  // of all rows

    Row<T, TO> r(a, (long long)seq * a.per_seq + j0, c0);
    Slot<T, TO, GRAD> s[kStreamSlots];
    int from, to, e;  // the places that the row's slots hold, and the thread's first slot
    auto load = [&]() {
        from = c0 > 0 ? -r.shift : 0;
        to = (int)min(a.V - c0, (long long)kPlaces - r.shift);
        e = tid * VEC - r.shift;
#pragma unroll
        for (int k = 0; k < kStreamSlots; ++k) s[k].load(r, e + k * kStep, from, to, c0, last_word);
    };
    load();
    constexpr int BATCH = 4;
    const int32_t* h = a.r.history != nullptr ? a.r.history + (size_t)seq * a.r.history_stride : nullptr;
    int t[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) t[k] = h != nullptr && tid + k * kThreadsP < a.r.history_width ? h[tid + k * kThreadsP] : -1;
    const int len = h == nullptr ? 0 : a.r.history_len != nullptr ? min(a.r.history_len[seq], a.r.history_width) : a.r.history_width;
    const int prompt = h != nullptr && a.r.prompt_len != nullptr ? a.r.prompt_len[seq] : 0;
    const int32_t* bias_ids = biased ? a.r.bias_ids + (size_t)seq * a.r.n_bias : nullptr;
    const int first_bias = biased && tid < a.r.n_bias ? bias_ids[tid] : -1;
    const int32_t* draft = a.r.draft_ids != nullptr && a.per_seq > 1 ? a.r.draft_ids + (size_t)seq * (a.per_seq - 1) : nullptr;

    for (int i = tid; i < (int)(Marks<false>::bytes(kPlaces + kBefore, biased) / 16); i += kThreadsP)
        reinterpret_cast<uint4*>(s_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (draft != nullptr && tid < j1 - 1 - j0) s_draft[tid] = draft[j0 + tid];
    if (tid == 0) s_marks = 0;
    __syncthreads();
    // f(place in the table) for a token of the chunk; the first to mark it puts it on the list
    auto with = [&](int token, auto f) {
        const long long at = (long long)token - c0;
        if (at < lo || at >= n) return;
        const int p = (int)at + kBefore;
        f(p);
        if (c.mark(p)) list[atomicAdd(&s_marks, 1)] = (uint16_t)p;
    };
    for (int base = tid; base < len; base += kThreadsP * BATCH) {
        int next[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = base + (k + BATCH) * kThreadsP;
            next[k] = i < len ? h[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = base + k * kThreadsP;
            if (i < len) with(t[k], [&](int p) { c.add(p, i < prompt); });
            t[k] = next[k];
        }
    }
    if (biased)
        for (int i = tid; i < a.r.n_bias; i += kThreadsP)
            with(i == tid ? first_bias : bias_ids[i], [&](int p) { c.bias(p, i); });
    if (draft != nullptr)
        for (int i = tid; i < j1 - 1; i += kThreadsP)
            with(draft[i], [&](int p) {
                if (i < j0) c.add(p, false);  // before all of the CTA's rows
            });
    Rules u;
    u.rep = a.r.repetition != nullptr ? a.r.repetition[seq] : 1.0f;
    u.freq = a.r.frequency != nullptr ? a.r.frequency[seq] : 0.0f;
    u.pres = a.r.presence != nullptr ? a.r.presence[seq] : 0.0f;
    const float temp = a.r.temperature != nullptr ? a.r.temperature[seq] : 1.0f;
    u.inv_temp = inverse(temp);
    u.bias = biased ? a.r.bias + (size_t)seq * a.r.n_bias : nullptr;
    u.draft = draft != nullptr ? s_draft : nullptr;
    __syncthreads();
    const int marks = s_marks;

    for (int j = j0; j < j1; ++j) {
        const Row<T, TO> now = r;
        const int begin = from, end = to;
        // a marked place that the row's slots hold, or begin - 1
        auto place = [&](int k) {
            const int at = k < marks ? (int)list[k] - kBefore : begin - 1;
            return at >= begin && at < end && (now.ok == nullptr || bit_at(now.ok, c0 + at)) ? at : begin - 1;
        };
        auto value = [&](int at) {
            const float v = to_f32(now.x[at]);
            return apply<GRAD, false>(u, c, at + kBefore, c0 + at, j - j0, GRAD ? to_f32(now.logits[at]) : v, v);
        };
        const int at = place(tid);
        float v = 0.0f;
        if (at >= begin) v = value(at);
#pragma unroll
        for (int k = 0; k < kStreamSlots; ++k)
            s[k].store(now, e + k * kStep, begin, end, c0, u.inv_temp, [](int, int) { return 0u; }, [](int, float x) { return x; });
        if (j + 1 < j1) {
            r = Row<T, TO>(a, (long long)seq * a.per_seq + j + 1, c0);
            load();
        }
        __syncthreads();
        if (at >= begin) now.y[at] = from_f32<TO>(v);
        for (int k = tid + kThreadsP; k < marks; k += kThreadsP) {
            const int more = place(k);
            if (more >= begin) now.y[more] = from_f32<TO>(value(more));
        }
    }
}

// ---------------------------------------------------------------------------

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
        inv_temp = inverse(temp);
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

// The marked places of some rows of a sequence.  Up to the wait this runs before the previous kernel has ended (the one that streams
// the rows, which had waited for its own predecessors before it let this one start), and reads past the first-level cache.
template <typename T, typename TO, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS) k_process_marked(const Args a) {
    extern __shared__ __align__(16) uint32_t smem[];
    const unsigned int block = blockIdx.x;
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
    rows_wait();
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

static int cut(long long n, long long by) { return (int)((n + by - 1) / by); }

template <typename... P, typename... A>
static cudaError_t launch(void (*kernel)(P...), long long ctas, int threads, size_t smem, size_t most, cudaStream_t s, A... args) {
    if (ctas > 2147483647ll) return cudaErrorInvalidValue;
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
    constexpr int VEC = kSlotBytes / (int)sizeof(T);
    const int S = p.R / p.per_seq;
    const bool biased = a.r.bias_ids != nullptr;
    const long long drafts = a.r.draft_ids != nullptr ? a.per_seq - 1ll : 0, tokens = (a.r.history != nullptr ? a.r.history_width : 0) + drafts;
    const long long marks = std::min<long long>(tokens + (biased ? a.r.n_bias : 0), a.V);  // at most
    const int stream_chunks = cut((long long)a.V + VEC - 1, kThreadsP * kStreamSlots * VEC);  // a slot less one may begin before the row
    const long long stream = (long long)p.R * stream_chunks;
    if (marks == 0) return launch(k_process_stream<T, TO, GRAD>, stream, kThreadsP, 0, 0, s, a, stream_chunks, false);

    // The rows of a sequence share a look through its history while the machine is filled.
    auto share = [&](int threads) {
        const long long resident = 152 * 1024 / threads;
        a.rows = std::min(a.per_seq, kMaxRows);
        while (a.rows > 1 && (long long)S * cut(a.per_seq, a.rows) * cut(a.V, threads * 16) < resident) a.rows = (a.rows + 1) / 2;
        a.groups = cut(a.per_seq, a.rows);
        return (long long)S * a.groups;
    };

    if (p.out != p.in && stream <= kOneLaunch && tokens <= kFewTokens) {
        constexpr int kPlaces = kThreadsP * VEC * kStreamSlots, kListed = kPlaces + VEC;
        a.chunks = stream_chunks;
        return launch(k_process_small<T, TO, GRAD>, share(kThreadsP) * a.chunks, kThreadsP,
                      Marks<false>::bytes(kPlaces + kBefore, biased) + (size_t)std::min<long long>(marks, kListed) * 2,
                      Marks<false>::bytes(kPlaces + kBefore, true) + kListed * 2, s, a);
    }
    if (p.out == p.in || stream <= kOneLaunch || (a.per_seq <= 2 && tokens > kLongTokens && marks * kDense > a.V)) {
        auto go = [&](auto kernel, auto wide, int threads) {
            using M = Marks<decltype(wide)::value>;
            const int most = threads * kChunkPerThread;
            const long long units = share(threads);
            a.chunks = (int)std::max<long long>(cut(a.V, most), std::min<long long>(cut(a.V, threads * 4), 152 * 1024 / threads / units));
            a.chunk = cut(cut(a.V, a.chunks), 128) * 128;
            a.chunks = cut(a.V, a.chunk);
            return launch(kernel, units * a.chunks, threads, M::bytes(a.chunk, biased), M::bytes(most, true), s, a);
        };
        if (tokens <= kFewTokens) return go(k_process<T, TO, GRAD, false, kThreadsP>, std::false_type(), kThreadsP);
        return tokens <= kMostNarrow ? go(k_process<T, TO, GRAD, false, 1024>, std::false_type(), 1024)
                                     : go(k_process<T, TO, GRAD, true, 1024>, std::true_type(), 1024);
    }

    const long long units = share(kThreadsP);
    a.hashed = marks <= kHashed;
    a.table = a.hashed ? 128 : kRange;
    while (a.hashed && a.table * 3ll < marks * 4) a.table *= 2;
    a.range = kRange;
    // a few hundred places per CTA while there are SMs left
    a.parts = a.hashed ? (int)std::max<long long>(1, std::min<long long>({marks / 256, 152 / units, 8})) : cut(a.V, kRange);
    const long long sparse = units * a.parts;
    if (sparse > 2147483647ll) return cudaErrorInvalidValue;
    const size_t table = (size_t)a.table * (a.hashed ? kHashBytes : kRangeBytes);
    const cudaError_t e = launch(k_process_stream<T, TO, GRAD>, stream, kThreadsP, 0, 0, s, a, stream_chunks, true);
    if (e != cudaSuccess) return e;
    return marks <= kFew && sparse > kManyCtas
               ? launch(k_process_marked<T, TO, GRAD, kThreadsFew>, sparse, kThreadsFew, table, kMostShort, s, a)
           : marks <= kShort ? launch(k_process_marked<T, TO, GRAD, kThreadsShort>, sparse, kThreadsShort, table, kMostShort, s, a)
                             : launch(k_process_marked<T, TO, GRAD, kThreadsLong>, sparse, kThreadsLong, table, kMostLong, s, a);
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
