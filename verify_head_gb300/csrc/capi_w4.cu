// C ABI of the 4-bit rows (quantisation, values, product) and of the processing of logits: host-side argument checks and
// dispatch.  The contract of every entry point: include/verifyhead.h.
#include <cmath>

#include "vh_capi.h"
#include "vh_nvfp4_tiles.h"
#include "vh_row_kernels.h"

using vh::aligned;
using vh::check_device;
using vh::dtype_size;
using vh::known_dtype;
using vh::launch_status;

namespace {

constexpr int kMaxWidth = 65536;
constexpr int kMaxBias = 65535;
constexpr int kMaxRows = vh::kMaxVocab;       // the rows of a block of threads still count in 32 bits
constexpr int kMaxHistory = 1 << 28;          // counts of a token, with two bits beside them

inline bool width_ok(int H) { return H >= 16 && H <= kMaxWidth && H % 16 == 0; }
inline bool scale_ok(float g) { return g > 0.0f && g <= 3.4028234e38f; }

vh_status check_rules(const vh_logits_rules& r, int R, int V, int per_seq) {
    if (per_seq < 1 || R % per_seq != 0) return VH_ERR_SHAPE;
    if (r.history != nullptr && (r.history_width < 0 || r.history_width > kMaxHistory || r.history_stride < r.history_width)) return VH_ERR_SHAPE;
    if ((r.bias_ids == nullptr) != (r.bias == nullptr)) return VH_ERR_NULL;
    if (r.bias_ids != nullptr && (r.n_bias < 0 || r.n_bias > kMaxBias)) return VH_ERR_SHAPE;
    if (r.allowed != nullptr && r.allowed_stride < ((long long)V + 31) / 32) return VH_ERR_SHAPE;
    for (const void* p : {static_cast<const void*>(r.history), static_cast<const void*>(r.history_len),
                          static_cast<const void*>(r.prompt_len), static_cast<const void*>(r.draft_ids),
                          static_cast<const void*>(r.repetition), static_cast<const void*>(r.frequency),
                          static_cast<const void*>(r.presence), static_cast<const void*>(r.temperature),
                          static_cast<const void*>(r.bias_ids), static_cast<const void*>(r.bias),
                          static_cast<const void*>(r.allowed)})
        if (!aligned(p, 4)) return VH_ERR_ALIGN;
    return VH_OK;
}

}  // namespace

extern "C" {

size_t vh_nvfp4_tiles_bytes(int rows, int H) { return rows < 1 || !width_ok(H) ? 0 : vh::nvfp4_tiles_bytes(rows, H); }

vh_status vh_nvfp4_quantize(const void* x, int dtype, int T, int H, int64_t x_stride, float tensor_scale, uint8_t* codes,
                            uint8_t* scales, float* row_scales, void* stream) {
    if (!x || !codes) return VH_ERR_NULL;
    if (!known_dtype(dtype) || T < 1 || T > kMaxRows || !width_ok(H) || x_stride < H) return VH_ERR_SHAPE;
    if (!row_scales && !scale_ok(tensor_scale)) return VH_ERR_SHAPE;
    if (!aligned(x, dtype_size(dtype)) || !aligned(codes, scales ? 8 : 16) || !aligned(row_scales, 4)) return VH_ERR_ALIGN;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    vh::Nvfp4QuantArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.T = T;
    a.H = H;
    a.tensor_scale = tensor_scale;
    a.codes = codes;
    a.scales = scales;
    a.row_scales = row_scales;
    return launch_status(vh::launch_nvfp4_quantize(a, dtype, static_cast<cudaStream_t>(stream)));
}

vh_status vh_nvfp4_tile(const uint8_t* codes, const uint8_t* scales, int V, int H, uint8_t* tiles, size_t tiles_bytes,
                        void* stream) {
    if (!codes || !scales || !tiles) return VH_ERR_NULL;
    if (V < 1 || V > kMaxRows || !width_ok(H)) return VH_ERR_SHAPE;
    if (!aligned(codes, 8) || !aligned(tiles, 16)) return VH_ERR_ALIGN;
    if (tiles_bytes < vh_nvfp4_tiles_bytes(V, H)) return VH_ERR_WORKSPACE;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    return launch_status(vh::launch_nvfp4_tile(codes, scales, V, H, tiles, static_cast<cudaStream_t>(stream)));
}

vh_status vh_nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int T, int H, float tensor_scale,
                              const float* row_scales, int dtype, void* y, int64_t y_stride, void* stream) {
    if (!codes || !y) return VH_ERR_NULL;
    if (!known_dtype(dtype) || T < 1 || T > kMaxRows || !width_ok(H) || y_stride < H) return VH_ERR_SHAPE;
    if (!row_scales && !(std::fabs(tensor_scale) <= 3.4028234e38f)) return VH_ERR_SHAPE;
    if (!aligned(codes, scales ? 8 : 16) || !aligned(row_scales, 4) || !aligned(y, dtype_size(dtype))) return VH_ERR_ALIGN;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    vh::Nvfp4DequantArgs a{};
    a.codes = codes;
    a.scales = scales;
    a.T = T;
    a.H = H;
    a.tensor_scale = tensor_scale;
    a.row_scales = row_scales;
    a.y = y;
    a.y_stride = y_stride;
    return launch_status(vh::launch_nvfp4_dequantize(a, dtype, static_cast<cudaStream_t>(stream)));
}

vh_status vh_nvfp4_matmul(const uint8_t* x, float x_scale, const float* x_scales, const uint8_t* w, float w_scale,
                          const float* w_scales, int T, int V, int H, int dtype, void* y, int64_t y_stride, void* stream) {
    if (!x || !w || !y) return VH_ERR_NULL;
    if (!known_dtype(dtype) || T < 1 || V < 1 || V > vh::kMaxVocab || T > kMaxRows || !width_ok(H) || y_stride < V)
        return VH_ERR_SHAPE;
    if ((!x_scales && !(std::fabs(x_scale) <= 3.4028234e38f)) || (!w_scales && !(std::fabs(w_scale) <= 3.4028234e38f)))
        return VH_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
        !aligned(y, dtype_size(dtype)))
        return VH_ERR_ALIGN;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    vh::Nvfp4MatmulArgs a{};
    a.x = x;
    a.w = w;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.x_scales = x_scales;
    a.w_scales = w_scales;
    a.T = T;
    a.V = V;
    a.H = H;
    a.y = y;
    a.y_stride = y_stride;
    return launch_status(vh::launch_nvfp4_matmul(a, dtype, static_cast<cudaStream_t>(stream)));
}

vh_status vh_logits_process(const void* logits, int dtype, int R, int V, int64_t stride, int rows_per_seq,
                            const vh_logits_rules* rules, void* out, int out_dtype, int64_t out_stride, void* stream) {
    if (!logits || !rules || !out) return VH_ERR_NULL;
    if (!known_dtype(dtype) || (out_dtype != dtype && out_dtype != VH_F32) || R < 1 || V < 1 || V > vh::kMaxVocab ||
        stride < V || out_stride < V)
        return VH_ERR_SHAPE;
    const vh_status rt = check_rules(*rules, R, V, rows_per_seq);
    if (rt != VH_OK) return rt;
    if (out == logits && (out_dtype != dtype || (R > 1 && out_stride != stride))) return VH_ERR_SHAPE;
    if (!aligned(logits, dtype_size(dtype)) || !aligned(out, dtype_size(out_dtype))) return VH_ERR_ALIGN;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    vh::ProcessArgs a{};
    a.in = logits;
    a.logits = logits;
    a.out = out;
    a.in_stride = a.logits_stride = stride;
    a.out_stride = out_stride;
    a.R = R;
    a.V = V;
    a.per_seq = rows_per_seq;
    a.rules = *rules;
    return launch_status(vh::launch_logits_process(a, dtype, out_dtype, static_cast<cudaStream_t>(stream)));
}

vh_status vh_logits_process_grad(const void* dout, const void* logits, int dtype, int R, int V, int64_t dout_stride,
                                 int64_t logits_stride, int rows_per_seq, const vh_logits_rules* rules, void* dlogits,
                                 int64_t dlogits_stride, void* stream) {
    if (!dout || !logits || !rules || !dlogits) return VH_ERR_NULL;
    if (!known_dtype(dtype) || R < 1 || V < 1 || V > vh::kMaxVocab || dout_stride < V || logits_stride < V ||
        dlogits_stride < V)
        return VH_ERR_SHAPE;
    const vh_status rt = check_rules(*rules, R, V, rows_per_seq);
    if (rt != VH_OK) return rt;
    if (dlogits == logits || (dlogits == dout && R > 1 && dlogits_stride != dout_stride)) return VH_ERR_SHAPE;
    const uintptr_t sz = dtype_size(dtype);
    if (!aligned(dout, sz) || !aligned(logits, sz) || !aligned(dlogits, sz)) return VH_ERR_ALIGN;
    const vh_status st = check_device();
    if (st != VH_OK) return st;
    vh::ProcessArgs a{};
    a.in = dout;
    a.logits = logits;
    a.out = dlogits;
    a.in_stride = dout_stride;
    a.logits_stride = logits_stride;
    a.out_stride = dlogits_stride;
    a.R = R;
    a.V = V;
    a.per_seq = rows_per_seq;
    a.rules = *rules;
    return launch_status(vh::launch_logits_process_grad(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
