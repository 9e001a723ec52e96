// Launchers of the operators on both sides of the head (add_rmsnorm.cu, logprobs.cu, head_logprobs.cu, logits_process.cu)
// and of those on 4-bit rows (nvfp4_rows.cu, nvfp4_matmul.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/verifyhead.h"

namespace vh {

// Residual addition and RMS norm of T rows of width H (add_rmsnorm.cu);
// r, h, w may be null; strides in elements.
struct NormArgs {
    const void *x, *r, *w;
    void *h, *y;
    float* scales;  // 8-bit outputs: one per row
    long long x_stride, r_stride, h_stride, y_stride;
    int T, H;
    int w32;        // w is fp32 (else the rows' type)
    int out;        // vh_norm_out
    float eps, w_offset, inv_h;
};
cudaError_t launch_add_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s);

// Its gradient; dh may be null.  part: fp32 [norm_grad_parts(T)][norm_grad_pitch(H)],
// or null when dw is not wanted.
struct NormGradArgs {
    const void *dy, *h, *w, *dh;
    void* dx;
    float* part;
    int part_pitch;  // set by the launcher, as is:
    bool summed;     // the shares' sum is left to a second kernel
    long long dy_stride, h_stride, dh_stride, dx_stride;
    int T, H;
    int w32;
    float eps, w_offset, inv_h;
};
constexpr int kNormGradParts = 608;  // CTAs that share the tokens, at most: four per SM
int norm_grad_parts(int T);
inline size_t norm_grad_pitch(int H) { return H % 8 == 0 ? H : ((size_t)H + 14) / 8 * 8; }  // odd widths by slots
cudaError_t launch_add_rmsnorm_grad(const NormGradArgs& a, int dtype, float* dweight, cudaStream_t s);

// Log probabilities from logits (logprobs.cu).
constexpr int kMaxTop = 32;  // alternatives per row (one per lane)
struct LogprobArgs {
    const void* logits;
    long long stride;
    int R, V, top_n;
    const int32_t* tokens;
    float *logprob, *entropy, *lse;  // each may be null
    int32_t* top_ids;
    float* top_logprobs;
    void* ws;
};
size_t logits_logprobs_ws_bytes(int R, int V, int top_n);
cudaError_t launch_logits_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s);

struct LogprobGradArgs {
    const void* logits;
    void* dlogits;
    long long stride, d_stride;
    int R, V;
    const int32_t* tokens;
    const float *lse, *entropy, *g_logprob, *g_entropy;  // entropy and either gradient may be null
};
cudaError_t launch_logits_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s);

// Log probabilities of hidden rows against a head (head_logprobs.cu), H % 8 == 0.
struct HeadLogprobArgs {
    const uint16_t *x, *W;
    int R, H, V, top_n;
    const int32_t* tokens;
    float *logprob, *entropy, *lse;
    int32_t* top_ids;
    float* top_logprobs;
    void* ws;
};
size_t head_logprobs_ws_bytes(int R, int V, int top_n);
cudaError_t launch_head_logprobs(const HeadLogprobArgs& a, cudaStream_t s);

// Rows to 4 bits (nvfp4_rows.cu), H % 16 == 0.  scales null: `codes` is the tiled layout (vh_nvfp4_tiles.h).
struct Nvfp4QuantArgs {
    const void* x;
    long long x_stride;
    int T, H;
    float tensor_scale;  // when row_scales is null
    uint8_t *codes, *scales;
    float* row_scales;
};
cudaError_t launch_nvfp4_quantize(const Nvfp4QuantArgs& a, int dtype, cudaStream_t s);

struct Nvfp4DequantArgs {
    const uint8_t *codes, *scales;
    int T, H;
    float tensor_scale;
    const float* row_scales;
    void* y;
    long long y_stride;
};
cudaError_t launch_nvfp4_dequantize(const Nvfp4DequantArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_nvfp4_tile(const uint8_t* codes, const uint8_t* scales, int V, int H, uint8_t* tiles, cudaStream_t s);

// Product of two tiled 4-bit matrices (nvfp4_matmul.cu): y[t][v] = x_scale(t) w_scale(v) sum_h X[t,h] W[v,h].
struct Nvfp4MatmulArgs {
    const uint8_t *x, *w;
    float x_scale, w_scale;               // when the arrays are null
    const float *x_scales, *w_scales;
    int T, V, H;
    void* y;
    long long y_stride;
};
cudaError_t launch_nvfp4_matmul(const Nvfp4MatmulArgs& a, int dtype, cudaStream_t s);

// Processing of logits (logits_process.cu).  `in` are the logits, or the gradient of the processed ones; `logits` is
// read by the gradient alone.
struct ProcessArgs {
    const void *in, *logits;
    void* out;
    long long in_stride, logits_stride, out_stride;
    int R, V, per_seq;
    vh_logits_rules rules;
};
cudaError_t launch_logits_process(const ProcessArgs& a, int dtype, int out_dtype, cudaStream_t s);
cudaError_t launch_logits_process_grad(const ProcessArgs& a, int dtype, cudaStream_t s);

}  // namespace vh
