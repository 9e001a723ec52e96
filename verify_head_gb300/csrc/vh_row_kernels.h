// Launchers of the operators on both sides of the head (add_rmsnorm.cu, logprobs.cu, head_logprobs.cu).
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

}  // namespace vh
