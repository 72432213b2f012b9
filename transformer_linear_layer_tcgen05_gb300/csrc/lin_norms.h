// lin_norms.h -- launch interface of the norms around a block.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lin {

enum NormGate : int { NORM_GATE_NONE = 0, NORM_GATE_CHANNEL, NORM_GATE_TOKEN, NORM_GATE_FULL };
constexpr int kNormMostWidth = 8192;

struct NormsArgs {
  const float* x;        // [tokens][width] (gradient: h)
  const void* y;         // the block's output, null: none
  const float* gate;     // [width], [tokens] or [tokens][width] by `form`
  const float *w_post, *w_pre;   // [width], null: no such norm
  float* h;              // null: not written
  void* n;
  const float* dh;       // gradient: null: none
  const void* dn;        // null: none (no norm behind)
  float* dx;
  void* dy;
  float* dgate;          // channel: from the partial sums; token, full: written by the rows
  float *dw_post, *dw_pre;
  float* partial;        // [CTAs][kinds][width]
  int32_t kinds;         // sums over the tokens: of w_pre, of w_post, of the gate (those there are)
  int64_t tokens;
  int32_t width, form, dtype;    // dtype: lin_dtype of y, n, dy, dn
  float residual_scale, block_scale, eps;
  int* status;
};

cudaError_t launch_block_norms(const NormsArgs& a, int sms, cudaStream_t stream);
// CTAs of the gradient's kernel (rows of its partial sums).
int block_norms_bwd_ctas(const NormsArgs& a, int sms);
// The gradient, and, where a.kinds > 0, the sums over its CTAs.
cudaError_t launch_block_norms_bwd(const NormsArgs& a, int sms, int ctas, cudaStream_t stream);
// The same for the type T of the block's tensors (its kernels alone).
template <int T>
cudaError_t launch_block_norms_of(const NormsArgs& a, int sms, cudaStream_t stream);
template <int T>
cudaError_t launch_block_norms_bwd_of(const NormsArgs& a, int sms, cudaStream_t stream);

}  // namespace lin
