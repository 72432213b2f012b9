// lin_rope.h -- launch interface of the norm and rotation kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "lin_attn.h"

namespace lin {

struct RopeArgs {
  const float* x;         // [tokens][(hq + 2 hk) dim]
  const float *wq, *wk;   // [dim]
  const float *cos, *sin; // [table_rows][rot / 2]
  const int32_t* pos;     // [tokens], null: 0, 1, 2, ...
  int64_t tokens, table_rows;
  int32_t hq, hk, dim, rot;
  float eps;
  HeadsPtr q, k, v;       // written (forward) or read (gradient)
  float* dx;              // gradient: as x
  float *dwq, *dwk;       // gradient: [dim]
  float* partial;         // gradient: [CTAs][dim]
  int32_t q_ctas;         // gradient: CTAs that take the query heads (set with their number)
  int* status;            // device status record (checked build)
};

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool inter, bool bf16, cudaStream_t stream);
// CTAs of the gradient's kernel (rows of its partial sums); sets a.q_ctas.
int qk_norm_rope_bwd_ctas(RopeArgs& a, int sms);
cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, bool inter, bool bf16, int ctas,
                                    cudaStream_t stream);

}  // namespace lin
