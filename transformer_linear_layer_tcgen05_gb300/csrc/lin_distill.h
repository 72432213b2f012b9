// lin_distill.h -- launch interface of the distillation loss.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lin {

struct DistillArgs {
  const float* logits;    // [M][ld]
  const int32_t* ids;     // [M][K]
  const float* teacher;   // [M][K]
  float* dlogits;         // [M][ldd], null: the losses alone
  float* losses;          // [M]
  int64_t M, V, ld, ldd;
  int32_t K;
  float tau, inv_norm;
  int32_t cluster, tile;  // CTAs of a row and the logits of each (set at launch)
};

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream);

}  // namespace lin
