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
  uint64_t timeout_ns;
  int* status;
  // set at launch: CTAs of a row, parts of a row to each of them, 16-byte
  // units of a part, parts that shared memory holds
  int32_t cluster, segs, tile, slots;
};

// The rows' losses and gradients, then the sum of the losses.
cudaError_t launch_distill(const DistillArgs& a, float* loss_sum, int sms, cudaStream_t stream);

}  // namespace lin
