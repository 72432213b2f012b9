// lin_adamw.h -- launch interface of the AdamW step over many tensors.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lin {

constexpr int kAdamwBlock = 256;      // entries of a tensor that share a scale (8-bit states)
constexpr int kAdamwMost = 384;       // tensors of a launch (its parameters: 64 bytes and 4 each)

struct AdamwTensor {
  float* p;
  const float* g;
  void *m, *v;               // f32, or e4m3 codes
  float *m_scale, *v_scale;  // of each block (8-bit states)
  uint16_t* w16;             // binary16 copy of p (null: none)
  int64_t n : 63;
  uint64_t wide : 1;         // every pointer allows the widest accesses
};

struct AdamwArgs {
  int32_t tensors;
  uint32_t blocks;           // of all tensors
  float beta1, beta1_rest, beta2, beta2_rest, eps;
  // the step's factors: of p, of m / denominator, of the root of v
  float keep, rate, root;
  // or, with device values (either may be null), what they are made from
  const float* lr;
  const int32_t* step;
  float lr_value, decay, log_beta1, log_beta2;
  const float* grad_scale;   // (null: 1)
  int* status;
};

// A launch's tensors and, for each, the blocks before it.
template <int N>
struct AdamwList {
  AdamwTensor t[N];
  uint32_t first[N];
};

// `tensors` has a.tensors entries, `first` their first blocks.
cudaError_t launch_adamw(const AdamwArgs& a, const AdamwTensor* tensors, const uint32_t* first,
                         bool bits8, int sms, cudaStream_t stream);

}  // namespace lin
