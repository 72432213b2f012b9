// lin_attn_scores_bwd.cu -- attention backward with a form of the scores
// (lin_attn_bwd.cuh).
#include "lin_attn_bwd.cuh"

namespace lin {

cudaError_t launch_attn_scores_bwd(bool bf16, const AttnBwdMaps& maps, const AttnBwdArgs& args,
                                   int heads_kv, int sequences, int* kernels, cudaStream_t stream) {
  return launch_attn_bwd_kernels<true>(bf16, maps, args, heads_kv, sequences, kernels, stream);
}

}  // namespace lin
