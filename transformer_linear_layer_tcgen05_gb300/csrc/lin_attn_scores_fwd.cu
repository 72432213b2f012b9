// lin_attn_scores_fwd.cu -- attention forward with a form of the scores
// (lin_attn_fwd.cuh).
#include "lin_attn_fwd.cuh"

namespace lin {

cudaError_t launch_attn_scores_fwd(bool bf16, const AttnFwdMaps& maps, const AttnFwdArgs& args,
                                   int heads_kv, int sequences, cudaStream_t stream) {
  return launch_attn_fwd_kernel<true>(bf16, maps, args, heads_kv, sequences, stream);
}

}  // namespace lin
