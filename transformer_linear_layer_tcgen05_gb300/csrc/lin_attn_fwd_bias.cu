// lin_attn_fwd_bias.cu -- attention forward (lin_attn_fwd.cuh) with a distance bias.
#include "lin_attn_fwd.cuh"

namespace lin {
template cudaError_t launch_attn_fwd<kBias>(bool, const AttnFwdMaps&, const AttnFwdArgs&, int, int,
                                        cudaStream_t);
}  // namespace lin
