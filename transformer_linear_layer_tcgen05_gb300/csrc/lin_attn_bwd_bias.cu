// lin_attn_bwd_bias.cu -- attention backward (lin_attn_bwd.cuh) with a distance bias.
#include "lin_attn_bwd.cuh"

namespace lin {
template cudaError_t launch_attn_bwd<kBias>(bool, const AttnBwdMaps&, const AttnBwdArgs&, int, int, int*,
                                        cudaStream_t);
}  // namespace lin
