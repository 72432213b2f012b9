// lin_attn_fwd_cap_bias.cu -- attention forward (lin_attn_fwd.cuh) with a cap and a distance bias.
#include "lin_attn_fwd.cuh"

namespace lin {
template cudaError_t launch_attn_fwd<kCap | kBias>(bool, const AttnFwdMaps&, const AttnFwdArgs&, int, int,
                                        cudaStream_t);
}  // namespace lin
