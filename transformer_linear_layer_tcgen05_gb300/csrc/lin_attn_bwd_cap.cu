// lin_attn_bwd_cap.cu -- attention backward (lin_attn_bwd.cuh) with a cap of the scores.
#include "lin_attn_bwd.cuh"

namespace lin {
template cudaError_t launch_attn_bwd<kCap>(bool, const AttnBwdMaps&, const AttnBwdArgs&, int, int, int*,
                                        cudaStream_t);
}  // namespace lin
