// lin_attn_fwd_cap.cu -- attention forward (lin_attn_fwd.cuh) with a cap of the scores.
#include "lin_attn_fwd.cuh"

namespace lin {
template cudaError_t launch_attn_fwd<kCap>(bool, const AttnFwdMaps&, const AttnFwdArgs&, int, int,
                                        cudaStream_t);
}  // namespace lin
