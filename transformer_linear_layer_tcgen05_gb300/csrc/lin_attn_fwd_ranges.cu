// lin_attn_fwd_ranges.cu -- attention forward (lin_attn_fwd.cuh) with ranges of keys alone.
#include "lin_attn_fwd.cuh"

namespace lin {
template cudaError_t launch_attn_fwd<0>(bool, const AttnFwdMaps&, const AttnFwdArgs&, int, int,
                                        cudaStream_t);
}  // namespace lin
