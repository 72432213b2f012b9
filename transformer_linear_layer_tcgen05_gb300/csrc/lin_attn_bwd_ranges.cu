// lin_attn_bwd_ranges.cu -- attention backward (lin_attn_bwd.cuh) with ranges of keys alone.
#include "lin_attn_bwd.cuh"

namespace lin {
template cudaError_t launch_attn_bwd<0>(bool, const AttnBwdMaps&, const AttnBwdArgs&, int, int, int*,
                                        cudaStream_t);
}  // namespace lin
