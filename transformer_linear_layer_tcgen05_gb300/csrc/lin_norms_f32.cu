// lin_norms_f32.cu -- the norms around a block (lin_norms.cuh) of binary32 outputs.
#include "lin_norms.cuh"

namespace lin {
template cudaError_t launch_block_norms_of<LIN_BINARY32>(const NormsArgs&, int, cudaStream_t);
template cudaError_t launch_block_norms_bwd_of<LIN_BINARY32>(const NormsArgs&, int, cudaStream_t);
}  // namespace lin
