// lin_norms.cu -- the launches of the norms around a block (lin_norms.cuh), and
// the sums over their gradient's partial rows.
#include "lin_norms.cuh"

namespace lin {

// (lin_norms_f16.cu, lin_norms_bf16.cu, lin_norms_f32.cu)
extern template cudaError_t launch_block_norms_of<LIN_BINARY16>(const NormsArgs&, int, cudaStream_t);
extern template cudaError_t launch_block_norms_bwd_of<LIN_BINARY16>(const NormsArgs&, int, cudaStream_t);
extern template cudaError_t launch_block_norms_of<LIN_BFLOAT16>(const NormsArgs&, int, cudaStream_t);
extern template cudaError_t launch_block_norms_bwd_of<LIN_BFLOAT16>(const NormsArgs&, int, cudaStream_t);
extern template cudaError_t launch_block_norms_of<LIN_BINARY32>(const NormsArgs&, int, cudaStream_t);
extern template cudaError_t launch_block_norms_bwd_of<LIN_BINARY32>(const NormsArgs&, int, cudaStream_t);

// The sums over the CTAs' partial rows: a CTA per 32 columns and kind, its 32
// warps each a share of the rows, then a fixed-order sum over the warps.
__global__ void __launch_bounds__(1024)
    lin_sum_norm_partials_kernel(const __grid_constant__ NormsArgs a, int rows) {
  __shared__ float part[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, kind = blockIdx.y;
  float sum = 0.0f;
  if (col < a.width)
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) sum += a.partial[((int64_t)r * a.kinds + kind) * a.width + col];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < a.width) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) sum += part[w][lane];
    int k = kind;
    float* out = a.dgate;
    if (a.dn && k-- == 0) out = a.dw_pre;
    else if (a.w_post && k-- == 0) out = a.dw_post;
    out[col] = sum;
  }
}

namespace {

template <typename F>
cudaError_t with_type(int dtype, F&& f) {
  if (dtype == LIN_BINARY32) return f(std::integral_constant<int, LIN_BINARY32>{});
  if (dtype == LIN_BFLOAT16) return f(std::integral_constant<int, LIN_BFLOAT16>{});
  return f(std::integral_constant<int, LIN_BINARY16>{});
}

}  // namespace

cudaError_t launch_block_norms(const NormsArgs& a, int sms, cudaStream_t stream) {
  return with_type(a.dtype, [&](auto t) { return launch_block_norms_of<decltype(t)::value>(a, sms, stream); });
}

int block_norms_bwd_ctas(const NormsArgs& a, int sms) { return bwd_shape(a, sms).ctas; }

cudaError_t launch_block_norms_bwd(const NormsArgs& a, int sms, int ctas, cudaStream_t stream) {
  const cudaError_t e = with_type(a.dtype, [&](auto t) {
    return launch_block_norms_bwd_of<decltype(t)::value>(a, sms, stream);
  });
  if (e != cudaSuccess || a.kinds == 0) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.width + 31) / 32), (unsigned)a.kinds, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lin_sum_norm_partials_kernel, a, ctas);
}

}  // namespace lin
