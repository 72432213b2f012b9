// lin_attn_fwd.cu -- attention forward without a form of the scores
// (lin_attn_fwd.cuh), and the joining of parts of the keys.
#include "lin_attn_fwd.cuh"

namespace lin {

// O and the log-sum-exps from the parts': weights 2^(L_p - L) of their rows,
// added in order. A CTA per 32 rows of a sequence and head, eight entries to
// a thread.
template <bool BF16>
__global__ void __launch_bounds__(256)
    lin_attn_join_parts_kernel(const __grid_constant__ AttnFwdArgs args) {
  const AttnArgs& a = args.s;
  const int h = blockIdx.x;
  const SeqRange r = seq_range(a.cu_q, blockIdx.z, a.tokens_q, a.max_q);
  const int groups = a.dim / 8;
  pdl_wait();
  for (int k = threadIdx.x; k < 32 * groups; k += 256) {
    const int i = blockIdx.y * 32 + k / groups, col = k % groups * 8;
    if (i >= r.len) continue;
    const int64_t token = (int64_t)r.start + i;
    const int row_at = (int)blockIdx.z * a.max_q + i;
    if (!q_row_ok(a, token, h) || !dcheck(row_at < args.part_rows, a.status, CHK_PART, row_at)) continue;
    const float* ls = args.lse_part + h * args.part_rows + row_at;
    const int ls_step = a.heads_q * args.part_rows;
    float top = -INFINITY;
    for (int q = 0; q < args.parts; ++q) top = fmaxf(top, ls[q * ls_step]);
    const float shift = top == -INFINITY ? 0.0f : top;   // (a row without a key)
    const float* p = args.o_part + (row_at * a.heads_q + h) * a.dim + col;
    const int step = ls_step * a.dim;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    float total = 0.0f;
    for (int q = 0; q < args.parts; ++q) {
      const float w = ex2_approx((ls[q * ls_step] - shift) * kLog2E);
      const float4 u = __ldcs(reinterpret_cast<const float4*>(p + q * step));
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p + q * step) + 1);
      total += w;
      x = make_float4(fmaf(w, u.x, x.x), fmaf(w, u.y, x.y), fmaf(w, u.z, x.z), fmaf(w, u.w, x.w));
      y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    store16(args.o.p + token * args.o.token_stride + (int64_t)h * args.o.head_stride + col,
            pack16<BF16>(x.x * inv, x.y * inv), pack16<BF16>(x.z * inv, x.w * inv),
            pack16<BF16>(y.x * inv, y.y * inv), pack16<BF16>(y.z * inv, y.w * inv));
    if (col == 0) args.lse[(int64_t)h * a.tokens_q + token] = top + logf(total);
  }
}

cudaError_t launch_attn_join_parts(bool bf16, const AttnFwdArgs& args, int heads, int sequences,
                                   cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)heads, (unsigned)((args.s.max_q + 31) / 32), (unsigned)sequences);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, lin_attn_join_parts_kernel<true>, args)
              : cudaLaunchKernelEx(&cfg, lin_attn_join_parts_kernel<false>, args);
}

template cudaError_t launch_attn_fwd<kNoForm>(bool, const AttnFwdMaps&, const AttnFwdArgs&, int, int,
                                              cudaStream_t);

}  // namespace lin
