// lin_attn_bwd.cu -- attention backward without a form of the scores
// (lin_attn_bwd.cuh), the sums of parts, and how many parts there are.
#include "lin_attn_bwd.cuh"

namespace lin {

// ---------------------------------------------------------------- parts

// Gradients from their parts' f32 sums [part][row][head][dim], added in
// order: one, or (dK and dV) two of the same shape in one launch. A CTA per 32
// rows of a sequence and head, eight entries to a thread.
struct SumParts {   // (step: entries of a part)
  const int32_t* cu;
  int* status;
  int32_t tokens, most, dim, parts, sequences;
  int64_t step;
  const float* part[2];
  HeadsPtr out[2];
};
template <bool BF16>
__global__ void __launch_bounds__(256)
    lin_attn_sum_parts_kernel(const __grid_constant__ SumParts a) {
  const int h = blockIdx.x, heads = gridDim.x;
  const int which = blockIdx.z >= a.sequences;
  const int b = blockIdx.z - which * a.sequences;
  const SeqRange r = seq_range(a.cu, b, a.tokens, a.most);
  const HeadsPtr& out = a.out[which];
  const int groups = a.dim / 8;
  pdl_wait();
  for (int k = threadIdx.x; k < 32 * groups; k += 256) {
    const int i = blockIdx.y * 32 + k / groups, col = k % groups * 8;
    if (i >= r.len) continue;
    const int64_t token = (int64_t)r.start + i;
    if (!dcheck(token < a.tokens && i < a.most, a.status, CHK_GLOBAL, token)) continue;
    const float* p = a.part[which] + ((b * a.most + i) * heads + h) * a.dim + col;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int q = 0; q < a.parts; ++q, p += a.step) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(p));
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    store16(out.p + token * out.token_stride + (int64_t)h * out.head_stride + col,
            pack16<BF16>(x.x, x.y), pack16<BF16>(x.z, x.w), pack16<BF16>(y.x, y.y),
            pack16<BF16>(y.z, y.w));
  }
}

// Parts of a launch of `ctas` CTAs whose longest runs over `rows` rows: as
// many as give every SM a CTA, while each keeps at least 256 rows, but not
// below 1024 rows, where the kernel that joins them costs what the shorter
// loops save, and not above 16, where its reading does (forward and backward,
// one head, us: 512 rows 8.1 and 18.8 whole, 9.8 and 18.9 in parts; 768: 9.7
// and 21.7, 10.3 and 19.7; 1024: 15.5 and 33.7, 13.4 and 28.6; 2000: 28.6 and
// 55, 17.3 and 33.3; 64 queries over 8000 keys, four heads, in 15 parts 15.5
// and 19.8, in 31 17.3 and 21.1).
int attn_parts(int64_t ctas, int64_t rows, int sms) {
  if (rows < 1024 || ctas < 1) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>({sms / ctas, rows / 256, 16}));
}

cudaError_t launch_attn_sum_parts(bool bf16, const AttnBwdArgs& args, int heads_kv, int sequences,
                                  int* kernels, cudaStream_t stream) {
  const unsigned hq = (unsigned)(heads_kv * args.s.group), hk = (unsigned)heads_kv;
  const unsigned seqs = (unsigned)sequences;
  auto sum = [&](const SumParts& p, unsigned heads, unsigned count) {
    const dim3 grid(heads, (unsigned)((p.most + 31) / 32), seqs * count);
    if (grid.y == 0) return cudaSuccess;
    ++*kernels;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, lin_attn_sum_parts_kernel<true>, p)
                : cudaLaunchKernelEx(&cfg, lin_attn_sum_parts_kernel<false>, p);
  };
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess && args.q_parts > 1)
    e = sum(SumParts{args.s.cu_q, args.s.status, args.s.tokens_q, args.s.max_q, args.s.dim, args.q_parts, sequences,
                     (int64_t)args.q_part_rows * (int)hq * args.s.dim, {args.dq_part, nullptr}, {args.dq, args.dq}},
            hq, 1);
  if (e == cudaSuccess && args.k_parts > 1)
    e = sum(SumParts{args.s.cu_k, args.s.status, args.s.tokens_k, args.s.max_k, args.s.dim, args.k_parts, sequences,
                     (int64_t)args.k_part_rows * (int)hk * args.s.dim, {args.dk_part, args.dv_part}, {args.dk, args.dv}},
            hk, 2);
  return e;
}

template cudaError_t launch_attn_bwd<kNoForm>(bool, const AttnBwdMaps&, const AttnBwdArgs&, int, int, int*,
                                              cudaStream_t);

}  // namespace lin
