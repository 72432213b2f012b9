// lin_rope.cu -- norms of the query and key heads and the position rotation
// in one pass, from the QKV projection's f32 rows to the 16-bit heads that
// attention reads, and the gradient:
//   n = x / sqrt(mean x^2 + eps),  y = turn(n w),  v: rounded only
//   dn = turn^-1(dy),  dw = sum dn n,  g = dn w,
//   dx = (g - n mean(g n)) / sqrt(mean x^2 + eps)
// turn() rotates the pairs (i, i + rot/2), or (2i, 2i + 1), of the first rot
// entries by the token's row of a cosine and a sine table.
//
// Bound by memory: a head's entries are held in registers between the norm
// and the rotation, so each is read and written once. A group of G lanes (the
// power of two that covers dim / 8) has a head, eight entries to a lane: both
// entries of four pairs, so that the rotation stays within the lane and the
// norm is a shuffle tree over the group. A group takes several heads of one
// token: the loads of all of them are in flight together, and the token's
// angles are read once for them.
#include "lin_common.cuh"
#include "lin_rope.h"

#include <algorithm>
#include <cuda_bf16.h>

namespace lin {

namespace {

constexpr int kRopeThreads = 256;
// Heads of a group's turn and CTAs whose registers an SM holds: the bytes in
// flight grow with either, and the registers allow one or the other. Two
// heads in 48 warps an SM (forward) and 32 (gradient) measured best; 16384
// tokens of 32 + 2 x 8 heads of 128, forward and gradient, us: two heads x 6
// and 4 CTAs 103 and 170 (5.9 and 6.0 TB/s), four heads x 3 and 2 CTAs 132
// and 208, one head x 8 and 8 CTAs 120 and 261.
constexpr int kFwdHeads = 2, kFwdCtas = 6;
constexpr int kBwdHeads = 2, kBwdCtas = 4;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_half2(lo, hi);
  }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's place in its head: entries o0 .. o0 + 3 and o1 .. o1 + 3. Lanes of
// the rotated part have four pairs (halves: entry i of the first run with
// entry i of the second; interleaved: neighbours).
struct Place {
  int o0, o1, pair;
  bool on, turned;
};
template <bool INTER>
__device__ __forceinline__ Place place(int t, int dim, int rot) {
  Place p;
  p.on = t * 8 < dim;
  p.turned = t * 8 < rot;
  p.pair = t * 4;
  const bool split = !INTER && p.turned;
  p.o0 = split ? t * 4 : t * 8;
  p.o1 = split ? rot / 2 + t * 4 : t * 8 + 4;
  return p;
}

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight load8f(const float* p, const Place& at) {
  const float4 a = *reinterpret_cast<const float4*>(p + at.o0);
  const float4 b = *reinterpret_cast<const float4*>(p + at.o1);
  return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Four pairs turned by the angles (c, s); BACK by the opposite ones.
template <bool INTER, bool BACK>
__device__ __forceinline__ void turn(Eight& x, const float4& c, const float4& s) {
  const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& a = x.v[INTER ? 2 * i : i];
    float& b = x.v[INTER ? 2 * i + 1 : 4 + i];
    const float si = BACK ? -sn[i] : sn[i];
    const float na = a * cs[i] - b * si, nb = a * si + b * cs[i];
    a = na;
    b = nb;
  }
}

// A position held inside the tables.
__device__ __forceinline__ int64_t held(const RopeArgs& a, int64_t p) {
  return min(max(p, (int64_t)0), (int64_t)a.table_rows - 1);
}
// Row of the tables for token t: its position.
__device__ __forceinline__ int64_t table_row(const RopeArgs& a, int64_t t) {
  return held(a, a.pos ? (int64_t)a.pos[t] : t);
}

// Checked build: head `head` of token t inside the tensors; a lane's entries
// inside the head; four angles inside the tables.
__device__ __forceinline__ bool head_ok(const RopeArgs& a, int64_t t, int head, const Place& at) {
  return dcheck(t >= 0 && t < a.tokens && head >= 0 && head < a.hq + 2 * a.hk, a.status, CHK_GLOBAL, t) &&
         dcheck(at.o0 + 4 <= a.dim && at.o1 + 4 <= a.dim, a.status, CHK_GLOBAL, at.o1);
}
__device__ __forceinline__ bool angles_ok(const RopeArgs& a, int64_t row) {
  return dcheck(row >= 0 && row + 4 <= a.table_rows * (a.rot / 2), a.status, CHK_GLOBAL, row);
}

// The angles of token t for a lane's four pairs. AXES: each pair goes by the
// position of its own axis (all positions of the token are read at once, with
// the pairs' axes); four pairs of one axis are read together.
template <bool AXES>
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t t, int pair, float4& c, float4& s) {
  const int half = a.rot / 2;
  if constexpr (!AXES) {
    const int64_t row = table_row(a, t) * half + pair;
    if (angles_ok(a, row)) {
      c = *reinterpret_cast<const float4*>(a.cos + row);
      s = *reinterpret_cast<const float4*>(a.sin + row);
    }
  } else {
    int32_t p[kMostAxes];
#pragma unroll
    for (int k = 0; k < kMostAxes; ++k) p[k] = k < a.axes ? a.pos[k * a.tokens + t] : 0;
    const int4 q = *reinterpret_cast<const int4*>(a.axis + pair);
    int ax[4] = {q.x, q.y, q.z, q.w};
    int64_t row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ax[i] = min(max(ax[i], 0), a.axes - 1);
      int32_t at = p[0];
#pragma unroll
      for (int k = 1; k < kMostAxes; ++k) at = ax[i] == k ? p[k] : at;
      row[i] = held(a, at) * half + pair;
    }
    if (!angles_ok(a, row[0]) || !angles_ok(a, row[1]) || !angles_ok(a, row[2]) || !angles_ok(a, row[3]))
      return;
    if (ax[0] == ax[1] && ax[0] == ax[2] && ax[0] == ax[3]) {
      c = *reinterpret_cast<const float4*>(a.cos + row[0]);
      s = *reinterpret_cast<const float4*>(a.sin + row[0]);
    } else {
      c = make_float4(a.cos[row[0]], a.cos[row[1] + 1], a.cos[row[2] + 2], a.cos[row[3] + 3]);
      s = make_float4(a.sin[row[0]], a.sin[row[1] + 1], a.sin[row[2] + 2], a.sin[row[3] + 3]);
    }
  }
}

// The 16-bit head `head` (of q, k and v in a row) of token t.
__device__ __forceinline__ uint16_t* head16(const RopeArgs& a, int64_t t, int head) {
  if (head < a.hq) return a.q.p + t * a.q.token_stride + (int64_t)head * a.q.head_stride;
  head -= a.hq;
  if (head < a.hk) return a.k.p + t * a.k.token_stride + (int64_t)head * a.k.head_stride;
  head -= a.hk;
  return a.v.p + t * a.v.token_stride + (int64_t)head * a.v.head_stride;
}

}  // namespace

template <int G, bool INTER, bool BF16, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, kFwdCtas)
    lin_qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int GROUPS = kRopeThreads / G;
  const int heads = a.hq + 2 * a.hk;
  const unsigned chunks = (unsigned)((heads + kFwdHeads - 1) / kFwdHeads);
  const int64_t t = (int64_t)(blockIdx.x / chunks) * GROUPS + threadIdx.x / G;
  // (a warp's shuffles need all of its lanes: groups behind the last token stay)
  const int h0 = t < a.tokens ? (int)(blockIdx.x % chunks) * kFwdHeads : heads;
  const Place at = place<INTER>(threadIdx.x % G, a.dim, a.rot);
  Eight x[kFwdHeads];
#pragma unroll
  for (int i = 0; i < kFwdHeads; ++i)
    x[i] = at.on && h0 + i < heads && head_ok(a, t, h0 + i, at)
               ? load8f(a.x + (t * heads + h0 + i) * a.dim, at)
               : Eight{};
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at.on && at.turned && h0 < heads) angles<AXES>(a, t, at.pair, c, s);
  float r[kFwdHeads];
#pragma unroll
  for (int i = 0; i < kFwdHeads; ++i) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[i].v[e], x[i].v[e], ss);
    r[i] = rsqrtf(group_sum<G>(ss) / (float)a.dim + a.eps);
  }
#pragma unroll
  for (int i = 0; i < kFwdHeads; ++i) {
    const int h = h0 + i;
    if (!at.on || h >= heads || !head_ok(a, t, h, at)) continue;
    if (h < a.hq + a.hk) {
      const Eight w = load8f(h < a.hq ? a.wq : a.wk, at);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i].v[e] *= r[i] * w.v[e];
      if (at.turned) turn<INTER, false>(x[i], c, s);
    }
    uint16_t* y = head16(a, t, h);
    const float* v = x[i].v;
    *reinterpret_cast<uint2*>(y + at.o0) = make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
    *reinterpret_cast<uint2*>(y + at.o1) = make_uint2(pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
  }
}

// The gradient. The CTAs below a.q_ctas take the query heads, the others the
// key and the value heads, so that a lane keeps one weight's gradient. Each
// group walks over (token, heads) items with a fixed stride; the CTA's groups
// are added in a fixed order and leave one partial row, and a second kernel
// adds those.
template <int G, bool INTER, bool BF16, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, kBwdCtas)
    lin_qk_norm_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int GROUPS = kRopeThreads / G;
  __shared__ float part[GROUPS][G * 8 + 4];
  const int heads = a.hq + 2 * a.hk;
  const bool isq = (int)blockIdx.x < a.q_ctas;
  const int h_lo = isq ? 0 : a.hq, h_hi = isq ? a.hq : heads;
  const int cta = isq ? (int)blockIdx.x : (int)blockIdx.x - a.q_ctas;
  const int ctas = isq ? a.q_ctas : (int)gridDim.x - a.q_ctas;
  const int chunks = (h_hi - h_lo + kBwdHeads - 1) / kBwdHeads;
  const int group = threadIdx.x / G;
  const Place at = place<INTER>(threadIdx.x % G, a.dim, a.rot);
  const Eight w = at.on ? load8f(isq ? a.wq : a.wk, at) : Eight{};
  const float inv_dim = 1.0f / (float)a.dim;
  Eight dw{};
  // items token * chunks + chunk, from cta * GROUPS + group in steps of ctas * GROUPS
  const int step = ctas * GROUPS, step_t = step / chunks, step_c = step % chunks;
  int64_t t = (cta * GROUPS + group) / chunks;
  int chunk = (cta * GROUPS + group) % chunks;
  // (all groups of a warp go round together: the shuffles need its lanes)
  for (; __any_sync(0xffffffffu, t < a.tokens); t += step_t) {
    const int h0 = t < a.tokens ? h_lo + chunk * kBwdHeads : h_hi;
    Eight x[kBwdHeads], g[kBwdHeads];
    const float* xt = a.x + (t * heads + h0) * a.dim;
#pragma unroll
    for (int i = 0; i < kBwdHeads; ++i) {
      const int h = h0 + i;
      x[i] = at.on && h < h_hi && h < a.hq + a.hk && head_ok(a, t, h, at) ? load8f(xt + i * a.dim, at)
                                                                          : Eight{};
    }
#pragma unroll
    for (int i = 0; i < kBwdHeads; ++i) {
      g[i] = Eight{};
      if (!at.on || h0 + i >= h_hi || !head_ok(a, t, h0 + i, at)) continue;
      const uint16_t* y = head16(a, t, h0 + i);
      const uint2 u0 = *reinterpret_cast<const uint2*>(y + at.o0);
      const uint2 u1 = *reinterpret_cast<const uint2*>(y + at.o1);
      const uint32_t us[4] = {u0.x, u0.y, u1.x, u1.y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<BF16>(us[e]);
        g[i].v[2 * e] = f.x;
        g[i].v[2 * e + 1] = f.y;
      }
    }
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at.on && at.turned && h0 < h_hi) angles<AXES>(a, t, at.pair, c, s);
    float* out = a.dx + (t * heads + h0) * a.dim;
#pragma unroll
    for (int i = 0; i < kBwdHeads; ++i) {
      const bool normed = h0 + i < a.hq + a.hk;
      if (normed && at.turned) turn<INTER, true>(g[i], c, s);   // dn
      float ss = 0.0f, sg = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[i].v[e], x[i].v[e], ss);
        sg = fmaf(g[i].v[e] * w.v[e], x[i].v[e], sg);
      }
      ss = group_sum<G>(ss);
      sg = group_sum<G>(sg);
      const float r = rsqrtf(fmaf(ss, inv_dim, a.eps));
      const float k = sg * r * r * inv_dim;   // mean(g n) / sqrt(...)
      if (!at.on || h0 + i >= h_hi || !head_ok(a, t, h0 + i, at)) continue;
      if (normed) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw.v[e] = fmaf(g[i].v[e], x[i].v[e] * r, dw.v[e]);
          g[i].v[e] = r * (g[i].v[e] * w.v[e] - x[i].v[e] * k);
        }
      }
      const float* d = g[i].v;
      *reinterpret_cast<float4*>(out + i * a.dim + at.o0) = make_float4(d[0], d[1], d[2], d[3]);
      *reinterpret_cast<float4*>(out + i * a.dim + at.o1) = make_float4(d[4], d[5], d[6], d[7]);
    }
    chunk += step_c;
    if (chunk >= chunks) {
      chunk -= chunks;
      ++t;
    }
  }
  if (at.on && dcheck(at.o1 + 4 <= G * 8, a.status, CHK_BUFFER, at.o1)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      part[group][at.o0 + e] = dw.v[e];
      part[group][at.o1 + e] = dw.v[4 + e];
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < a.dim; col += kRopeThreads) {
    float sum = 0.0f;
#pragma unroll 8
    for (int q = 0; q < GROUPS; ++q) sum += part[q][col];
    a.partial[(int64_t)blockIdx.x * a.dim + col] = sum;
  }
}

// The angles of every token, gathered by its pairs' axes into tables of a row
// to each token.
__global__ void __launch_bounds__(kRopeThreads)
    lin_gather_angles_kernel(const __grid_constant__ RopeArgs a, float* __restrict__ cos_out,
                             float* __restrict__ sin_out) {
  const int fours = a.rot / 8;
  const int64_t k = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const int64_t t = k / fours;
  if (t >= a.tokens) return;
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  angles<true>(a, t, (int)(k % fours) * 4, c, s);
  reinterpret_cast<float4*>(cos_out)[k] = c;
  reinterpret_cast<float4*>(sin_out)[k] = s;
}

// dwq (y 0) from the first q_rows of the CTAs' partial rows, dwk (y 1) from
// the others: a CTA per 32 columns, its 32 warps each a share of the rows,
// then a fixed-order sum over the warps.
__global__ void __launch_bounds__(1024)
    lin_sum_partial_rows_kernel(const float* __restrict__ partial, int q_rows, int all_rows, int dim,
                                float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float part[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int lo = blockIdx.y ? q_rows : 0, hi = blockIdx.y ? all_rows : q_rows;
  float sum = 0.0f;
  if (col < dim)
#pragma unroll 8
    for (int r = lo + warp; r < hi; r += 32) sum += partial[(int64_t)r * dim + col];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < dim) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) sum += part[w][lane];
    (blockIdx.y ? dwk : dwq)[col] = sum;
  }
}

namespace {

// Calls f with the kernel's template arguments for the shape.
template <typename F>
cudaError_t with_shape(const RopeArgs& a, bool inter, bool bf16, F&& f) {
  auto kind = [&](auto g, auto i, auto b) {
    return a.axis ? f(g, i, b, std::true_type{}) : f(g, i, b, std::false_type{});
  };
  auto types = [&](auto g) {
    if (inter)
      return bf16 ? kind(g, std::true_type{}, std::true_type{}) : kind(g, std::true_type{}, std::false_type{});
    return bf16 ? kind(g, std::false_type{}, std::true_type{})
                : kind(g, std::false_type{}, std::false_type{});
  };
  if (a.dim <= 32) return types(std::integral_constant<int, 4>{});
  if (a.dim <= 64) return types(std::integral_constant<int, 8>{});
  if (a.dim <= 128) return types(std::integral_constant<int, 16>{});
  return types(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_gather_angles(RopeArgs& a, float* room, cudaStream_t stream) {
  float* const sines = room + a.tokens * (a.rot / 2);
  const int64_t threads = a.tokens * (a.rot / 8);
  lin_gather_angles_kernel<<<(unsigned)((threads + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0,
                             stream>>>(a, room, sines);
  a.cos = room;
  a.sin = sines;
  a.pos = nullptr;
  a.axis = nullptr;
  a.table_rows = a.tokens;
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool inter, bool bf16, cudaStream_t stream) {
  return with_shape(a, inter, bf16, [&](auto g, auto i, auto b, auto x) {
    constexpr int G = decltype(g)::value;
    constexpr int GROUPS = kRopeThreads / G;
    const int64_t grid = (a.tokens + GROUPS - 1) / GROUPS *
                         ((a.hq + 2 * a.hk + kFwdHeads - 1) / kFwdHeads);
    lin_qk_norm_rope_kernel<G, decltype(i)::value, decltype(b)::value, decltype(x)::value>
        <<<(unsigned)grid, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

int qk_norm_rope_bwd_ctas(RopeArgs& a, int sms) {
  const int groups = kRopeThreads / (a.dim <= 32 ? 4 : a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32);
  auto need = [&](int heads) {
    return (a.tokens * ((heads + kBwdHeads - 1) / kBwdHeads) + groups - 1) / groups;
  };
  // the CTAs that run at once, shared out by the heads
  const int64_t q = need(a.hq), kv = need(2 * a.hk);
  const int64_t all = std::min<int64_t>(q + kv, kBwdCtas * (int64_t)sms);
  a.q_ctas = (int32_t)std::min(std::max<int64_t>(all * q / (q + kv), 1), std::max<int64_t>(all - 1, 1));
  return (int)std::max<int64_t>(all, 2);
}

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, bool inter, bool bf16, int ctas,
                                    cudaStream_t stream) {
  const cudaError_t e = with_shape(a, inter, bf16, [&](auto g, auto i, auto b, auto x) {
    lin_qk_norm_rope_bwd_kernel<decltype(g)::value, decltype(i)::value, decltype(b)::value,
                                decltype(x)::value>
        <<<(unsigned)ctas, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.dim + 31) / 32), 2, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lin_sum_partial_rows_kernel, (const float*)a.partial, a.q_ctas,
                            ctas, a.dim, a.dwq, a.dwk);
}

}  // namespace lin
