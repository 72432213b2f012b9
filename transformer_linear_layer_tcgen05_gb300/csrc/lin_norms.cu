// lin_norms.cu -- what stands between two blocks of the residual stream, in
// one pass:
//   b = w_post y / sqrt(mean y^2 + eps)      (or b = y without a norm behind the block)
//   h = residual_scale x + block_scale gate b
//   n = w_pre h / sqrt(mean h^2 + eps)       (the next block's input)
// and its gradient, with r_h, r_y the two reciprocal roots and W the width:
//   d = dh + r_h (dn w_pre - h r_h^2 / W sum(dn w_pre h)),  dx = residual_scale d
//   u = block_scale gate d
//   dy = r_y (u w_post - y r_y^2 / W sum(u w_post y))       (or dy = u)
//   dw_pre = sum dn h r_h,  dw_post = sum u y r_y,  dgate = sum block_scale d b
// the last over the tokens, over the width, or not at all, as the gate's form
// has it.
//
// Bound by memory: a row's entries stay in registers from its first sum to its
// results, so each tensor is read or written once. A team of warps has a row,
// V units of four entries to a thread. The gradient's threads copy the units of
// their next rows into shared memory of their own meanwhile (nobody else's: a
// copy's end is all that its reader waits for).
#include "lin_norms.h"

#include "lin_common.cuh"

#include <algorithm>
#include <cuda_bf16.h>
#include <type_traits>

namespace lin {

namespace {

constexpr int kNormThreads = 512;   // of a CTA, at most

// Four entries of an f32 (T 2), binary16 (0) or bfloat16 (1) row.
struct Four {
  float v[4];
};
template <int T>
__device__ __forceinline__ Four load4(const void* base, int64_t at) {
  if constexpr (T == LIN_BINARY32) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    return Four{{f.x, f.y, f.z, f.w}};
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    if constexpr (T == LIN_BFLOAT16)
      return Four{{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                   __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)}};
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return Four{{a.x, a.y, b.x, b.y}};
  }
}
template <int T>
__device__ __forceinline__ void store4(void* base, int64_t at, const Four& x) {
  if constexpr (T == LIN_BINARY32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) =
        make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  } else {
    uint2 u;
    if constexpr (T == LIN_BFLOAT16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(x.v[0], x.v[1]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(x.v[2], x.v[3]);
      u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      u = make_uint2(pack_half2(x.v[0], x.v[1]), pack_half2(x.v[2], x.v[3]));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = u;
  }
}
__device__ __forceinline__ Four load4f(const float* p, int64_t at) { return load4<LIN_BINARY32>(p, at); }
__device__ __forceinline__ Four ones() { return Four{{1.0f, 1.0f, 1.0f, 1.0f}}; }

// A CTA's warps as teams of `warps` (threads to a row); sums over a team go
// through shared memory, two buffers in turn, so that one barrier a sum is
// enough: what a buffer held is read before the barrier of the sum between.
struct Team {
  int warps, team, thread, threads;   // of this thread: its team, its place in it
  float4* red;                        // [2][warps of the CTA]
  int turn;
  __device__ __forceinline__ Team(int warps_, float4* red_)
      : warps(warps_), team((int)(threadIdx.x >> 5) / warps_),
        thread((int)threadIdx.x - team * warps_ * 32), threads(warps_ * 32), red(red_), turn(0) {}
  __device__ __forceinline__ float4 sum(float4 s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
      s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    }
    if (warps == 1) return s;
    float4* r = red + turn * (kNormThreads / 32) + team * warps;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) r[thread >> 5] = s;
    named_bar_sync(1 + team, threads);
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < warps; ++w) {
      const float4 q = r[w];
      s.x += q.x;
      s.y += q.y;
      s.z += q.z;
    }
    return s;
  }
};

// Checked build: a unit's four entries inside the row, the row inside the tensors.
__device__ __forceinline__ bool unit_ok(const NormsArgs& a, int64_t t, int col) {
  return dcheck(t >= 0 && t < a.tokens && col >= 0 && col + 4 <= a.width, a.status, CHK_GLOBAL, t);
}

}  // namespace

template <int T, int V>
__global__ void __launch_bounds__(kNormThreads, 2)
    lin_block_norms_kernel(const __grid_constant__ NormsArgs a, int warps) {
  __shared__ float4 red[2 * kNormThreads / 32];
  Team team(warps, red);
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / team.threads) + team.team;
  if (t >= a.tokens) return;   // (the whole team)
  const int64_t row = t * a.width;
  Four y[V], x[V];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * team.threads + team.thread) * 4;
    const bool in = col < a.width && unit_ok(a, t, col);
    y[i] = in && a.y ? load4<T>(a.y, row + col) : Four{};
    x[i] = in ? load4f(a.x, row + col) : Four{};
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(y[i].v[e], y[i].v[e], ss);
  }
  float ry = 1.0f;
  if (a.w_post) ry = rsqrtf(team.sum(make_float4(ss, 0.f, 0.f, 0.f)).x / (float)a.width + a.eps);
  const float k = a.block_scale * (a.form == NORM_GATE_TOKEN ? a.gate[t] : 1.0f) * ry;
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * team.threads + team.thread) * 4;
    if (col >= a.width) continue;
    const Four w = a.w_post ? load4f(a.w_post, col) : ones();
    Four g = ones();
    if (a.form == NORM_GATE_CHANNEL) g = load4f(a.gate, col);
    if (a.form == NORM_GATE_FULL) g = load4f(a.gate, row + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float& h = x[i].v[e];
      h *= a.residual_scale;
      if (a.y) h = fmaf(k * g.v[e], w.v[e] * y[i].v[e], h);
      ss = fmaf(h, h, ss);
    }
    if (a.h && unit_ok(a, t, col)) store4<LIN_BINARY32>(a.h, row + col, x[i]);
  }
  if (!a.n) return;
  const float rh = rsqrtf(team.sum(make_float4(ss, 0.f, 0.f, 0.f)).x / (float)a.width + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * team.threads + team.thread) * 4;
    if (col >= a.width || !unit_ok(a, t, col)) continue;
    const Four w = load4f(a.w_pre, col);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i].v[e] *= rh * w.v[e];
    store4<T>(a.n, row + col, x[i]);
  }
}

// Bytes of a thread's units of a row in shared memory, and rows on their way.
template <int T, int V>
struct NormStage {
  static constexpr int kUnit = T == LIN_BINARY32 ? 16 : 8;   // of y and dn
  static constexpr int kThread = V * (32 + 2 * kUnit);
  static constexpr int kRows = V == 4 ? 1 : V == 2 ? 2 : 4;
  static constexpr int kBytes = kRows * kThread * kNormThreads;
  static_assert(kBytes + 4 * kNormMostWidth <= 227 * 1024, "shared memory");
};
// A unit's copy; complete after cp_async_wait.
__device__ __forceinline__ void copy_unit8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The gradient. A CTA's teams walk over the rows with a fixed stride and keep
// the sums over the tokens of their columns in registers; the teams' are added
// in order and leave one partial row of each kind, and a second kernel adds
// those: the same call gives the same bits.
template <int T, int V>
__global__ void __launch_bounds__(kNormThreads, 1)
    lin_block_norms_bwd_kernel(const __grid_constant__ NormsArgs a, int warps) {
  using Stage = NormStage<T, V>;
  extern __shared__ float4 shared[];
  float4* const sums = shared;       // [units of a row] of a team's sums
  uint8_t* const staged = reinterpret_cast<uint8_t*>(shared) + ((a.width + 3) / 4) * 16;
  __shared__ float4 red[2 * kNormThreads / 32];
  Team team(warps, red);
  const int teams = blockDim.x / team.threads;
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv_w = 1.0f / (float)a.width;
  // Unit i of tensor k (h, dh, y, dn) of the row in place `at`: units of a
  // tensor side by side over the threads.
  auto place = [&](int at, int k, int i) {
    const int before = at * Stage::kThread + V * (k < 2 ? k * 16 : 32 + (k - 2) * Stage::kUnit);
    const int unit = k < 2 ? 16 : Stage::kUnit;
    return staged + before * blockDim.x + (i * blockDim.x + threadIdx.x) * unit;
  };
  auto copy = [&](int64_t t, int at) {
    if (t < a.tokens) {
      const int64_t row = t * a.width;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = (i * team.threads + team.thread) * 4;
        if (col >= a.width || !unit_ok(a, t, col)) continue;
        if (a.dn) cp_async_16(smem_u32(place(at, 0, i)), a.x + row + col);
        if (a.dh) cp_async_16(smem_u32(place(at, 1, i)), a.dh + row + col);
        auto block = [&](const void* from, int k) {
          if constexpr (T == LIN_BINARY32)
            cp_async_16(smem_u32(place(at, k, i)), static_cast<const float*>(from) + row + col);
          else
            copy_unit8(smem_u32(place(at, k, i)), static_cast<const uint16_t*>(from) + row + col);
        };
        if (a.y) block(a.y, 2);
        if (a.dn) block(a.dn, 3);
      }
    }
    copies_commit();   // (a group for each row, also behind the last one)
  };
  Four d_pre[V]{}, d_post[V]{}, d_gate[V]{};
  int64_t t = (int64_t)blockIdx.x * teams + team.team;
#pragma unroll
  for (int s = 0; s < Stage::kRows; ++s) copy(t + s * step, s);
  int at = 0;
  for (; t < a.tokens; t += step) {
    const int64_t row = t * a.width;
    Four h[V], y[V], dn[V], d[V];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    copies_wait<Stage::kRows - 1>();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      const bool in = col < a.width;
      h[i] = in && a.dn ? load4<LIN_BINARY32>(place(at, 0, i), 0) : Four{};
      d[i] = in && a.dh ? load4<LIN_BINARY32>(place(at, 1, i), 0) : Four{};
      y[i] = in && a.y ? load4<T>(place(at, 2, i), 0) : Four{};
      dn[i] = in && a.dn ? load4<T>(place(at, 3, i), 0) : Four{};
    }
    const float gt = a.form == NORM_GATE_TOKEN ? a.gate[t] : 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      const Four w = col < a.width && a.w_pre ? load4f(a.w_pre, col) : Four{};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s.x = fmaf(h[i].v[e], h[i].v[e], s.x);
        s.y = fmaf(dn[i].v[e] * w.v[e], h[i].v[e], s.y);
        s.z = fmaf(y[i].v[e], y[i].v[e], s.z);
      }
    }
    if (a.dn || a.w_post) s = team.sum(s);
    __syncwarp();   // (what the row's place held has been read: it may change)
    copy(t + Stage::kRows * step, at);
    at = at + 1 == Stage::kRows ? 0 : at + 1;
    const float rh = rsqrtf(fmaf(s.x, inv_w, a.eps)), kh = s.y * rh * rh * inv_w;
    const float ry = a.w_post ? rsqrtf(fmaf(s.z, inv_w, a.eps)) : 1.0f;
    s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      if (col >= a.width) continue;
      if (a.dn) {
        const Four w = load4f(a.w_pre, col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[i].v[e] = fmaf(rh, fmaf(dn[i].v[e], w.v[e], -h[i].v[e] * kh), d[i].v[e]);
          d_pre[i].v[e] = fmaf(dn[i].v[e], h[i].v[e] * rh, d_pre[i].v[e]);
        }
      }
      if (unit_ok(a, t, col)) {
        Four o = d[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) o.v[e] *= a.residual_scale;
        store4<LIN_BINARY32>(a.dx, row + col, o);
      }
      if (!a.y) continue;
      const Four w = a.w_post ? load4f(a.w_post, col) : ones();
      Four g = ones();
      if (a.form == NORM_GATE_CHANNEL) g = load4f(a.gate, col);
      if (a.form == NORM_GATE_FULL) g = load4f(a.gate, row + col);
      Four dg;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float db = a.block_scale * d[i].v[e];      // gradient of gate * b
        const float wy = w.v[e] * y[i].v[e];
        s.x = fmaf(db * g.v[e], wy, s.x);                // (a token's gate stands outside)
        dg.v[e] = db * wy * ry;
        d[i].v[e] = db * g.v[e] * gt;                    // u
      }
      if (a.form == NORM_GATE_CHANNEL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d_gate[i].v[e] += dg.v[e];
      } else if (a.form == NORM_GATE_FULL && unit_ok(a, t, col)) {
        store4<LIN_BINARY32>(a.dgate, row + col, dg);
      }
    }
    if (!a.y) continue;
    if (a.w_post || a.form == NORM_GATE_TOKEN) s = team.sum(s);
    if (a.form == NORM_GATE_TOKEN && team.thread == 0) a.dgate[t] = s.x * ry;
    const float ky = s.x * gt * ry * ry * inv_w;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      if (col >= a.width || !unit_ok(a, t, col)) continue;
      if (a.w_post) {
        const Four w = load4f(a.w_post, col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = d[i].v[e];
          d_post[i].v[e] = fmaf(u, y[i].v[e] * ry, d_post[i].v[e]);
          d[i].v[e] = ry * fmaf(u, w.v[e], -y[i].v[e] * ky);
        }
      }
      store4<T>(a.dy, row + col, d[i]);
    }
  }
  if (a.kinds == 0) return;
  int kind = 0;
  auto leave = [&](const Four (&mine)[V]) {
    // the teams' sums, one after another
    for (int q = 0; q < teams; ++q) {
      if (q == team.team) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = i * team.threads + team.thread;
          if (u * 4 >= a.width) continue;
          float4 v = make_float4(mine[i].v[0], mine[i].v[1], mine[i].v[2], mine[i].v[3]);
          if (q > 0) {
            const float4 o = sums[u];
            v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
          }
          sums[u] = v;
        }
      }
      __syncthreads();
    }
    float4* out = reinterpret_cast<float4*>(a.partial + ((int64_t)blockIdx.x * a.kinds + kind) * a.width);
    for (int u = threadIdx.x; u * 4 < a.width; u += blockDim.x) out[u] = sums[u];
    __syncthreads();
    ++kind;
  };
  if (a.dn) leave(d_pre);
  if (a.w_post) leave(d_post);
  if (a.form == NORM_GATE_CHANNEL) leave(d_gate);
}

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

// Units of four entries to a thread and warps of a team.
struct NormShape {
  int v, warps, teams;
};
NormShape norm_shape(int width, int most_threads) {
  const int units = width / 4;
  NormShape s;
  s.v = units <= 256 ? 1 : units <= 1024 ? 2 : 4;
  s.warps = (units + 32 * s.v - 1) / (32 * s.v);
  s.teams = std::max(1, most_threads / 32 / s.warps);
  if (s.warps > 1) s.teams = std::min(s.teams, 15);   // (a named barrier to each)
  return s;
}

template <typename F>
cudaError_t with_types(int dtype, int v, F&& f) {
  auto size = [&](auto t) {
    if (v == 1) return f(t, std::integral_constant<int, 1>{});
    if (v == 2) return f(t, std::integral_constant<int, 2>{});
    return f(t, std::integral_constant<int, 4>{});
  };
  if (dtype == LIN_BINARY32) return size(std::integral_constant<int, LIN_BINARY32>{});
  if (dtype == LIN_BFLOAT16) return size(std::integral_constant<int, LIN_BFLOAT16>{});
  return size(std::integral_constant<int, LIN_BINARY16>{});
}

}  // namespace

cudaError_t launch_block_norms(const NormsArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(a.width, 128);
  return with_types(a.dtype, s.v, [&](auto t, auto v) {
    lin_block_norms_kernel<decltype(t)::value, decltype(v)::value>
        <<<(unsigned)((a.tokens + s.teams - 1) / s.teams), s.teams * s.warps * 32, 0, stream>>>(a, s.warps);
    return cudaGetLastError();
  });
}

int block_norms_bwd_ctas(const NormsArgs& a, int sms) {
  const NormShape s = norm_shape(a.width, kNormThreads);
  return (int)std::min<int64_t>((a.tokens + s.teams - 1) / s.teams, sms);
}

cudaError_t launch_block_norms_bwd(const NormsArgs& a, int ctas, cudaStream_t stream) {
  const NormShape s = norm_shape(a.width, kNormThreads);
  const cudaError_t e = with_types(a.dtype, s.v, [&](auto t, auto v) {
    constexpr int T = decltype(t)::value, V = decltype(v)::value;
    using Stage = NormStage<T, V>;
    auto kernel = lin_block_norms_bwd_kernel<T, V>;
    const int threads = s.teams * s.warps * 32;
    const size_t smem = (size_t)a.width * 4 + (size_t)Stage::kRows * Stage::kThread * threads;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)ctas, threads, smem, stream>>>(a, s.warps);
    return cudaGetLastError();
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
