// lin_norms.cuh -- what stands between two blocks of the residual stream, in
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
// V units of four entries to a thread. The threads copy the units of their next
// rows into shared memory of their own meanwhile (nobody else's: a copy's end is
// all that its reader waits for). In TB/s, a copy at 6.8, f32 and bfloat16:
// 16384 x 2048 forward 5.8 and 5.7, gradient 5.9 and 5.7 (without the copies
// 4.4); 4096 x 8192 6.2 and 5.1, 4.6 and 4.1 (a row takes a whole CTA, and the
// gradient's shared memory holds one). Short calls are launches: 512 x 768 in
// 3.0-3.3 us.
//
// KIND: what a call has, the compiler's parameter (asked for in the loops, each
// question ends a run of independent instructions): 4 a norm of the block's
// output, + the gate's form, with the norm behind and, in the gradient, both
// gradients that arrive; -1: anything else, asked for at run time.
#pragma once

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

// A team's rows on their way: `slots` places in shared memory, each of a row's
// units of up to four tensors. A thread copies and reads its own units only, so
// a copy's end is all that it waits for.
template <int T, int V, int F32, int BLOCK>
struct Staged {
  static constexpr int kUnit = T == LIN_BINARY32 ? 16 : 8;             // of the block's tensors
  static constexpr int kThread = V * (F32 * 16 + BLOCK * kUnit);       // bytes of a thread and slot
  uint8_t* base;   // of this thread
  int threads;     // of the CTA
  // Unit i of tensor k (the f32 ones first): units of a tensor side by side
  // over the threads.
  __device__ __forceinline__ uint8_t* place(int slot, int k, int i) const {
    const int before = slot * kThread + V * (k < F32 ? k * 16 : F32 * 16 + (k - F32) * kUnit);
    const int unit = k < F32 ? 16 : kUnit;
    return base + (before + i * unit) * threads + threadIdx.x * unit;
  }
  __device__ __forceinline__ void copy_f32(int slot, int k, int i, const float* from) const {
    cp_async_16(smem_u32(place(slot, k, i)), from);
  }
  __device__ __forceinline__ void copy_block(int slot, int k, int i, const void* tensor, int64_t at) const {
    if constexpr (T == LIN_BINARY32)
      cp_async_16(smem_u32(place(slot, k, i)), static_cast<const float*>(tensor) + at);
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(place(slot, k, i))),
                   "l"(static_cast<const uint16_t*>(tensor) + at)
                   : "memory");
  }
  __device__ __forceinline__ Four f32(int slot, int k, int i) const {
    return load4<LIN_BINARY32>(place(slot, k, i), 0);
  }
  __device__ __forceinline__ Four block(int slot, int k, int i) const {
    return load4<T>(place(slot, k, i), 0);
  }
};
// A row's copies are GROUPS groups; the oldest of `slots` rows' are complete.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int GROUPS>
__device__ __forceinline__ void copies_wait(int slots) {
  if (slots == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (slots == 2) asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS) : "memory");
  else asm volatile("cp.async.wait_group %0;" ::"n"(3 * GROUPS) : "memory");
}

}  // namespace

// What a call has.
template <int KIND>
struct NormParts {
  bool y, post, behind, dh;
  int form;
  __device__ __forceinline__ explicit NormParts(const NormsArgs& a, bool gradient)
      : y(KIND >= 0 || a.y), post(KIND >= 0 ? KIND >= 4 : a.w_post != nullptr),
        behind(KIND >= 0 || a.w_pre), dh(KIND >= 0 ? gradient : a.dh != nullptr),
        form(KIND >= 0 ? KIND & 3 : a.form) {}
};

// The teams of the grid walk over the rows with a fixed stride.
template <int T, int V, int KIND>
__global__ void __launch_bounds__(kNormThreads, 2)
    lin_block_norms_kernel(const __grid_constant__ NormsArgs a, int warps, int slots) {
  extern __shared__ float4 shared[];
  __shared__ float4 red[2 * kNormThreads / 32];
  Team team(warps, red);
  const NormParts<KIND> has(a, false);
  const Staged<T, V, 1, 1> staged{reinterpret_cast<uint8_t*>(shared), (int)blockDim.x};
  const int teams = blockDim.x / team.threads;
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv_w = 1.0f / (float)a.width;
  auto copy = [&](int64_t t, int slot) {
    if (t < a.tokens) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = (i * team.threads + team.thread) * 4;
        if (col >= a.width || !unit_ok(a, t, col)) continue;
        staged.copy_f32(slot, 0, i, a.x + t * a.width + col);
        if (has.y) staged.copy_block(slot, 1, i, a.y, t * a.width + col);
      }
    }
    copies_commit();   // (a group for each row, also behind the last one)
  };
  int64_t t = (int64_t)blockIdx.x * teams + team.team;
  for (int s = 0; s < slots; ++s) copy(t + s * step, s);
  int slot = 0;
  for (; t < a.tokens; t += step) {
    const int64_t row = t * a.width;
    const float gt = has.form == NORM_GATE_TOKEN ? a.gate[t] : 1.0f;
    copies_wait<1>(slots);
    float ry = 1.0f;
    if (has.post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if ((i * team.threads + team.thread) * 4 >= a.width) continue;
        const Four y = staged.block(slot, 1, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(y.v[e], y.v[e], ss);
      }
      ry = rsqrtf(fmaf(team.sum(make_float4(ss, 0.f, 0.f, 0.f)).x, inv_w, a.eps));
    }
    const float k = a.block_scale * gt * ry;
    float ss = 0.0f;
    Four h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      if (col >= a.width) continue;
      h[i] = staged.f32(slot, 0, i);
      Four y{};
      if (has.y) y = staged.block(slot, 1, i);
      const Four w = has.post ? load4f(a.w_post, col) : ones();
      Four g = ones();
      if (has.form == NORM_GATE_CHANNEL) g = load4f(a.gate, col);
      if (has.form == NORM_GATE_FULL) g = load4f(a.gate, row + col);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& x = h[i].v[e];
        x *= a.residual_scale;
        if (has.y) x = fmaf(k * g.v[e], w.v[e] * y.v[e], x);
        ss = fmaf(x, x, ss);
      }
      if (a.h && unit_ok(a, t, col)) store4<LIN_BINARY32>(a.h, row + col, h[i]);
    }
    __syncwarp();   // (what the slot held has been read: it may change)
    copy(t + slots * step, slot);
    slot = slot + 1 == slots ? 0 : slot + 1;
    if (!has.behind) continue;
    const float rh = rsqrtf(fmaf(team.sum(make_float4(ss, 0.f, 0.f, 0.f)).x, inv_w, a.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      if (col >= a.width || !unit_ok(a, t, col)) continue;
      const Four w = load4f(a.w_pre, col);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[i].v[e] *= rh * w.v[e];
      store4<T>(a.n, row + col, h[i]);
    }
  }
}

// The gradient. A CTA's teams keep the sums over the tokens of their columns in
// registers (and read a row's units from shared memory as often as they want
// them, for which registers are short); the teams' are added in order and leave
// one partial row of each kind, and a second kernel adds those: the same call
// gives the same bits. The weights and a channel's gate are in shared memory:
// beside the rows' slots the first-level cache is too small for them (16384 x
// 2048, bfloat16: 171 us, its time spent on their way).
template <int T, int V, int KIND>
__global__ void __launch_bounds__(kNormThreads, 1)
    lin_block_norms_bwd_kernel(const __grid_constant__ NormsArgs a, int warps, int slots) {
  extern __shared__ float4 shared[];
  // w_pre, w_post and a channel's gate; later a team's sums
  float* const weights[3] = {reinterpret_cast<float*>(shared), reinterpret_cast<float*>(shared) + a.width,
                             reinterpret_cast<float*>(shared) + 2 * a.width};
  float4* const sums = shared;
  __shared__ float4 red[2 * kNormThreads / 32];
  Team team(warps, red);
  const NormParts<KIND> has(a, true);
  // h, dh, y, dn
  const Staged<T, V, 2, 2> staged{reinterpret_cast<uint8_t*>(shared) + a.width * 12, (int)blockDim.x};
  const int teams = blockDim.x / team.threads;
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv_w = 1.0f / (float)a.width;
  // a row's copies: what the first two of its three turns read, and y
  auto copy = [&](int64_t t, int slot, bool first) {
    if (t < a.tokens) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = (i * team.threads + team.thread) * 4;
        if (col >= a.width || !unit_ok(a, t, col)) continue;
        const int64_t at = t * a.width + col;
        if (first && has.behind) staged.copy_f32(slot, 0, i, a.x + at);
        if (first && has.dh) staged.copy_f32(slot, 1, i, a.dh + at);
        if (!first && has.y) staged.copy_block(slot, 2, i, a.y, at);
        if (first && has.behind) staged.copy_block(slot, 3, i, a.dn, at);
      }
    }
    copies_commit();   // (two groups for each row, also behind the last one)
  };
  Four d_pre[V]{}, d_post[V]{}, d_gate[V]{};
  int64_t t = (int64_t)blockIdx.x * teams + team.team;
  for (int s = 0; s < slots; ++s) {
    copy(t + s * step, s, true);
    copy(t + s * step, s, false);
  }
  for (int u = threadIdx.x; u * 4 < a.width; u += blockDim.x) {
    if (has.behind) reinterpret_cast<float4*>(weights[0])[u] = reinterpret_cast<const float4*>(a.w_pre)[u];
    if (has.post) reinterpret_cast<float4*>(weights[1])[u] = reinterpret_cast<const float4*>(a.w_post)[u];
    if (has.form == NORM_GATE_CHANNEL)
      reinterpret_cast<float4*>(weights[2])[u] = reinterpret_cast<const float4*>(a.gate)[u];
  }
  __syncthreads();
  int slot = 0;
  for (; t < a.tokens; t += step) {
    const int64_t row = t * a.width;
    const float gt = has.form == NORM_GATE_TOKEN ? a.gate[t] : 1.0f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    copies_wait<2>(slots);
    if (has.behind || has.post) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = (i * team.threads + team.thread) * 4;
        if (col >= a.width) continue;
        if (has.behind) {
          const Four h = staged.f32(slot, 0, i), dn = staged.block(slot, 3, i), w = load4f(weights[0], col);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s.x = fmaf(h.v[e], h.v[e], s.x);
            s.y = fmaf(dn.v[e] * w.v[e], h.v[e], s.y);
          }
        }
        if (has.post) {
          const Four y = staged.block(slot, 2, i);
#pragma unroll
          for (int e = 0; e < 4; ++e) s.z = fmaf(y.v[e], y.v[e], s.z);
        }
      }
      s = team.sum(s);
    }
    const float rh = rsqrtf(fmaf(s.x, inv_w, a.eps)), kh = s.y * rh * rh * inv_w;
    const float ry = has.post ? rsqrtf(fmaf(s.z, inv_w, a.eps)) : 1.0f;
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    Four d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * team.threads + team.thread) * 4;
      if (col >= a.width) continue;
      d[i] = has.dh ? staged.f32(slot, 1, i) : Four{};
      if (has.behind) {
        const Four h = staged.f32(slot, 0, i), dn = staged.block(slot, 3, i), w = load4f(weights[0], col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[i].v[e] = fmaf(rh, fmaf(dn.v[e], w.v[e], -h.v[e] * kh), d[i].v[e]);
          d_pre[i].v[e] = fmaf(dn.v[e], h.v[e] * rh, d_pre[i].v[e]);
        }
      }
      if (unit_ok(a, t, col)) {
        Four o = d[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) o.v[e] *= a.residual_scale;
        store4<LIN_BINARY32>(a.dx, row + col, o);
      }
      if (!has.y) continue;
      const Four y = staged.block(slot, 2, i), w = has.post ? load4f(weights[1], col) : ones();
      Four g = ones();
      if (has.form == NORM_GATE_CHANNEL) g = load4f(weights[2], col);
      if (has.form == NORM_GATE_FULL) g = load4f(a.gate, row + col);
      Four dg;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float db = a.block_scale * d[i].v[e];      // gradient of gate * b
        const float wy = w.v[e] * y.v[e];
        s.x = fmaf(db * g.v[e], wy, s.x);                // (a token's gate stands outside)
        dg.v[e] = db * wy * ry;
        d[i].v[e] = db * g.v[e] * gt;                    // u
      }
      if (has.form == NORM_GATE_CHANNEL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d_gate[i].v[e] += dg.v[e];
      } else if (has.form == NORM_GATE_FULL && unit_ok(a, t, col)) {
        store4<LIN_BINARY32>(a.dgate, row + col, dg);
      }
    }
    __syncwarp();   // (what the slot held has been read, but y: it may change)
    copy(t + slots * step, slot, true);
    if (has.y) {
      if (has.post || has.form == NORM_GATE_TOKEN) s = team.sum(s);
      if (has.form == NORM_GATE_TOKEN && team.thread == 0) a.dgate[t] = s.x * ry;
      const float ky = s.x * gt * ry * ry * inv_w;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = (i * team.threads + team.thread) * 4;
        if (col >= a.width || !unit_ok(a, t, col)) continue;
        if (has.post) {
          const Four y = staged.block(slot, 2, i), w = load4f(weights[1], col);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = d[i].v[e];
            d_post[i].v[e] = fmaf(u, y.v[e] * ry, d_post[i].v[e]);
            d[i].v[e] = ry * fmaf(u, w.v[e], -y.v[e] * ky);
          }
        }
        store4<T>(a.dy, row + col, d[i]);
      }
    }
    __syncwarp();
    copy(t + slots * step, slot, false);
    slot = slot + 1 == slots ? 0 : slot + 1;
  }
  if (a.kinds == 0) return;
  __syncthreads();   // (the weights are done with)
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
  if (has.behind) leave(d_pre);
  if (has.post) leave(d_post);
  if (has.form == NORM_GATE_CHANNEL) leave(d_gate);
}

namespace {

// Units of four entries to a thread and warps of a team (small teams, so that
// an SM has many rows in hand: what a row takes is the way of its sums), teams of
// a CTA, slots of each of them, and CTAs.
struct NormShape {
  int v, warps, teams, slots, ctas;
  size_t smem;
};
template <typename Bytes>
inline NormShape norm_shape(int64_t tokens, int width, int64_t ctas, size_t room, Bytes&& bytes_of_thread) {
  const int units = width / 4;
  NormShape s;
  // as many units to a thread as let all rows have warps of their own at once
  for (s.v = 1; s.v < 4; ++s.v)
    if (tokens * ((units + 32 * s.v - 1) / (32 * s.v)) <= kNormThreads / 32 * ctas) break;
  s.warps = (units + 32 * s.v - 1) / (32 * s.v);
  if (s.warps > kNormThreads / 32) s.warps = kNormThreads / 32;
  s.v = std::max(1, (units + 32 * s.warps - 1) / (32 * s.warps));
  // (a named barrier to each team of several warps; few rows: on many SMs)
  s.teams = std::min(std::max(1, kNormThreads / 32 / s.warps), s.warps > 1 ? 15 : 16);
  s.teams = (int)std::min<int64_t>(s.teams, std::max<int64_t>(1, (tokens + ctas - 1) / ctas));
  s.ctas = (int)std::min<int64_t>((tokens + s.teams - 1) / s.teams, ctas);
  // slots: four, or what a team has rows and shared memory room for
  const size_t slot = (size_t)s.teams * s.warps * 32 * bytes_of_thread(s.v);
  const int64_t rows = (tokens + (int64_t)s.ctas * s.teams - 1) / ((int64_t)s.ctas * s.teams);
  s.slots = rows > 2 && slot * 4 <= room ? 4 : rows > 1 && slot * 2 <= room ? 2 : 1;
  s.smem = slot * s.slots;
  return s;
}
// Shared memory that a CTA may have of a launch's own.
constexpr size_t kNormFwdShared = 112 * 1024, kNormBwdShared = 226 * 1024;
inline NormShape fwd_shape(const NormsArgs& a, int sms) {   // (two CTAs an SM)
  const int b = a.dtype == LIN_BINARY32 ? 16 : 8;
  return norm_shape(a.tokens, a.width, 2 * (int64_t)sms, kNormFwdShared, [&](int v) { return v * (16 + b); });
}
inline NormShape bwd_shape(const NormsArgs& a, int sms) {
  const int b = a.dtype == LIN_BINARY32 ? 16 : 8;
  return norm_shape(a.tokens, a.width, sms, kNormBwdShared - (size_t)a.width * 12,
                    [&](int v) { return v * (32 + 2 * b); });
}

}  // namespace

// The kernel of a call of the type T: its units to a thread and its kind.
template <int T, typename F>
cudaError_t with_norm(int v, int kind, F&& f) {
  auto size = [&](auto k) {
    if (v == 1) return f(std::integral_constant<int, 1>{}, k);
    if (v == 2) return f(std::integral_constant<int, 2>{}, k);
    if (v == 3) return f(std::integral_constant<int, 3>{}, k);
    return f(std::integral_constant<int, 4>{}, k);
  };
  switch (kind) {
    case 0: return size(std::integral_constant<int, 0>{});
    case 1: return size(std::integral_constant<int, 1>{});
    case 2: return size(std::integral_constant<int, 2>{});
    case 3: return size(std::integral_constant<int, 3>{});
    case 4: return size(std::integral_constant<int, 4>{});
    case 5: return size(std::integral_constant<int, 5>{});
    case 6: return size(std::integral_constant<int, 6>{});
    case 7: return size(std::integral_constant<int, 7>{});
    default: return size(std::integral_constant<int, -1>{});
  }
}

// Leave for more shared memory than a launch may have without: always up to
// `most`, not this call's `bytes`. The leave is the kernel's, in the whole
// process: set to what a call needs, a smaller call of another host thread could
// take it back before this one's launch.
template <typename Kernel>
cudaError_t more_shared(Kernel kernel, size_t bytes, size_t most) {
  if (bytes + 1024 <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

template <int T>
cudaError_t launch_block_norms_of(const NormsArgs& a, int sms, cudaStream_t stream) {
  const NormShape s = fwd_shape(a, sms);
  const int kind = a.y && a.n && a.h ? (a.w_post ? 4 : 0) + a.form : -1;
  return with_norm<T>(s.v, kind, [&](auto v, auto k) {
    auto kernel = lin_block_norms_kernel<T, decltype(v)::value, decltype(k)::value>;
    const cudaError_t e = more_shared(kernel, s.smem, kNormFwdShared);
    if (e != cudaSuccess) return e;
    kernel<<<s.ctas, s.teams * s.warps * 32, s.smem, stream>>>(a, s.warps, s.slots);
    return cudaGetLastError();
  });
}

template <int T>
cudaError_t launch_block_norms_bwd_of(const NormsArgs& a, int sms, cudaStream_t stream) {
  const NormShape s = bwd_shape(a, sms);
  const int kind = a.y && a.dn && a.dh ? (a.w_post ? 4 : 0) + a.form : -1;
  return with_norm<T>(s.v, kind, [&](auto v, auto k) {
    auto kernel = lin_block_norms_bwd_kernel<T, decltype(v)::value, decltype(k)::value>;
    const size_t smem = (size_t)a.width * 12 + s.smem;
    const cudaError_t e = more_shared(kernel, smem, kNormBwdShared);
    if (e != cudaSuccess) return e;
    kernel<<<s.ctas, s.teams * s.warps * 32, smem, stream>>>(a, s.warps, s.slots);
    return cudaGetLastError();
  });
}

}  // namespace lin
