// lin_adamw.cu -- the AdamW step over many tensors in one launch:
//   g = grad_scale * grad
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// and p's binary16 copy. States in f32, or in 8 bits: blocks of 256 entries of
// a tensor, each with the scale amax / 448 (f32), hold m and the root of v as
// e4m3 codes of entry / scale. The root, not v: a code spans 2^-9 .. 448, which
// for v itself would lose what is 500 times smaller than a block's largest
// gradient. A root above zero has at least the smallest code, so that m never
// meets a v that was rounded away. An entry that is no finite number is held
// as NaN and does not count in its block's scale.
//
// Bound by memory: 28 bytes an entry (f32), 16 (8 bits), 2 more for the copy.
// A warp takes a block of 256 entries at a time, eight to a lane: the 32-byte
// accesses of a lane use whole sectors, and the block's largest entries are a
// shuffle tree, so the codes never leave registers before they are final. 520
// million entries, 8 bits and copies, 1495 us, 6.3 TB/s of a copy's 6.8; 12.4
// million, f32 and copies, 62 us, 6.0 TB/s. Four CTAs an SM: with 3, 5, 6 and 8
// the first of these takes 1600, 1583, 1743 and 2429 us. The
// tensors' addresses are parameters of the launch: no table in memory, nothing
// to copy ahead of it, and a captured launch carries its own.
//
// Each operation is rounded by itself (no contraction), so that the states of
// a step are those of its formula in f32, whatever else a compiler might merge:
// a code next to a border does not flip with it.
#include "lin_adamw.h"

#include "lin_common.cuh"

#include <algorithm>
#include <type_traits>

namespace lin {

namespace {

constexpr int kAdamwThreads = 256;
constexpr int kAdamwCtas = 4;   // of an SM

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 load8(const float* p) {
  F8 x;
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x.v[0]), "=f"(x.v[1]), "=f"(x.v[2]), "=f"(x.v[3]), "=f"(x.v[4]),
                 "=f"(x.v[5]), "=f"(x.v[6]), "=f"(x.v[7])
               : "l"(p));
  return x;
}
__device__ __forceinline__ void store8(float* p, const F8& x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x.v[0]),
               "f"(x.v[1]), "f"(x.v[2]), "f"(x.v[3]), "f"(x.v[4]), "f"(x.v[5]), "f"(x.v[6]),
               "f"(x.v[7])
               : "memory");
}
// Entries 0 .. left - 1 (left >= 8: all), zeros behind them.
__device__ __forceinline__ F8 load_some(const float* p, int left) {
  F8 x;
#pragma unroll
  for (int e = 0; e < 8; ++e) x.v[e] = e < left ? p[e] : 0.0f;
  return x;
}
__device__ __forceinline__ void store_some(float* p, const F8& x, int left) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = x.v[e];
}

// Two e4m3 codes from two values (round to nearest even; beyond 448: 448),
// and back (exact).
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 value2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ F8 values(uint2 c, float scale) {
  F8 x;
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = value2(w[i >> 1] >> ((i & 1) * 16));
    x.v[2 * i] = __fmul_rn(f.x, scale);
    x.v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
  return x;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The codes of a block's entries (eight a lane) and its scale. LEAST: above
// zero at least the smallest code.
template <bool LEAST>
__device__ __forceinline__ uint2 codes(const F8& x, float* scale) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = finite(x.v[e]) ? fmaxf(top, fabsf(x.v[e])) : top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // (blocks below 2^-100 are zero: their scale's reciprocal would be infinite)
  *scale = top >= 0x1p-100f ? __fmul_rn(top, 1.0f / 448.0f) : 0.0f;
  const float inv = *scale > 0.0f ? __frcp_rn(*scale) : 0.0f;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float y = x.v[2 * i + k];
      c[k] = __fmul_rn(y, inv);
      if (LEAST) c[k] = c[k] > 0.0f ? fmaxf(c[k], 0x1p-9f) : c[k];
      if (!finite(y)) c[k] = NAN;
    }
    w[i] = code2(c[0], c[1]);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ uint2 load_codes(const void* base, int64_t at, bool wide, int left) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  if (wide && left >= 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e >> 2] |= (uint32_t)p[e] << ((e & 3) * 8);
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* base, int64_t at, bool wide, int left, uint2 c) {
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if (wide && left >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = (uint8_t)(w[e >> 2] >> ((e & 3) * 8));
}

}  // namespace

template <int N, bool BITS8>
__global__ void __launch_bounds__(kAdamwThreads, kAdamwCtas)
    lin_adamw_kernel(const __grid_constant__ AdamwArgs a, const __grid_constant__ AdamwList<N> list) {
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * (kAdamwThreads / 32);
  uint32_t b = blockIdx.x * (kAdamwThreads / 32) + (threadIdx.x >> 5);
  float keep = a.keep, rate = a.rate, root = a.root;
  if (a.lr || a.step) {
    const float lr = a.lr ? *a.lr : a.lr_value;
    float c1 = rate, c2 = root;   // (with the step's value: 1 / (1 - b1^t), 1 / sqrt(1 - b2^t))
    if (a.step) {
      const float t = (float)max(*a.step, 1);
      c1 = 1.0f / -expm1f(t * a.log_beta1);
      c2 = 1.0f / sqrtf(-expm1f(t * a.log_beta2));
    }
    keep = 1.0f - lr * a.decay;
    rate = lr * c1;
    root = c2;
  }
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  int i = 0;          // tensor of block b
  uint32_t next = 0;  // the first block behind it
  for (; b < a.blocks; b += warps) {
    if (b >= next) {   // the last tensor that begins at b or before (a warp's blocks only go up)
      int hi = a.tensors;
      while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (list.first[mid] <= b) i = mid; else hi = mid;
      }
      next = i + 1 < a.tensors ? list.first[i + 1] : a.blocks;
    }
    const AdamwTensor& t = list.t[i];
    const uint32_t block = b - list.first[i];
    const int64_t at = (int64_t)block * kAdamwBlock + lane * 8;
    const int64_t rest = t.n - at;
    const int left = rest >= 8 ? 8 : rest > 0 ? (int)rest : 0;
    if (!dcheck(at < (int64_t)((t.n + kAdamwBlock - 1) / kAdamwBlock) * kAdamwBlock && i < N, a.status,
                CHK_GLOBAL, at))
      continue;
    const bool whole = t.wide && left == 8;
    F8 p = whole ? load8(t.p + at) : load_some(t.p + at, left);
    const F8 g = whole ? load8(t.g + at) : load_some(t.g + at, left);
    F8 m, v;
    if constexpr (BITS8) {
      m = values(load_codes(t.m, at, t.wide, left), t.m_scale[block]);
      v = values(load_codes(t.v, at, t.wide, left), t.v_scale[block]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] = __fmul_rn(v.v[e], v.v[e]);
    } else {
      const float *mp = static_cast<const float*>(t.m) + at, *vp = static_cast<const float*>(t.v) + at;
      m = whole ? load8(mp) : load_some(mp, left);
      v = whole ? load8(vp) : load_some(vp, left);
    }
    F8 r;   // the root of v
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a.grad_scale ? __fmul_rn(g.v[e], gs) : g.v[e];
      m.v[e] = __fadd_rn(__fmul_rn(m.v[e], a.beta1), __fmul_rn(x, a.beta1_rest));
      v.v[e] = __fadd_rn(__fmul_rn(v.v[e], a.beta2), __fmul_rn(__fmul_rn(x, x), a.beta2_rest));
      r.v[e] = __fsqrt_rn(v.v[e]);
      const float d = fmaf(r.v[e], root, a.eps);
      p.v[e] = fmaf(p.v[e], keep, -rate * __fdividef(m.v[e], d));
    }
    if (whole) store8(t.p + at, p); else store_some(t.p + at, p, left);
    if constexpr (BITS8) {
      // (entries behind the tensor's end are zero and stay it)
      float ms, vs;
      const uint2 mc = codes<false>(m, &ms);
      const uint2 vc = codes<true>(r, &vs);
      store_codes(t.m, at, t.wide, left, mc);
      store_codes(t.v, at, t.wide, left, vc);
      if (lane == 0) {
        t.m_scale[block] = ms;
        t.v_scale[block] = vs;
      }
    } else {
      float *mp = static_cast<float*>(t.m) + at, *vp = static_cast<float*>(t.v) + at;
      if (whole) store8(mp, m); else store_some(mp, m, left);
      if (whole) store8(vp, v); else store_some(vp, v, left);
    }
    if (t.w16) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = pack_half2(p.v[2 * k], p.v[2 * k + 1]);
      if (whole) {
        *reinterpret_cast<uint4*>(t.w16 + at) = make_uint4(h[0], h[1], h[2], h[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) t.w16[at + e] = (uint16_t)(h[e >> 1] >> ((e & 1) * 16));
      }
    }
  }
}

cudaError_t launch_adamw(const AdamwArgs& a, const AdamwTensor* tensors, const uint32_t* first,
                         bool bits8, int sms, cudaStream_t stream) {
  constexpr int kWarps = kAdamwThreads / 32;
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.blocks + kWarps - 1) / kWarps,
                                                    (int64_t)sms * kAdamwCtas);
  auto go = [&](auto size) {
    constexpr int N = decltype(size)::value;
    AdamwList<N> list;
    for (int i = 0; i < a.tensors; ++i) {
      list.t[i] = tensors[i];
      list.first[i] = first[i];
    }
    if (bits8)
      lin_adamw_kernel<N, true><<<grid, kAdamwThreads, 0, stream>>>(a, list);
    else
      lin_adamw_kernel<N, false><<<grid, kAdamwThreads, 0, stream>>>(a, list);
    return cudaGetLastError();
  };
  // (a launch copies its parameters, whatever it uses of them: few tensors in
  // a short list)
  if (a.tensors <= 16) return go(std::integral_constant<int, 16>{});
  if (a.tensors <= 128) return go(std::integral_constant<int, 128>{});
  return go(std::integral_constant<int, kAdamwMost>{});
}

}  // namespace lin
