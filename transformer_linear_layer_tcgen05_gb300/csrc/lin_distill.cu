// lin_distill.cu -- distillation from a teacher's top logits: per row,
//   q = softmax(z / tau) over the vocabulary, p = softmax(t / tau) over the
//   row's listed entries,  loss = tau^2 sum_k p_k (log p_k - log q_id(k)),
//   dz = tau (q - p) inv_norm.
//
// Bound by memory: 4 bytes read and, with the gradient, 4 written per logit.
// A row is loaded once into the registers of a cluster of CTAs (512 threads
// of 32 logits each: 16384 to a CTA, up to eight CTAs along the row), whose
// maxima and sums of exponentials meet through distributed shared memory, and
// the gradient is written from the registers. What a row has beyond the
// cluster's registers is read again for the gradient. The teacher's few
// entries are done by one warp while the row is on its way; their places in
// dz are written once more, behind the row, with p taken off.
#include "lin_common.cuh"
#include "lin_distill.h"

#include <algorithm>

namespace lin {

namespace {

constexpr int kDThreads = 512;
constexpr int kDRegs = 32;                        // logits of a thread
constexpr int kDTile = kDThreads * kDRegs;        // logits of a CTA
constexpr float kDLog2E = 1.4426950408889634f;
constexpr float kDLn2 = 0.6931471805599453f;

// (m, s): maximum and sum of 2^(x - m), joined; -inf maxima (nothing) are no-ops.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) {
    s += s2;   // (both 0, or NaN)
    return;
  }
  s = (m == -INFINITY ? 0.0f : s * ex2_approx(m - mx)) +
      (m2 == -INFINITY ? 0.0f : s2 * ex2_approx(m2 - mx));
  m = mx;
}

// Logits `at` .. `end` - 1 of the row in accesses of VEC: thread t has the
// accesses t, t + 512, ... (kDRegs logits at most); -inf behind the end.
template <int VEC>
__device__ __forceinline__ void load_tile(float (&x)[kDRegs], const float* row, int at, int end) {
#pragma unroll
  for (int u = 0; u < kDRegs / VEC; ++u) {
    const int v = at + (u * kDThreads + (int)threadIdx.x) * VEC;
    if (VEC == 4 && v + 4 <= end) {
      const float4 f = *reinterpret_cast<const float4*>(row + v);
      x[u * VEC] = f.x;
      x[u * VEC + (1 % VEC)] = f.y;
      x[u * VEC + (2 % VEC)] = f.z;
      x[u * VEC + (3 % VEC)] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[u * VEC + e] = v + e < end ? row[v + e] : -INFINITY;
    }
  }
}

template <int VEC>
__device__ __forceinline__ void store_tile(const float (&x)[kDRegs], float* row, int at, int end) {
#pragma unroll
  for (int u = 0; u < kDRegs / VEC; ++u) {
    const int v = at + (u * kDThreads + (int)threadIdx.x) * VEC;
    if (VEC == 4 && v + 4 <= end) {
      *reinterpret_cast<float4*>(row + v) = make_float4(x[u * VEC], x[u * VEC + (1 % VEC)],
                                                        x[u * VEC + (2 % VEC)], x[u * VEC + (3 % VEC)]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (v + e < end) row[v + e] = x[u * VEC + e];
    }
  }
}

}  // namespace

template <int VEC>
__global__ void __launch_bounds__(kDThreads, 2)
    lin_distill_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ float red[2][kDThreads / 32];
  __shared__ float2 stats[8];            // (m, s) of each CTA of the cluster
  __shared__ int has_any;
  extern __shared__ float entries[];     // ids (as ints), p, z of the row's entries: 3 x K
  int* ids = reinterpret_cast<int*>(entries);
  float* ps = entries + a.K;
  float* zs = ps + a.K;
  const int C = a.cluster;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int64_t i = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* row = a.logits + i * a.ld;
  const float c = kDLog2E / a.tau;   // base-2 exponent of a logit
  // (a peer's shared memory is written below: it has to have begun)
  if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // This CTA's logits: tiles rank, rank + C, ... of the row; the first stays
  // in registers.
  const int V = (int)a.V;
  auto end_of = [&](int at) { return V - at < a.tile ? V : at + a.tile; };
  const int first = rank * a.tile, step = C * a.tile;
  const bool longer = step < V;   // (uniform over the cluster)
  float x[kDRegs];
  load_tile<VEC>(x, row, first, end_of(first));

  // The teacher's entries, by the last warp: p over the valid ones.
  float kl = 0.0f;   // sum p (log p - z c ln 2), without the row's log-sum-exp
  if (warp == kDThreads / 32 - 1) {
    float m = -INFINITY;
    for (int k = lane; k < a.K; k += 32) {
      const int id = a.ids[i * a.K + k];
      const bool ok = id >= 0 && id < a.V;
      const float t = ok ? a.teacher[i * a.K + k] * c : -INFINITY;
      const float z = ok ? row[id] : 0.0f;
      ids[k] = ok ? id : -1;
      ps[k] = t;
      zs[k] = z;
      m = fmaxf(m, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.0f;
    for (int k = lane; k < a.K; k += 32) s += m == -INFINITY ? 0.0f : ex2_approx(ps[k] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float ls = log2f(s);
    for (int k = lane; k < a.K; k += 32) {
      const float lp = ps[k] - m - ls;   // base 2
      const float p = m == -INFINITY ? 0.0f : ex2_approx(lp);
      ps[k] = p;
      if (p > 0.0f) kl += p * (lp - zs[k] * c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
    if (lane == 0) has_any = m != -INFINITY;
  }

  // Maximum and sum of exponentials, in base 2.
  auto tile_stats = [&](float& m, float& s) {
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < kDRegs; ++e) mx[e & 3] = fmaxf(mx[e & 3], x[e]);
    m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
    const float shift = m == -INFINITY ? 0.0f : -m;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kDRegs; ++e) sum[e & 3] += ex2_approx(fmaf(x[e], c, shift));
    s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  };
  float m, s;
  tile_stats(m, s);
  if (longer) {
    for (int at = first; at < V - step;) {
      at += step;
      load_tile<VEC>(x, row, at, end_of(at));
      float m2, s2;
      tile_stats(m2, s2);
      join(m, s, m2, s2);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
  if (lane == 0) {
    red[0][warp] = m;
    red[1][warp] = s;
  }
  __syncthreads();
  // every warp joins the warps' values by itself, in the same order
  m = lane < kDThreads / 32 ? red[0][lane] : -INFINITY;
  s = lane < kDThreads / 32 ? red[1][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
  if (C > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the peers have begun
    if (warp == 0 && lane < C) {
      const uint32_t to = mapa_shared(smem_u32(&stats[rank]), (uint32_t)lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
    }
    cluster_sync_all();
    m = stats[0].x;
    s = stats[0].y;
    for (int r = 1; r < C; ++r) join(m, s, stats[r].x, stats[r].y);
  }
  const float lse = m + log2f(s);   // base 2
  const bool any = has_any != 0;
  if (rank == 0 && warp == kDThreads / 32 - 1 && lane == 0)
    a.losses[i] = any ? a.tau * a.tau * kDLn2 * (kl + lse) : 0.0f;
  if (!a.dlogits) return;

  float* out = a.dlogits + i * a.ldd;
  const float f = any ? a.tau * a.inv_norm : 0.0f;
  auto gradient = [&](int at) {
#pragma unroll
    for (int e = 0; e < kDRegs; ++e) x[e] = any ? f * ex2_approx(fmaf(x[e], c, -lse)) : 0.0f;
    store_tile<VEC>(x, out, at, end_of(at));
  };
  if (longer) {
    for (int at = first;; at += step) {
      load_tile<VEC>(x, row, at, end_of(at));
      gradient(at);
      if (at >= V - step) break;
    }
  } else {
    gradient(first);
  }
  if (!any) return;
  __syncthreads();   // the row's stores come before the entries'
  for (int k = tid; k < a.K; k += kDThreads) {
    const int id = ids[k];
    if (id < 0 || (id / a.tile) % C != rank) continue;
    float p = 0.0f;   // an entry listed twice: the first place takes all of it
    bool mine = true;
    for (int q = 0; q < a.K; ++q)
      if (ids[q] == id) {
        mine = mine && q >= k;
        p += ps[q];
      }
    if (mine) out[id] = f * (ex2_approx(fmaf(zs[k], c, -lse)) - p);
  }
}

cudaError_t launch_distill(const DistillArgs& args, cudaStream_t stream) {
  DistillArgs a = args;
  // CTAs along the row: as many as its logits fill, a power of two up to the
  // portable cluster size
  a.cluster = 1;
  while (a.cluster < 8 && (int64_t)a.cluster * kDTile < a.V) a.cluster *= 2;
  // an even share each (a multiple of four), or the most a CTA holds
  a.tile = (int32_t)std::min<int64_t>(((a.V + a.cluster - 1) / a.cluster + 3) / 4 * 4, kDTile);
  const bool vec = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 &&
                   (!a.dlogits || (a.ldd % 4 == 0 &&
                                   (reinterpret_cast<uintptr_t>(a.dlogits) & 15u) == 0));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * a.cluster), 1, 1);
  cfg.blockDim = dim3(kDThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.K * 12;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  return vec ? cudaLaunchKernelEx(&cfg, lin_distill_kernel<4>, a)
             : cudaLaunchKernelEx(&cfg, lin_distill_kernel<1>, a);
}

}  // namespace lin
