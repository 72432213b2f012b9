// lin_distill.cu -- distillation from a teacher's top logits: per row,
//   q = softmax(z / tau) over the vocabulary, p = softmax(t / tau) over the
//   row's listed entries,  loss = tau^2 sum_k p_k (log p_k - log q_id(k)),
//   dz = tau (q - p) inv_norm.
//
// Bound by memory: 4 bytes read and, with the gradient, 4 written per logit.
// Persistent CTAs (clusters of up to eight along a long row) walk over the
// rows. A bulk copy brings a CTA's part of a row into shared memory, from
// where it is read twice: for the maximum and the sum of exponentials, the
// CTA's and the cluster's (through distributed shared memory), and for the
// gradient, written straight out; the next row's copy follows at once.
// Several CTAs share an SM, so that one's copy and waits are filled by the
// others' arithmetic and stores. A warp of its own prepares the teacher's
// entries one row ahead, since their two dependent loads (id, then its logit)
// would otherwise stand in every row's way; their places in dz are written
// again, behind the row, with p taken off.
//
// A row is handled in the 16-byte units of memory that it touches, so rows
// may start anywhere: only the first and the last unit can be partial, and
// their entries are loaded one by one.
#include "lin_common.cuh"
#include "lin_distill.h"

#include <algorithm>

namespace lin {

namespace {

constexpr int kSlots = 3;                // parts of a row in shared memory, at most
constexpr int kChunk = 4;                // 16-byte units of a thread in registers at once

// CTAs that an SM's registers are to hold, and the 16-byte units of a slot.
__host__ __device__ constexpr int distill_ctas(int warps) {
  return warps == 8 ? 4 : warps == 4 ? 7 : 16;
}
__host__ __device__ constexpr int distill_units(int warps) {
  return warps == 8 ? 4096 : warps * 256;
}
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

__device__ __forceinline__ void warp_join(float& m, float& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
}

// A row as units of 16 bytes: its first logit is entry `phase` of unit 0.
struct Row {
  const float* unit0;   // 16-byte aligned
  int phase, units;     // units that the row touches
  int full0, full1;     // units full0 .. full1 - 1 lie inside the row
};
__device__ __forceinline__ Row row_units(const float* p, int V) {
  Row r;
  r.phase = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3u);
  r.unit0 = p - r.phase;
  r.units = (r.phase + V + 3) / 4;
  r.full0 = r.phase ? 1 : 0;
  r.full1 = (r.phase + V) / 4;
  return r;
}

}  // namespace

// WARPS warps (and the teacher's) per CTA; a slot of shared memory holds a
// CTA's part of a row of up to distill_units() units. A row of more parts
// than there are slots is streamed twice, for its sum and for its gradient.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32 + 32, distill_ctas(WARPS))
    lin_distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int MAIN = WARPS * 32;
  __shared__ __align__(8) uint64_t bars[kSlots + 6];
  __shared__ float2 red[2][WARPS];
  __shared__ float2 stats[2][8];         // (m, s) of each CTA of the cluster, by the row's parity
  __shared__ float2 teacher[2];          // sum p (log2 p - z c); whether the row has an entry
  __shared__ volatile int abort;
  extern __shared__ float4 ring[];       // slots x tile units, then 2 x (ids, p, z)[KP]
  const int KP = (a.K + 3) & ~3;         // (whole groups of four, the last one padded with -1)
  int* const ids = reinterpret_cast<int*>(ring + a.slots * a.tile);
  float* const ps = reinterpret_cast<float*>(ids + 2 * KP);
  float* const zs = ps + 2 * KP;
  const int C = a.cluster, rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int V = (int)a.V;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = blockIdx.x / C, row_step = gridDim.x / C;
  const float c = kDLog2E / a.tau;       // base-2 exponent of a logit
  const uint32_t full = smem_u32(bars);                    // [kSlots] the copies
  const uint32_t stat_full = full + 8 * kSlots;           // [2] the cluster's (m, s)
  const uint32_t ent_full = stat_full + 16;                // [2] the teacher's entries
  const uint32_t ent_empty = ent_full + 16;                // [2]
  const WaitCtl ctl{a.timeout_ns, &abort, a.status};
  if (tid == 0) {
    abort = 0;
    for (int i = 0; i < kSlots; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(stat_full + 8 * i, (uint32_t)C);
      mbar_init(ent_full + 8 * i, 1);
      mbar_init(ent_empty + 8 * i, WARPS);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (C > 1) cluster_sync_all();   // the peers' barriers are ready

  if (warp == WARPS) {   // the teacher's entries of each row, one row ahead
    int it = 0;
    for (int64_t i = row0; i < a.M; i += row_step, ++it) {
      const int b = it & 1;
      if (it >= 2 && !warp_wait_phase(ent_empty + 8 * b, ((it >> 1) - 1) & 1, ctl)) return;
      int* id_b = ids + b * KP;
      float *p_b = ps + b * KP, *z_b = zs + b * KP;
      const float* row = a.logits + i * a.ld;
      float m = -INFINITY;
      if (lane < KP - a.K) id_b[a.K + lane] = -1;
#pragma unroll 4
      for (int k = lane; k < a.K; k += 32) {
        const int id = a.ids[i * a.K + k];
        const bool ok = id >= 0 && id < V;
        const float t = ok ? a.teacher[i * a.K + k] * c : -INFINITY;
        id_b[k] = ok ? id : -1;
        p_b[k] = t;
        z_b[k] = ok ? row[id] : 0.0f;
        m = fmaxf(m, t);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool any = m != -INFINITY;
      float s = 0.0f;
      for (int k = lane; k < a.K; k += 32) s += any ? ex2_approx(p_b[k] - m) : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float ls = log2f(s);
      float kl = 0.0f;
      for (int k = lane; k < a.K; k += 32) {
        const float lp = p_b[k] - m - ls;
        const float p = any ? ex2_approx(lp) : 0.0f;
        p_b[k] = p;
        if (p > 0.0f) kl += p * (lp - z_b[k] * c);   // (0 log 0 = 0)
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
      __syncwarp();
      // An entry listed twice: its first place takes all of its probability,
      // the others are marked (-2 - id, so that they are still told apart).
      auto entry = [](int id) { return id < -1 ? -2 - id : id; };
      bool twins = false;
      for (int k0 = 0; k0 < a.K; k0 += 32) {
        const int k = k0 + lane;
        const int id = k < a.K ? id_b[k] : -1;
        bool twin = false;
        for (int q = 0; q <= k0 + 28 && q < KP; q += 4) {
          const int4 o = *reinterpret_cast<const int4*>(id_b + q);
          twin = twin || (q < k && entry(o.x) == id) || (q + 1 < k && entry(o.y) == id) ||
                 (q + 2 < k && entry(o.z) == id) || (q + 3 < k && entry(o.w) == id);
        }
        __syncwarp();
        if (twin && id >= 0) {
          id_b[k] = -2 - id;
          twins = true;
        }
        __syncwarp();
      }
      if (__any_sync(0xffffffffu, twins)) {
        for (int k = lane; k < a.K; k += 32) {
          const int id = id_b[k];
          if (id < 0) continue;
          float p = p_b[k];
          for (int q = k + 1; q < a.K; ++q)
            if (id_b[q] == -2 - id) p += p_b[q];
          p_b[k] = p;   // (the marked places' own stay as they were)
        }
      }
      if (lane == 0) teacher[b] = make_float2(kl, any ? 1.0f : 0.0f);
      __syncwarp();
      if (lane == 0) mbar_arrive(ent_full + 8 * b);
    }
    return;
  }

  // The CTA's copies in the order of their use: the row's parts seg * C +
  // rank, once, or twice in a row for one that does not fit the slots.
  const int S = a.segs;
  const bool twice = S > a.slots;
  const int per_row = twice && a.dlogits ? 2 * S : S;
  int64_t load_row = row0;
  int load_job = 0, loads = 0, load_slot = 0;
  auto unit_begin = [&](int seg) { return (seg * C + rank) * a.tile; };
  auto issue = [&]() {   // (thread 0) the next copy into its slot
    if (load_row >= a.M) return;
    const int seg = load_job < S ? load_job : load_job - S;
    const Row r = row_units(a.logits + load_row * a.ld, V);
    const int u0 = unit_begin(seg);
    const int lo = max(u0, r.full0), hi = min(min(u0 + a.tile, r.units), r.full1);
    const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16u : 0u;
    mbar_arrive_expect_tx(full + 8 * load_slot, bytes);
    if (bytes)
      bulk_load(smem_u32(ring + load_slot * a.tile + (lo - u0)), r.unit0 + (int64_t)lo * 4, bytes,
                full + 8 * load_slot);
    ++loads;
    if (++load_slot == a.slots) load_slot = 0;
    if (++load_job == per_row) {
      load_job = 0;
      load_row += row_step;
    }
  };
  if (tid == 0)
    for (int i = 0; i < a.slots; ++i) issue();

  // Unit u of row r: entry u - u0 of a slot, or one by one if it is partial;
  // -inf outside the row.
  auto unit = [&](const Row& r, const float4* slot, int u, int u0, int u1) -> float4 {
    if (u >= u1) return make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (u >= r.full0 && u < r.full1) return slot[u - u0];
    float e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = 4 * u + j - r.phase;
      e[j] = v >= 0 && v < V ? r.unit0[4 * (int64_t)u + j] : -INFINITY;
    }
    return make_float4(e[0], e[1], e[2], e[3]);
  };
  int slot_i = 0, slot_round = 0;   // slot and round of the next copy to use
  auto next_slot = [&]() {
    if (++slot_i == a.slots) {
      slot_i = 0;
      slot_round ^= 1;
    }
  };

  int it = 0;   // rows done
  bool ok = true;
  for (int64_t i = row0; i < a.M && ok; i += row_step, ++it) {
    const int b = it & 1;
    const Row r = row_units(a.logits + i * a.ld, V);
    float m = -INFINITY, s = 0.0f;
    const int slot_first = slot_i, round_first = slot_round;
    for (int seg = 0; seg < S; ++seg) {
      ok = warp_wait_phase(full + 8 * slot_i, slot_round, ctl);
      if (!ok) break;
      const int u0 = unit_begin(seg), u1 = min(u0 + a.tile, r.units);
      const float4* slot = ring + slot_i * a.tile;
#pragma unroll 1
      for (int k = u0 + tid; k < u1; k += kChunk * MAIN) {
        float4 x[kChunk];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          x[j] = unit(r, slot, k + j * MAIN, u0, u1);
          mx = fmaxf(mx, fmaxf(fmaxf(x[j].x, x[j].y), fmaxf(x[j].z, x[j].w)));
        }
        mx *= c;
        const float shift = mx == -INFINITY ? 0.0f : -mx;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          t0 += ex2_approx(fmaf(x[j].x, c, shift)) + ex2_approx(fmaf(x[j].y, c, shift));
          t1 += ex2_approx(fmaf(x[j].z, c, shift)) + ex2_approx(fmaf(x[j].w, c, shift));
        }
        join(m, s, mx, t0 + t1);
      }
      next_slot();
      if (twice) {   // the slot is free again
        named_bar_sync(1, MAIN);
        if (tid == 0) issue();
      }
    }
    if (!ok) break;
    warp_join(m, s);
    if (lane == 0) red[b][warp] = make_float2(m, s);
    named_bar_sync(1, MAIN);
    if (!a.dlogits && !twice && tid == 0)   // (the losses alone: the row is done with)
      for (int seg = 0; seg < S; ++seg) issue();
    // every warp joins the warps' values by itself, in the same order
    m = lane < WARPS ? red[b][lane].x : -INFINITY;
    s = lane < WARPS ? red[b][lane].y : 0.0f;
    warp_join(m, s);
    // (before the exchange: a peer may overwrite the row behind it, and the
    // teacher's warp has read its logits by now)
    ok = warp_wait_phase(ent_full + 8 * b, (it >> 1) & 1, ctl);
    if (!ok) break;
    if (C > 1) {
      if (warp == 0 && lane < C) {
        const uint32_t to = mapa_shared(smem_u32(&stats[b][rank]), (uint32_t)lane);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
        mbar_arrive_remote(mapa_shared(stat_full + 8 * b, (uint32_t)lane));
      }
      ok = warp_wait_phase_cluster(stat_full + 8 * b, (it >> 1) & 1, ctl);
      if (!ok) break;
      m = stats[b][0].x;
      s = stats[b][0].y;
      for (int q = 1; q < C; ++q) join(m, s, stats[b][q].x, stats[b][q].y);
    }
    const float lse = m + log2f(s);   // base 2
    const bool any = teacher[b].y != 0.0f;
    if (rank == 0 && tid == 0)
      a.losses[i] = any ? a.tau * a.tau * kDLn2 * (teacher[b].x + lse) : 0.0f;
    if (a.dlogits) {
      float* out = a.dlogits + i * a.ldd;
      const float f = any ? a.tau * a.inv_norm : 0.0f;
      // 16-byte stores where the gradient's units lie as the logits' do
      const bool vec = (((reinterpret_cast<uintptr_t>(out) >> 2) - r.phase) & 3u) == 0;
      float* out0 = out - r.phase;
      if (!twice) {   // the same slots once more
        slot_i = slot_first;
        slot_round = round_first;
      }
      for (int seg = 0; seg < S; ++seg) {
        if (twice) {
          ok = warp_wait_phase(full + 8 * slot_i, slot_round, ctl);
          if (!ok) break;
        }
        const int u0 = unit_begin(seg), u1 = min(u0 + a.tile, r.units);
        const float4* slot = ring + slot_i * a.tile;
#pragma unroll 1
        for (int k = u0 + tid; k < u1; k += kChunk * MAIN) {
          float4 x[kChunk];
#pragma unroll
          for (int j = 0; j < kChunk; ++j) x[j] = unit(r, slot, k + j * MAIN, u0, u1);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) {
            const int u = k + j * MAIN;
            if (u >= u1) continue;
            float e[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) e[q] = any ? f * ex2_approx(fmaf(e[q], c, -lse)) : 0.0f;
            if (vec && u >= r.full0 && u < r.full1) {
              *reinterpret_cast<float4*>(out0 + 4 * (int64_t)u) = make_float4(e[0], e[1], e[2], e[3]);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int v = 4 * u + q - r.phase;
                if (v >= 0 && v < V) out[v] = e[q];
              }
            }
          }
        }
        next_slot();
        if (twice) {
          named_bar_sync(1, MAIN);
          if (tid == 0) issue();
        }
      }
      if (!ok) break;
      named_bar_sync(1, MAIN);   // the slots are read; the row's stores come before the entries'
      if (!twice && tid == 0)
        for (int seg = 0; seg < S; ++seg) issue();
      const int* id_b = ids + b * KP;
      const float *p_b = ps + b * KP, *z_b = zs + b * KP;
      if (any)
        for (int k = tid; k < a.K; k += MAIN) {
          const int id = id_b[k];
          if (id >= 0 && ((id + r.phase) / 4 / a.tile) % C == rank)
            out[id] = f * (ex2_approx(fmaf(z_b[k], c, -lse)) - p_b[k]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ent_empty + 8 * b);
  }
  // no copy may still be in flight when the CTA ends (only after a wait that
  // ran out: every copy is otherwise used)
  if (tid == 0 && abort)
    for (int k = max(0, loads - a.slots); k < loads; ++k)
      wait_phase(full + 8 * (k % a.slots), (k / a.slots) & 1, ctl, false);
}

// The sum of the losses in a fixed order: one CTA, a strided sum, then a tree.
__global__ void __launch_bounds__(1024)
    lin_sum_rows_kernel(const float* __restrict__ losses, int M, float* __restrict__ out) {
  __shared__ float part[32];
  pdl_wait();
  float v = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < M; i += 1024) v += __ldcg(losses + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = part[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x == 0) *out = v;
  }
}

namespace {

template <int WARPS>
cudaError_t launch_rows(DistillArgs a, int sms, cudaStream_t stream) {
  constexpr int kMax = distill_units(WARPS);
  // (a row of V logits touches at most (V + 6) / 4 units)
  const int64_t units = (a.V + 6) / 4;
  a.cluster = 1;
  while (a.cluster < 8 && (int64_t)a.cluster * kMax < units) a.cluster *= 2;
  const int64_t part = (units + a.cluster - 1) / a.cluster;
  a.segs = (int32_t)((part + kMax - 1) / kMax);
  a.tile = (int32_t)((part + a.segs - 1) / a.segs);
  // slots: what a row needs, and up to two more for the next rows' copies
  // where they cost no CTA of the SM
  const size_t entries = (size_t)((a.K + 3) & ~3) * 24, slot = (size_t)a.tile * 16;
  auto resident_ctas = [&](int slots) {
    return std::min<int64_t>(distill_ctas(WARPS), 225 * 1024 / (slots * slot + entries + 1536));
  };
  a.slots = std::min(a.segs, kSlots);
  while (a.slots < kSlots && resident_ctas(a.slots + 1) == resident_ctas(a.segs)) ++a.slots;
  const size_t smem = a.slots * slot + entries;
  auto kernel = lin_distill_kernel<WARPS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(WARPS * 32 + 32, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  // Clusters that run at once. The query takes longer than the launch, so its
  // last answer is kept for calls of the same sizes.
  struct Resident {
    int sms, cluster;
    size_t smem;
    int64_t n;
  };
  static thread_local Resident last{0, 0, 0, 0};
  if (last.sms != sms || last.cluster != a.cluster || last.smem != smem) {
    int n = 0;
    cfg.gridDim = dim3((unsigned)a.cluster, 1, 1);
    e = a.cluster > 1
            ? cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)
            : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, WARPS * 32 + 32, smem);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    last = Resident{sms, a.cluster, smem, a.cluster > 1 ? n : (int64_t)n * sms};
  }
  const int64_t resident = last.n;
  cfg.gridDim = dim3((unsigned)(std::min(resident, a.M) * a.cluster), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, float* loss_sum, int sms, cudaStream_t stream) {
  // Rows share an SM as far as they fit, so that the waits of one row are
  // filled by others: as few warps to a row as hold it.
  const int64_t units = (a.V + 6) / 4;
  cudaError_t e = units <= distill_units(1)   ? launch_rows<1>(a, sms, stream)
                  : units <= distill_units(4) ? launch_rows<4>(a, sms, stream)
                                              : launch_rows<8>(a, sms, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lin_sum_rows_kernel, (const float*)a.losses, (int)a.M, loss_sum);
}

}  // namespace lin
