// lin_distill.cu -- distillation from a teacher's top logits: per row,
//   q = softmax(z / tau) over the vocabulary, p = softmax(t / tau) over the
//   row's listed entries,  loss = tau^2 sum_k p_k (log p_k - log q_id(k)),
//   dz = tau (q - p) inv_norm.
//
// Bound by memory: 4 bytes read and, with the gradient, 4 written per logit.
// Persistent CTAs (clusters of up to 16 along a long row) walk over the rows.
// Bulk copies bring a CTA's part of the coming rows into a ring of slots in
// shared memory, from where a row is read twice: for the maximum and the sum
// of exponentials, the CTA's and the cluster's (through distributed shared
// memory), and for the gradient, written straight out. The gradient comes one
// row later than the sums, so that the exchange between the CTAs, whose
// latency is near the time of a whole row, stands in nobody's way. A warp of
// its own prepares the teacher's entries ahead, since their two dependent
// loads (id, then its logit) would do the same; their places in dz are
// written again, behind the row, with p taken off.
//
// Logits enter as differences, from the row's maximum, the teacher's largest
// and the largest listed one, before they are multiplied by log2 e / tau.
//
// Measured: 4096 rows of 131072 with the gradient 760 us, 5.7 TB/s (floor 641);
// 512 rows of 16384 17.0 us (10.0); 1000 rows of 50001, the losses alone, 40
// us, 5.0 TB/s (29.9). On the way there: a row by one CTA of 16 warps 3278 us
// at 131072 entries (each warp's fixed work for a row), clusters of 16 CTAs
// with slots of 32 KB 1167 and of 8 with 64 KB 937 (the exchange waited for),
// the same with the gradient a row behind 745, and with every wait's end told
// from its running out 760.
//
// A row is handled in the 16-byte units of memory that it touches, so rows
// may start anywhere: only the first and the last unit can be partial, and
// their entries are loaded one by one.
#include "lin_common.cuh"
#include "lin_distill.h"

#include <algorithm>

namespace lin {

namespace {

constexpr int kExch = 4;                 // rows whose exchange may be under way (a peer is at
                                         // most three ahead)
constexpr int kRed = 3;                  // rows whose warps' (m, s) are held: a warp may write the
                                         // next row's while another reads the one before last, and
                                         // only the barrier between two rows' writes parts them
constexpr int kChunk = 4;                // 16-byte units of a thread in registers at once
constexpr float kDLog2E = 1.4426950408889634f;
constexpr float kDLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e+38f;

// (m, s): maximum of x and sum of 2^((x - m) c), joined over the warp's lanes.
// m starts at the type's lowest value, not at -inf, so that a difference of
// maxima is always a number.
__device__ __forceinline__ void warp_join(float& m, float& s, float c) {
  float mx = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  s *= ex2_approx((m - mx) * c);
  m = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
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

// WARPS warps (and one for the teacher's entries) per CTA; a slot of shared memory holds a
// CTA's part of a row of up to distill_units() units. A row of more parts
// than there are slots is streamed twice, for its sum and for its gradient.
template <int WARPS>
__global__ void __launch_bounds__(distill_threads(WARPS), distill_ctas(WARPS))
    lin_distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int MAIN = WARPS * 32;
  constexpr int BARS = kSlots + kExch + 2 * kEnt;
  static_assert(BARS * 8 + kRed * WARPS * 8 + kExch * kMaxCluster * 8 + kEnt * 16 + 16 <=
                    (int)kDistillStatic, "shared memory beside the slots");
  __shared__ __align__(8) uint64_t bars[BARS];
  __shared__ float2 red[kRed][WARPS];   // (m, s) of each warp
  __shared__ float2 stats[kExch][kMaxCluster];   // (m, s) of each CTA of the cluster
  __shared__ float4 teacher[kEnt];       // sum p log2 p, sum p (z - w), whether the row has an entry, w
  __shared__ volatile int abort;
  extern __shared__ float4 ring[];       // slots x tile units, then kEnt x (ids, p, z)[KP]
  const int KP = (a.K + 3) & ~3;         // (whole groups of four, the last one padded with -1)
#if LIN_DEVICE_CHECKS
  {   // the slots and the entries inside what the launch gave
    uint32_t given;
    asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(given));
    const int64_t want = (int64_t)a.slots * a.tile * 16 + (int64_t)kEnt * KP * 12;
    if (!dcheck(want <= given && a.slots >= 1 && a.slots <= kSlots && a.cluster <= kMaxCluster, a.status,
                CHK_BUFFER, want))
      return;   // (every thread of every CTA)
  }
#endif
  int* const ids = reinterpret_cast<int*>(ring + a.slots * a.tile);
  float* const ps = reinterpret_cast<float*>(ids + kEnt * KP);
  float* const zs = ps + kEnt * KP;
  const int C = a.cluster, rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int V = (int)a.V;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = blockIdx.x / C, row_step = gridDim.x / C;
  const float c = kDLog2E / a.tau;       // base-2 exponent of a logit
  const uint32_t full = smem_u32(bars);                    // [kSlots] the copies
  const uint32_t stat_full = full + 8 * kSlots;            // [kExch] the cluster's (m, s)
  const uint32_t ent_full = stat_full + 8 * kExch;         // [kEnt] the teacher's entries
  const uint32_t ent_empty = ent_full + 8 * kEnt;          // [kEnt]
  const WaitCtl ctl{a.timeout_ns, &abort, a.status};
  if (tid == 0) {
    abort = 0;
    for (int i = 0; i < kSlots; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < kExch; ++i) mbar_init(stat_full + 8 * i, (uint32_t)C);
    for (int i = 0; i < kEnt; ++i) {
      mbar_init(ent_full + 8 * i, 1);
      mbar_init(ent_empty + 8 * i, WARPS);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (C > 1) cluster_sync_all();   // the peers' barriers are ready
  pdl_launch_dependents();         // (the sum of the losses waits for this grid's end)

  if (warp == WARPS) {   // the teacher's entries of each row
    // (the first 32 are loaded a row ahead of their use)
    int id_next = -1;
    float t_next = 0.0f;
    auto prefetch = [&](int64_t i) {
      if (i < a.M && lane < a.K) {
        id_next = a.ids[i * a.K + lane];
        t_next = a.teacher[i * a.K + lane];
      }
    };
    prefetch(row0);
    int it = 0;
    for (int64_t i = row0; i < a.M; i += row_step, ++it) {
      const int b = it % kEnt;
      const int id_first = id_next;
      const float t_first = t_next;
      prefetch(i + row_step);
      if (it >= kEnt) {
        // (this warp is rows ahead: it leaves the issue slots to the others
        // while it waits, for about a limit's time at most)
        int64_t naps = (int64_t)(a.timeout_ns / 200);
        while (!mbar_try_wait(ent_empty + 8 * b, (it / kEnt - 1) & 1)) {
          if (abort || --naps < 0) return;
          __nanosleep(200);
        }
        __syncwarp();
      }
      int* id_b = ids + b * KP;
      float *p_b = ps + b * KP, *z_b = zs + b * KP;
      const float* row = a.logits + i * a.ld;
      const int phase = row_units(row, V).phase;
      float m = -INFINITY, ref = -INFINITY;
      bool has = false;   // an entry: not -inf (a NaN is one, which the maximum passes over)
      if (lane < KP - a.K) id_b[a.K + lane] = -1;
#pragma unroll 4
      for (int k = lane; k < a.K; k += 32) {
        const int id = k < 32 ? id_first : a.ids[i * a.K + k];
        const bool ok = id >= 0 && id < V;
        const float t = ok ? (k < 32 ? t_first : a.teacher[i * a.K + k]) : -INFINITY;
        p_b[k] = t;
        // (the loss, by rank 0, needs every entry's logit; the gradient those
        // of the CTA's own part)
        const bool mine = ok && (C == 1 || ((id + phase) / 4 / a.tile) % C == rank);
        id_b[k] = mine ? id : -1;
        const float z = mine || (ok && rank == 0) ? row[id] : -INFINITY;
        z_b[k] = z;
        ref = fmaxf(ref, z);
        has = has || !(t == -INFINITY);
        m = fmaxf(m, t);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      }
      // Both sides' logits enter as differences (from the largest of the
      // teacher's, and of the row's listed ones), before anything is rounded:
      // what they have in common costs no accuracy.
      if (!(fabsf(ref) < INFINITY)) ref = 0.0f;
      const bool any = __any_sync(0xffffffffu, has);
      float s = 0.0f;
      for (int k = lane; k < a.K; k += 32) s += any ? ex2_approx((p_b[k] - m) * c) : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float ls = log2f(s);
      float plp = 0.0f, pz = 0.0f;
      for (int k = lane; k < a.K; k += 32) {
        const float lp = fmaf(p_b[k] - m, c, -ls);
        const float p = p_b[k] == -INFINITY ? 0.0f : ex2_approx(lp);
        p_b[k] = p;
        if (!(p == 0.0f)) {   // (0 log 0 = 0; a NaN counts)
          plp = fmaf(p, lp, plp);
          pz = fmaf(p, z_b[k] - ref, pz);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        plp += __shfl_xor_sync(0xffffffffu, plp, o);
        pz += __shfl_xor_sync(0xffffffffu, pz, o);
      }
      __syncwarp();
      // An entry listed twice: its first place takes all of its probability,
      // the others are marked (-2 - id).
      uint32_t twin_at = 0;   // the lane's places k0 + lane that have an equal before them
      for (int k0 = 0; k0 < a.K; k0 += 32) {
        const int id = k0 + lane < a.K ? id_b[k0 + lane] : -1;
        bool twin = (__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1u)) != 0;
#pragma unroll 4
        for (int q = 0; q < k0; q += 4) {
          const int4 o = *reinterpret_cast<const int4*>(id_b + q);
          twin = twin || o.x == id || o.y == id || o.z == id || o.w == id;
        }
        if (twin && id >= 0) twin_at |= 1u << (k0 >> 5);
      }
      __syncwarp();
      const bool twins = twin_at != 0;
      for (int k = lane; twin_at != 0; k += 32, twin_at >>= 1)
        if (twin_at & 1u) id_b[k] = -2 - id_b[k];
      __syncwarp();
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
      if (lane == 0) teacher[b] = make_float4(plp, pz, any ? 1.0f : 0.0f, ref);
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
  // Checked build: units lo .. hi - 1 inside the row and the part that begins
  // at u0, the slot inside the ring.
  auto units_ok = [&](const Row& r, int u0, int lo, int hi, int slot) -> bool {
    return dcheck(lo >= u0 && hi - u0 <= a.tile && 4 * (int64_t)lo >= r.phase &&
                      4 * (int64_t)hi - r.phase <= V, a.status, CHK_GLOBAL, lo) &&
           dcheck(slot >= 0 && slot < a.slots, a.status, CHK_STAGE, slot);
  };
  auto issue = [&]() {   // (thread 0) the next copy into its slot
    if (load_row >= a.M) return;
    const int seg = load_job < S ? load_job : load_job - S;
    const Row r = row_units(a.logits + load_row * a.ld, V);
    const int u0 = unit_begin(seg);
    const int lo = max(u0, r.full0), hi = min(min(u0 + a.tile, r.units), r.full1);
    const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16u : 0u;
    mbar_arrive_expect_tx(full + 8 * load_slot, bytes);
    if (bytes && units_ok(r, u0, lo, hi, load_slot))
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

  // The row's entries outside its whole units (at most three before, three
  // behind) that are in units u0 .. u1 - 1: lanes 0 .. 3 and 4 .. 7 of warp 0
  // have one each; -1: none.
  auto edge_entry = [&](const Row& r, int u0, int u1) -> int {
    if (warp != 0 || lane >= 8) return -1;
    int v;
    if (lane < 4) {   // in unit 0
      if (r.phase == 0 || u0 > 0 || u1 < 1) return -1;
      v = lane - r.phase;
    } else {          // in the last unit
      if (r.full1 < r.full0 || r.full1 >= r.units || r.full1 < u0 || r.full1 >= u1) return -1;
      v = 4 * r.full1 + (lane - 4) - r.phase;
    }
    return v >= 0 && v < V ? v : -1;
  };
  // The slot of the next copy to use, for the sums and for the gradients (one
  // after the other from the same one where a row is streamed twice).
  struct Cursor {
    int slot, parity;
  };
  Cursor at_sums{0, 0}, at_grad{0, 0};
  auto wait_copy = [&](const Cursor& q) {
    return warp_wait_phase(full + 8 * q.slot, (uint32_t)q.parity, ctl);
  };
  auto advance = [&](Cursor& q) {
    if (++q.slot == a.slots) {
      q.slot = 0;
      q.parity ^= 1;
    }
  };

  // False for a warp after a wait that ran out: it then waits, reads and
  // writes no more, but still goes through the rows, since the warps meet at
  // barriers that have no limit of their own.
  bool ok = true;

  // Row `it` of the CTA: maximum and sum of its part, sent to the cluster.
  auto sums = [&](int it, int64_t i) {
    const float* row = a.logits + i * a.ld;
    const Row r = row_units(row, V);
    float m = kLowest, s = 0.0f;
    for (int seg = 0; seg < S; ++seg) {
      ok = ok && wait_copy(at_sums);
      const int u0 = unit_begin(seg), u1 = min(u0 + a.tile, r.units);
      const int lo = max(u0, r.full0);
      int hi = ok ? min(u1, r.full1) : 0;
      if (hi > lo && !units_ok(r, u0, lo, hi, at_sums.slot)) hi = 0;
      const float4* slot = ring + at_sums.slot * a.tile - u0;
      auto add = [&](const float4* x, int count) {   // (count: a constant)
        float mx = m;
#pragma unroll
        for (int j = 0; j < count; ++j)
          mx = fmaxf(mx, fmaxf(fmaxf(x[j].x, x[j].y), fmaxf(x[j].z, x[j].w)));
        const float2 low = make_float2(-mx, -mx), cc = make_float2(c, c);
        float2 t0 = make_float2(s * ex2_approx((m - mx) * c), 0.0f), t1 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < count; ++j) {
          const float2 u = mul2(add2(make_float2(x[j].x, x[j].y), low), cc);
          const float2 v = mul2(add2(make_float2(x[j].z, x[j].w), low), cc);
          t0 = add2(t0, make_float2(ex2_approx(u.x), ex2_approx(u.y)));
          t1 = add2(t1, make_float2(ex2_approx(v.x), ex2_approx(v.y)));
        }
        t0 = add2(t0, t1);
        m = mx;
        s = t0.x + t0.y;
      };
      int k = lo + tid;
      for (; k + (kChunk - 1) * MAIN < hi; k += kChunk * MAIN) {
        float4 x[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) x[j] = slot[k + j * MAIN];
        add(x, kChunk);
      }
      for (; k < hi; k += MAIN) {
        const float4 x = slot[k];
        add(&x, 1);
      }
      const int v = edge_entry(r, u0, u1);
      if (v >= 0) {
        const float x = row[v], mx = fmaxf(m, x);
        s = s * ex2_approx((m - mx) * c) + ex2_approx((x - mx) * c);
        m = mx;
      }
      advance(at_sums);
      if (twice) {   // the slot is free again
        named_bar_sync(1, MAIN);
        if (tid == 0 && ok) issue();
      }
    }
    warp_join(m, s, c);
    if (lane == 0) red[it % kRed][warp] = make_float2(m, s);
    named_bar_sync(1, MAIN);
    if (!a.dlogits && !twice && tid == 0 && ok)   // (the losses alone: the row is done with)
      for (int seg = 0; seg < S; ++seg) issue();
    if (C > 1 && warp == 0) {
      // (before the exchange: a peer may overwrite the row behind it, and
      // this CTA's teacher warp has to have read its logits by then)
      ok = ok && warp_wait_phase(ent_full + 8 * (it % kEnt), (it / kEnt) & 1, ctl);
      m = lane < WARPS ? red[it % kRed][lane].x : kLowest;
      s = lane < WARPS ? red[it % kRed][lane].y : 0.0f;
      warp_join(m, s, c);
      if (lane < C && ok && dcheck(rank < kMaxCluster, a.status, CHK_PEER, rank)) {
        const int e = it % kExch;
        const uint32_t to = mapa_shared(smem_u32(&stats[e][rank]), (uint32_t)lane);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
        mbar_arrive_remote(mapa_shared(stat_full + 8 * e, (uint32_t)lane));
      }
    }
  };

  // Row `it`: its loss and gradient.
  auto finish = [&](int it, int64_t i) {
    const int b = it % kEnt;
    ok = ok && warp_wait_phase(ent_full + 8 * b, (it / kEnt) & 1, ctl);
    float m, s;
    if (C > 1) {
      const int e = it % kExch;
      ok = ok && warp_wait_phase_cluster(stat_full + 8 * e, (it / kExch) & 1, ctl);
      m = lane < C ? stats[e][lane].x : kLowest;
      s = lane < C ? stats[e][lane].y : 0.0f;
    } else {
      m = lane < WARPS ? red[it % kRed][lane].x : kLowest;
      s = lane < WARPS ? red[it % kRed][lane].y : 0.0f;
    }
    warp_join(m, s, c);   // (each warp by itself, in the same order)
    const float ls = log2f(s);   // the row's log-sum-exp less its maximum, base 2
    const float4 tp = teacher[b];
    const bool any = tp.z != 0.0f;
    if (rank == 0 && tid == 0 && ok && dcheck(i >= 0 && i < a.M, a.status, CHK_GLOBAL, i))
      a.losses[i] = any ? a.tau * a.tau * kDLn2 * (tp.x - (tp.y + (tp.w - m)) * c + ls) : 0.0f;
    if (a.dlogits) {
      const float* row = a.logits + i * a.ld;
      const Row r = row_units(row, V);
      float* out = a.dlogits + i * a.ldd;
      const float f = any ? a.tau * a.inv_norm : 0.0f;
      // 16-byte stores where the gradient's units lie as the logits' do
      const bool vec = (((reinterpret_cast<uintptr_t>(out) >> 2) - r.phase) & 3u) == 0;
      float* out0 = out - r.phase;
      for (int seg = 0; seg < S; ++seg) {
        Cursor& at = twice ? at_sums : at_grad;
        if (twice) ok = ok && wait_copy(at);
        const int u0 = unit_begin(seg), u1 = min(u0 + a.tile, r.units);
        const int lo = max(u0, r.full0);
        int hi = ok ? min(u1, r.full1) : 0;
        if (hi > lo && !units_ok(r, u0, lo, hi, at.slot)) hi = 0;
        const float4* slot = ring + at.slot * a.tile - u0;
        const int ve = ok ? edge_entry(r, u0, u1) : -1;
        const float edge = ve >= 0 ? row[ve] : 0.0f;   // (before it may be overwritten)
        auto grad = [&](float x) { return f * ex2_approx(fmaf(x - m, c, -ls)); };
        const float2 low = make_float2(-m, -m), cc = make_float2(c, c), ll = make_float2(-ls, -ls),
                     ff = make_float2(f, f);
        auto put = [&](int u, const float4& x) {
          const float2 p = fma2(add2(make_float2(x.x, x.y), low), cc, ll);
          const float2 q = fma2(add2(make_float2(x.z, x.w), low), cc, ll);
          const float2 g = mul2(make_float2(ex2_approx(p.x), ex2_approx(p.y)), ff);
          const float2 h = mul2(make_float2(ex2_approx(q.x), ex2_approx(q.y)), ff);
          float4 y = make_float4(g.x, g.y, h.x, h.y);
          if (!any) y = make_float4(0.f, 0.f, 0.f, 0.f);   // (whatever the logits hold)
          float* o = out0 + 4 * (int64_t)u;
          if (vec) {
            __stcs(reinterpret_cast<float4*>(o), y);
          } else {
            o[0] = y.x;
            o[1] = y.y;
            o[2] = y.z;
            o[3] = y.w;
          }
        };
        int k = lo + tid;
        for (; k + (kChunk - 1) * MAIN < hi; k += kChunk * MAIN) {
          float4 x[kChunk];
#pragma unroll
          for (int j = 0; j < kChunk; ++j) x[j] = slot[k + j * MAIN];
#pragma unroll
          for (int j = 0; j < kChunk; ++j) put(k + j * MAIN, x[j]);
        }
        for (; k < hi; k += MAIN) put(k, slot[k]);
        if (ve >= 0) out[ve] = any ? grad(edge) : 0.0f;
        advance(at);
        if (twice) {
          named_bar_sync(1, MAIN);
          if (tid == 0 && ok) issue();
        }
      }
      named_bar_sync(1, MAIN);   // the slots are read; the row's stores come before the entries'
      if (!twice && tid == 0 && ok)
        for (int seg = 0; seg < S; ++seg) issue();
      const int* id_b = ids + b * KP;
      const float *p_b = ps + b * KP, *z_b = zs + b * KP;
      if (any && ok)
        for (int k = tid; k < a.K; k += MAIN) {
          const int id = id_b[k];
          if (id >= 0 && dcheck(id < V, a.status, CHK_GLOBAL, id))
            out[id] = f * (ex2_approx(fmaf(z_b[k] - m, c, -ls)) - p_b[k]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ent_empty + 8 * b);
  };

  // The gradient one row behind the sums where the slots hold two rows' parts
  // (the losses alone: always), else right behind them.
  const int delay = a.dlogits && a.slots < 2 * S ? 0 : 1;
  const int rows = row0 < a.M ? (int)((a.M - row0 + row_step - 1) / row_step) : 0;
  for (int it = 0; it < rows + delay; ++it) {
    if (it < rows) sums(it, row0 + it * row_step);
    if (it >= delay) finish(it - delay, row0 + (it - delay) * row_step);
  }
  // no copy may still be in flight when the CTA ends (only after a wait that
  // ran out: every copy is otherwise used)
  if (tid == 0 && abort)
    for (int k = max(0, loads - a.slots); k < loads; ++k)
      wait_phase(full + 8 * (k % a.slots), (k / a.slots) & 1, ctl, false);
  // and its shared memory stays while a peer may still write to it
  if (C > 1 && __any_sync(0xffffffffu, abort)) cluster_sync_all();
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
cudaError_t launch_rows(DistillArgs a, int64_t units, int sms, cudaStream_t stream) {
  const DistillLayout d = distill_layout(WARPS, units, a.K);
  a.cluster = d.cluster;
  a.segs = d.segs;
  a.tile = d.tile;
  a.slots = d.slots;
  const size_t smem = d.smem;
  auto kernel = lin_distill_kernel<WARPS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e == cudaSuccess && a.cluster > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(distill_threads(WARPS), 1, 1);
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
            : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, distill_threads(WARPS), smem);
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
  // 16-byte units that a row touches: V / 4 where every row starts on one
  const bool whole = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0;
  const int64_t units = whole ? (a.V + 3) / 4 : (a.V + 6) / 4;
  // Rows share an SM as far as they fit, so that the waits of one row are
  // filled by others: as few warps to a row as hold it (16384 rows of 2048 by
  // two warps 56 us, by four 72; of 8000 by eight 174, by four in clusters of
  // two 221; more CTAs of one or two warps to an SM would spill: 16384 rows of
  // 1000 45 us in 16 CTAs, 50 in 20).
  cudaError_t e = units <= distill_units(1)   ? launch_rows<1>(a, units, sms, stream)
                  : units <= distill_units(2) ? launch_rows<2>(a, units, sms, stream)
                  : units <= distill_units(4) ? launch_rows<4>(a, units, sms, stream)
                                              : launch_rows<8>(a, units, sms, stream);
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
