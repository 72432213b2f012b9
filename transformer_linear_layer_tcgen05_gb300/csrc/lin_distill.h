// lin_distill.h -- launch interface of the distillation loss.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace lin {

constexpr int kSlots = 3;                // parts of a row in shared memory, at most
constexpr int kMaxCluster = 16;          // CTAs along a row
constexpr int kEnt = 3;                  // rows whose entries are held

// CTAs that an SM's registers are to hold, the 16-byte units of a slot, and a
// CTA's threads (the last warp has the teacher's entries).
constexpr int distill_ctas(int warps) {
  return warps == 8 ? 4 : warps == 4 ? 7 : warps == 2 ? 12 : 16;
}
constexpr int distill_units(int warps) { return warps == 8 ? 4096 : warps * 256; }
constexpr int distill_threads(int warps) { return (warps + 1) * 32; }

// Shared memory that a CTA may have, and what the kernel declares of it at most.
constexpr size_t kDistillSmem = 227 * 1024, kDistillStatic = 1024;

// How a row of `units` 16-byte units with K entries is laid out over CTAs of
// `warps` warps.
struct DistillLayout {
  int cluster;   // CTAs of a row
  int segs;      // parts of a row to each of them
  int tile;      // 16-byte units of a part
  int slots;     // parts that shared memory holds
  size_t smem;   // bytes: the slots, then the entries
};
inline DistillLayout distill_layout(int warps, int64_t units, int K) {
  const int most = distill_units(warps);
  DistillLayout d{};
  d.cluster = 1;
  while (d.cluster < kMaxCluster && (int64_t)d.cluster * most < units) d.cluster *= 2;
  const int64_t part = (units + d.cluster - 1) / d.cluster;
  d.segs = (int)((part + most - 1) / most);
  d.tile = (int)((part + d.segs - 1) / d.segs);
  // slots: what a row needs, and up to two more for the next rows' copies
  // where they cost no CTA of the SM
  const size_t entries = (size_t)((K + 3) & ~3) * 12 * kEnt, slot = (size_t)d.tile * 16;
  auto resident_ctas = [&](int slots) {
    return std::min<size_t>((size_t)distill_ctas(warps),
                            225 * 1024 / (slots * slot + entries + 2048));
  };
  d.slots = std::min(d.segs, kSlots);
  while (d.slots < kSlots && resident_ctas(d.slots + 1) == resident_ctas(d.segs)) ++d.slots;
  // Many entries leave room for two slots of 64 KB only; a row of more parts
  // is then streamed twice.
  while (d.slots > 1 && d.slots * slot + entries + kDistillStatic > kDistillSmem) --d.slots;
  d.smem = d.slots * slot + entries;
  return d;
}

struct DistillArgs {
  const float* logits;    // [M][ld]
  const int32_t* ids;     // [M][K]
  const float* teacher;   // [M][K]
  float* dlogits;         // [M][ldd], null: the losses alone
  float* losses;          // [M]
  int64_t M, V, ld, ldd;
  int32_t K;
  float tau, inv_norm;
  uint64_t timeout_ns;
  int* status;
  // set at launch: CTAs of a row, parts of a row to each of them, 16-byte
  // units of a part, parts that shared memory holds
  int32_t cluster, segs, tile, slots;
};

// The rows' losses and gradients, then the sum of the losses.
cudaError_t launch_distill(const DistillArgs& a, float* loss_sum, int sms, cudaStream_t stream);

}  // namespace lin
