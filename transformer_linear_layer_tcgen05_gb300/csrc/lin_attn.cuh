// lin_attn.cuh -- what the attention kernels share: tile geometry, the
// sequences' extents, operand descriptors and the 16-bit conversions.
//
// The kernels work in tiles of 128 queries x 128 keys. An operand tile is 128
// tokens of one head, [128 rows][64 entries] of 16 bits with the 128-byte
// swizzle, one such sub-tile for heads of up to 64 entries and two for up to
// 128 (entries past the head's size are zero-filled by the copy). Products
// run over 64, 96 or 128 entries: DP, the least that holds the head. The same
// tile serves as a K-major operand (the contraction runs over the entries: S
// = Q K^T, dP = dO V^T) and as an MN-major one (it runs over the tokens: P V,
// P^T dO, dS^T Q, dS K).
#pragma once

#include <cuda_bf16.h>

#include "lin_attn.h"
#include "lin_common.cuh"

namespace lin {

constexpr float kLog2E = 1.4426950408889634f;

constexpr int kAttnThreads = 320;   // 8 element-wise warps, 1 copying, 1 issuing products
constexpr int kAttnCopyWarp = 8;
constexpr int kAttnMmaWarp = 9;

// A place in a ring of N stages and the parity of its round.
template <int N>
struct RingAt {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      parity ^= 1;
    }
  }
};

// Waiting for a barrier. The kernels' loops are long and compete for the
// instruction caches, so what follows a failed first look stands out of line
// (heads of 128, 8192 tokens: forward 346 -> 333 us, backward 672 -> 645); a
// look may suspend its thread for a microsecond, which leaves issue slots and
// power to the warps at work (backward 645 -> 632; looks without any pause
// cost it 15 %).
constexpr uint32_t kAttnNapNs = 1000;
static __device__ __noinline__ bool attn_wait_on(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                                 volatile int* abort, int* status, bool honor_abort) {
  return wait_phase<kAttnNapNs>(bar, parity, WaitCtl{timeout_ns, abort, status}, honor_abort);
}
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, const WaitCtl& c,
                                          bool honor_abort = true) {
  return mbar_try_wait<kAttnNapNs>(bar, parity) ||
         attn_wait_on(bar, parity, c.timeout_ns, c.abort, c.status, honor_abort);
}
// Every lane waits; the warp goes on only if all of them saw the phase.
__device__ __forceinline__ bool warp_attn_wait(uint32_t bar, uint32_t parity, const WaitCtl& c) {
  const bool ok = attn_wait(bar, parity, c);
  return __all_sync(0xffffffffu, ok);
}

// Sequence b's first row and length in a packed tensor of `tokens` rows; the
// offsets come from device memory, so they are held inside the tensor and
// the length at `most` (the grid's extent).
struct SeqRange {
  int start, len;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* cu, int b, int tokens, int most) {
  if (!cu) return SeqRange{0, min(tokens, most)};
  const int s = min(max(cu[b], 0), tokens);
  const int e = min(max(cu[b + 1], s), tokens);
  return SeqRange{s, min(e - s, most)};
}

// The sequence and the part of a CTA whose grid has `parts` of them to each
// sequence, and the part's share of n turns.
struct PartOf {
  int b, part, parts;
  __device__ __forceinline__ int begin(int n) const {
    return parts == 1 ? 0 : (int)((int64_t)n * part / parts);
  }
  __device__ __forceinline__ int end(int n) const {
    return parts == 1 ? n : (int)((int64_t)n * (part + 1) / parts);
  }
};
__device__ __forceinline__ PartOf part_of(int z, int parts) {
  return parts == 1 ? PartOf{z, 0, 1} : PartOf{z / parts, z % parts, parts};
}

// Sub-tiles, bytes and descriptors of a [ROWS tokens][DP entries] operand
// tile. A descriptor's address field counts 16-byte units from bit 0, so the
// steps of a product add constants to the tile's descriptor.
template <int DP, int ROWS = 128>
struct AttnTile {
  static constexpr int SUB = (DP + 63) / 64;
  static constexpr uint32_t SUB_BYTES = ROWS * 128;
  static constexpr uint32_t BYTES = SUB * SUB_BYTES;
  static constexpr uint64_t UNITS = BYTES / 16;
  // K-major (steps of 16 entries), MN-major (steps of 16 tokens)
  static __device__ __forceinline__ uint64_t k_major(uint32_t tile) {
    return umma_desc_sw128(tile, 16, 1024);
  }
  static __device__ __forceinline__ uint64_t mn_major(uint32_t tile) {
    return umma_desc_sw128(tile, SUB_BYTES, 1024);
  }
  static constexpr uint64_t entry_step(int kk) {
    return (uint64_t)((kk >> 2) * SUB_BYTES + (kk & 3) * 32) / 16;
  }
  static constexpr uint64_t token_step(int kk) { return (uint64_t)kk * 2048 / 16; }
};

template <bool BF16, bool B_MN, int N>
__host__ __device__ constexpr uint32_t attn_idesc() {
  return umma_idesc(BF16 ? 1u : 0u, false, B_MN, 128, N);
}

// Two values rounded to nearest even in the tensors' 16-bit type, the first
// in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_half2(lo, hi);
  }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

// D[128 x ROWS] = A B^T over the DP entries of two operand tiles, A of 128
// tokens, B of ROWS (K-major descriptors).
template <int DP, bool BF16, int ROWS = 128>
__device__ __forceinline__ void umma_entries(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t idesc = attn_idesc<BF16, false, ROWS>();
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk)
    umma_f16(d, a + AttnTile<DP>::entry_step(kk), b + AttnTile<DP, ROWS>::entry_step(kk), idesc,
             kk > 0);
}

// The same with A's 128 rows in tensor memory (entries 2c, 2c + 1 in column c).
template <int DP, int ROWS, bool BF16>
__device__ __forceinline__ void umma_entries_tmem(uint32_t d, uint32_t a, uint64_t b) {
  constexpr uint32_t idesc = attn_idesc<BF16, false, ROWS>();
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk)
    umma_f16_tmem_a(d, a + kk * 8, b + AttnTile<DP, ROWS>::entry_step(kk), idesc, kk > 0);
}

// D[128 x DP] (+)= A B over 16 STEPS tokens from token 16 `from` of an operand
// tile B (MN-major descriptor); A in tensor memory, these tokens in the 8
// STEPS columns at `a`. `first`: the accumulator starts here.
template <int DP, bool BF16, int STEPS>
__device__ __forceinline__ void umma_tokens(uint32_t d, uint32_t a, uint64_t b, int from, bool first) {
  constexpr uint32_t idesc = attn_idesc<BF16, true, DP>();
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk)
    umma_f16_tmem_a(d, a + kk * 8, b + AttnTile<DP>::token_step(from + kk), idesc, kk > 0 || !first);
}

// Zeroes rows [first, last) of an operand tile: a contraction over tokens must
// not meet what lies behind a sequence's end (another sequence's rows, or
// padding), nor rows that a causal mask leaves no key: they may hold infinities
// or NaN, which a zero weight would not remove. One warp, after the copy has
// landed; a fence then orders the stores before the tensor core's reads.
template <int DP, int ROWS>
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int last, int lane) {
  for (int s = 0; s < AttnTile<DP, ROWS>::SUB; ++s)
    for (int i = first * 8 + lane; i < last * 8; i += 32)
      st_shared_v4(tile + s * AttnTile<DP, ROWS>::SUB_BYTES + i * 16, 0u, 0u, 0u, 0u);
}

// One operand tile (tokens z .. z + ROWS - 1 of head h; the map's box has as
// many) into shared memory.
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int h, int z,
                                          uint32_t bar) {
#pragma unroll
  for (int s = 0; s < AttnTile<DP, ROWS>::SUB; ++s)
    tma_load_3d(dst + s * AttnTile<DP, ROWS>::SUB_BYTES, map, s * 64, h, z, bar);
}

// Part `part` of PARTS of a head's row (null: zeros) in registers, two entries
// to each: zero behind the head's size.
template <int DP, int PARTS>
__device__ __forceinline__ void load_row_part(uint32_t (&r)[DP / PARTS / 2], const uint16_t* row,
                                              int part, int dim) {
#pragma unroll
  for (int e = 0; e < DP / PARTS / 8; ++e) {
    const int col = part * (DP / PARTS) + e * 8;
    const uint4 x = row && col < dim ? __ldg(reinterpret_cast<const uint4*>(row + col))
                                     : make_uint4(0u, 0u, 0u, 0u);
    r[e * 4] = x.x;
    r[e * 4 + 1] = x.y;
    r[e * 4 + 2] = x.z;
    r[e * 4 + 3] = x.w;
  }
}

// Checked build: row `token` (of the keys or the queries) and head h inside
// their tensor; a place of the ring inside it.
__device__ __forceinline__ bool q_row_ok(const AttnArgs& a, int64_t token, int h) {
  return dcheck(token >= 0 && token < a.tokens_q && h >= 0 && h < a.heads_q, a.status, CHK_GLOBAL,
                token);
}
__device__ __forceinline__ bool k_row_ok(const AttnArgs& a, int64_t token, int h) {
  return dcheck(token >= 0 && token < a.tokens_k && h >= 0 && h < a.heads_q / a.group, a.status,
                CHK_GLOBAL, token);
}
__device__ __forceinline__ bool stage_ok(const AttnArgs& a, int s, int stages) {
  return dcheck(s >= 0 && s < stages, a.status, CHK_STAGE, s);
}

// Eight 16-bit entries of a row to global memory.
__device__ __forceinline__ void store16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

}  // namespace lin
