// lin_attn.h -- launch interface of the attention kernels (host and device).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace lin {

// One [tokens][heads][dim] tensor of 16-bit entries, strides in entries.
struct HeadsPtr {
  uint16_t* p;
  int64_t token_stride, head_stride;
};

struct AttnArgs {
  const int32_t* cu_q;   // [sequences + 1] row offsets (null: one sequence)
  const int32_t* cu_k;
  int32_t tokens_q, tokens_k, max_q, max_k;
  int32_t heads_q, group, dim;   // group: query heads per key head
  int32_t causal;
  float scale;
  uint64_t timeout_ns;
  int* status;
};

struct AttnFwdArgs {
  AttnArgs s;
  HeadsPtr o;
  float* lse;   // [heads_q][tokens_q]
  // parts of the keys, and, where there are several, their results in f32:
  // [part][row][head][dim], [part][head][row], the rows of the sequences one
  // after another, max_q to each (part_rows in all; with at most half as many
  // CTAs as SMs, parts hold some million entries: 32-bit indices)
  int32_t parts, part_rows;
  float *o_part, *lse_part;
  // tiles of a CTA (1 or 2), query heads of a tile (1, or all that share a key
  // head), and its queries: 128 / pack
  int32_t tiles, pack, tile_q;
};

struct AttnBwdArgs {
  AttnArgs s;
  HeadsPtr q, k, v;       // the CTAs' own rows (the streamed ones come by the maps)
  HeadsPtr o, dout;
  const float* lse;       // [heads_q][tokens_q]
  float* delta;           // [heads_q][tokens_q]: sum of dO * O of each row
  float* norm;            // [sequences][heads_q >> shift][row tiles]: largest row norm of dO
  int64_t norms;          // (their number)
  HeadsPtr dq, dk, dv;
  // parts of the keys for dQ and of the queries for dK, dV, and, where there
  // are several, their f32 sums [part][row][head][dim], the rows of the
  // sequences one after another, max_q (max_k) to each
  int32_t q_parts, k_parts;
  int32_t q_part_rows, k_part_rows;
  // log2 of the query heads that are rows of one tile: 1, or all that share a
  // key head
  int32_t shift;
  float *dq_part, *dk_part, *dv_part;
};

struct AttnFwdMaps {
  CUtensorMap q, k, v;
};
struct AttnBwdMaps {
  CUtensorMap q, k, v, dout;
};

// Parts that the other side of a launch of `ctas` CTAs is cut into (`rows`: of
// the other side that the longest runs over).
int attn_parts(int64_t ctas, int64_t rows, int sms);
// One kernel; with several parts another one that joins them.
cudaError_t launch_attn_fwd(bool bf16, const AttnFwdMaps& maps, const AttnFwdArgs& args,
                            int heads_kv, int sequences, cudaStream_t stream);
// Tokens of a box of the backward kernels' maps.
constexpr int kAttnBwdBox = 64;
// The dQ kernel (which also leaves delta and norm), the dK, dV kernel, and the
// sums of their parts; *kernels: how many that were.
cudaError_t launch_attn_bwd(bool bf16, const AttnBwdMaps& maps, const AttnBwdArgs& args,
                            int heads_kv, int sequences, int* kernels, cudaStream_t stream);

}  // namespace lin
