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

// A form of the scores: z = cap tanh(scale s / cap) - slope |distance| (cap 0:
// scale s; slopes null: no bias), and the keys first .. end - 1 of a query,
// counted in its sequence (null: from the first, to the last).
constexpr int kTanhTerms = 5, kFewTerms = 3;
constexpr int kNoForm = -1, kCap = 1, kBias = 2;   // (forms of ranges alone: 0)
struct ScoreForm {
  float cap;
  const float* slopes;             // [heads_q]
  const int32_t *first, *end;      // [tokens_q]
  // (a cap, forward) tanh's polynomials of few and of more terms as those of
  // products q k in z log2 e, twice each, for two at a time, and how large a
  // product they take (below zero: none)
  float few_up_to, up_to;
  float2 few[kFewTerms], terms[kTanhTerms];
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
  ScoreForm scores;
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
  ScoreForm scores;
  int2* extents;          // as norm: the keys that a tile's rows see (ranges of keys; null: none)
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
// One kernel for a form of the scores (kNoForm, or kCap and kBias, or 0); and,
// with several parts, another one that joins them.
template <int FORM>
cudaError_t launch_attn_fwd(bool bf16, const AttnFwdMaps& maps, const AttnFwdArgs& args,
                            int heads_kv, int sequences, cudaStream_t stream);
cudaError_t launch_attn_join_parts(bool bf16, const AttnFwdArgs& args, int heads, int sequences,
                                   cudaStream_t stream);
// Tokens of a box of the backward kernels' maps.
constexpr int kAttnBwdBox = 64;
// The dQ kernel (which also leaves delta and norm) and the dK, dV kernel for a
// form of the scores, and the sums of their parts; *kernels: how many that were.
template <int FORM>
cudaError_t launch_attn_bwd(bool bf16, const AttnBwdMaps& maps, const AttnBwdArgs& args,
                            int heads_kv, int sequences, int* kernels, cudaStream_t stream);
cudaError_t launch_attn_sum_parts(bool bf16, const AttnBwdArgs& args, int heads_kv, int sequences,
                                  int* kernels, cudaStream_t stream);

}  // namespace lin
