// lin_attn_api.cu -- the attention entry points of include/lin.h: checks of
// the arguments, tensor maps, workspace and launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "lin.h"
#include "lin_attn.h"
#include "lin_heads.h"
#include "lin_internal.h"

namespace lin_detail {

namespace {

struct Checked {
  int dev;
  int* word;
  int64_t max_q, max_k;
  bool nothing;   // nothing to compute
};

// The checks that both directions share. `views`: every tensor of the call;
// `lse` is read (backward) or written (forward).
lin_status check_attention(const lin_attention_shape* s, View* views, int nviews, const float* lse,
                           bool lse_out, Checked* got) {
  got->nothing = false;
  if (!s) return LIN_ERROR_INVALID_VALUE;
  for (int i = 0; i < nviews; ++i)
    if (!views[i].t) return LIN_ERROR_INVALID_VALUE;
  if (s->dtype != LIN_BINARY16 && s->dtype != LIN_BFLOAT16) return LIN_ERROR_INVALID_VALUE;
  if (s->tokens_q < 0 || s->tokens_k < 0 || s->sequences < 0 || s->max_q < 0 || s->max_k < 0 ||
      s->heads_q < 1 || s->heads_kv < 1 || s->dim < 1)
    return LIN_ERROR_INVALID_VALUE;
  if (!(s->scale > 0.0f) || std::isinf(s->scale)) return LIN_ERROR_INVALID_VALUE;
  if ((!s->cu_q || !s->cu_k) && s->sequences != 1) return LIN_ERROR_INVALID_VALUE;
  if (s->tokens_q > kMaxExtent || s->tokens_k > kMaxExtent || s->sequences > 65535 ||
      s->heads_q > kMaxExtent / 65536 || s->heads_kv > s->heads_q ||
      s->heads_q % s->heads_kv != 0 || s->dim % 8 != 0 || s->dim > 128)
    return LIN_ERROR_UNSUPPORTED_SHAPE;
  got->max_q = s->cu_q ? std::min(s->max_q, s->tokens_q) : s->tokens_q;
  got->max_k = s->cu_k ? std::min(s->max_k, s->tokens_k) : s->tokens_k;
  if (got->max_q > 65535LL * 128 || got->max_k > 65535LL * 128) return LIN_ERROR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < nviews; ++i) {
    views[i].tokens = views[i].tokens < 0 ? s->tokens_k : s->tokens_q;   // (-1: of the keys)
    const lin_status st = check_view(views[i], s->dim);
    if (st != LIN_SUCCESS) return st;
  }
  const uint64_t lse_bytes = (uint64_t)s->heads_q * (uint64_t)s->tokens_q * 4;
  if (lse_bytes && !lse) return LIN_ERROR_INVALID_VALUE;
  auto misaligned4 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) != 0; };
  if (misaligned4(lse) || misaligned4(s->cu_q) || misaligned4(s->cu_k)) return LIN_ERROR_MISALIGNED;
  const uint64_t cu_bytes = ((uint64_t)s->sequences + 1) * 4;
  for (int i = 0; i < nviews; ++i) {
    const View& v = views[i];
    if (overlaps(lse, lse_bytes, v.t->data, v.extent) && (v.out || lse_out)) return LIN_ERROR_ALIASING;
    if (!v.out) continue;
    if ((s->cu_q && overlaps(s->cu_q, cu_bytes, v.t->data, v.extent)) ||
        (s->cu_k && overlaps(s->cu_k, cu_bytes, v.t->data, v.extent)))
      return LIN_ERROR_ALIASING;
    for (int k = 0; k < nviews; ++k)
      if (k != i && views_overlap(v, views[k], s->dim)) return LIN_ERROR_ALIASING;
  }
  if (lse_out && ((s->cu_q && overlaps(lse, lse_bytes, s->cu_q, cu_bytes)) ||
                  (s->cu_k && overlaps(lse, lse_bytes, s->cu_k, cu_bytes))))
    return LIN_ERROR_ALIASING;
  lin_status st = current_device(&got->dev, &got->word);
  if (st != LIN_SUCCESS) return st;
  SeenRange seen;
  for (int i = 0; i < nviews; ++i)
    if (views[i].extent &&
        (st = check_buffer(views[i].t->data, views[i].extent, got->dev, &seen)) != LIN_SUCCESS)
      return st;
  if (lse_bytes && (st = check_buffer(lse, lse_bytes, got->dev, &seen)) != LIN_SUCCESS) return st;
  if (s->cu_q && (st = check_buffer(s->cu_q, cu_bytes, got->dev, &seen)) != LIN_SUCCESS) return st;
  if (s->cu_k && (st = check_buffer(s->cu_k, cu_bytes, got->dev, &seen)) != LIN_SUCCESS) return st;
  got->nothing = s->sequences == 0;
  return LIN_SUCCESS;
}

bool encode_view(CUtensorMap* m, const View& v, int64_t dim, int box_tokens, int box_heads = 1) {
  return encode_heads(m, v.t->data, (uint64_t)dim, (uint64_t)v.heads, (uint64_t)v.tokens,
                      (uint64_t)v.hs * 2, (uint64_t)v.ts * 2, (uint32_t)box_tokens,
                      (uint32_t)box_heads);
}

lin::AttnArgs attn_args(const lin_attention_shape* s, const Checked& c) {
  lin::AttnArgs a{};
  a.cu_q = s->cu_q;
  a.cu_k = s->cu_k;
  a.tokens_q = (int32_t)s->tokens_q;
  a.tokens_k = (int32_t)s->tokens_k;
  a.max_q = (int32_t)c.max_q;
  a.max_k = (int32_t)c.max_k;
  a.heads_q = (int32_t)s->heads_q;
  a.group = (int32_t)(s->heads_q / s->heads_kv);
  a.dim = (int32_t)s->dim;
  a.causal = s->causal != 0;
  a.scale = s->scale;
  a.timeout_ns = wait_limit_ns();
  a.status = c.word;
  return a;
}

lin_status attention(const lin_attention_shape* s, const lin_heads* Q, const lin_heads* K,
                     const lin_heads* V, const lin_heads* O, float* LSE, cudaStream_t stream) {
  set_last_launch_info(0, 0);
  const int64_t hq = s ? s->heads_q : 0, hk = s ? s->heads_kv : 0;
  View v[] = {{Q, 0, hq, false}, {K, -1, hk, false}, {V, -1, hk, false}, {O, 0, hq, true}};
  Checked c;
  const lin_status st = check_attention(s, v, 4, LSE, true, &c);
  if (st != LIN_SUCCESS) return st;
  if (c.nothing || c.max_q == 0) return LIN_SUCCESS;
  lin::AttnFwdArgs a{attn_args(s, c), heads_ptr(v[3]), LSE, 1, 0, nullptr,
                     nullptr, 2, 1, 128};
  const int sms = sm_count(c.dev);
  auto tiles = [&] {
    return (c.max_q + a.tile_q - 1) / a.tile_q * (s->heads_q / a.pack) * s->sequences;
  };
  // The query heads that share a key head as rows of one tile, unless that
  // makes more tiles (a number of heads that does not divide 128 leaves rows
  // unused). 32 heads over 8 of 128, us: one query on 8192 keys 33 -> 17, 16
  // sequences of one on 2048 114 -> 31, 8192 tokens 337 -> 335; nine sequences
  // of 600, 12 heads over 6, 23.6 -> 20.2.
  if (a.s.group <= 128) {
    const int64_t apart = tiles();
    a.pack = a.s.group;
    a.tile_q = 128 / a.pack;
    // (a grid has 65535 tiles of queries at most)
    if (tiles() > apart || c.max_q > 65535LL * a.tile_q) a.pack = 1, a.tile_q = 128;
  }
  // One tile to a CTA while every CTA then has an SM to itself (512 tokens, 12
  // heads: 10.3 -> 8.9 us); beyond that the second tile's exponentials hide
  // the products' latency and K, V are read half as often.
  if (tiles() <= sms) a.tiles = 1;
  const int64_t rows = (int64_t)a.tiles * a.tile_q;
  // (a CTA of two tiles: more than half as many CTAs as SMs, no parts)
  if (a.tiles == 1)
    a.parts = lin::attn_parts((c.max_q + rows - 1) / rows * (s->heads_q / a.pack) * s->sequences,
                              c.max_k, sms);
  if (a.parts > 1) a.part_rows = (int32_t)(s->sequences * c.max_q);
  lin::AttnFwdMaps maps;
  bool ok = encode_view(&maps.q, v[0], s->dim, a.tile_q, a.pack);
  // without keys the K and V maps are never used
  ok &= encode_view(&maps.k, v[1].extent ? v[1] : v[0], s->dim, 128);
  ok &= encode_view(&maps.v, v[2].extent ? v[2] : v[0], s->dim, 128);
  if (!ok) return cuda_fail(cudaErrorInvalidValue);
  const uint64_t part_rows = (uint64_t)a.parts * (uint64_t)a.part_rows * (uint64_t)s->heads_q;
  const size_t bytes = a.parts > 1 ? (size_t)(part_rows * (uint64_t)(s->dim + 1) * 4) : 0;
  if (bytes) {
    a.o_part = static_cast<float*>(take_stream_workspace(c.dev, bytes, stream));
    if (!a.o_part) return LIN_ERROR_CUDA;
    a.lse_part = a.o_part + part_rows * (uint64_t)s->dim;
  }
  cudaError_t e = lin::launch_attn_fwd(s->dtype == LIN_BFLOAT16, maps, a, (int)s->heads_kv,
                                       (int)s->sequences, stream);
  if (bytes) {
    const cudaError_t ef = cudaFreeAsync(a.o_part, stream);
    if (e == cudaSuccess) e = ef;
  }
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info(a.parts > 1 ? 2 : 1, bytes);
  return LIN_SUCCESS;
}

lin_status attention_backward(const lin_attention_shape* s, const lin_heads* Q, const lin_heads* K,
                              const lin_heads* V, const lin_heads* O, const float* LSE,
                              const lin_heads* DO, const lin_heads* DQ, const lin_heads* DK,
                              const lin_heads* DV, cudaStream_t stream) {
  set_last_launch_info(0, 0);
  const int64_t hq = s ? s->heads_q : 0, hk = s ? s->heads_kv : 0;
  View v[] = {{Q, 0, hq, false},  {K, -1, hk, false}, {V, -1, hk, false}, {O, 0, hq, false},
              {DO, 0, hq, false}, {DQ, 0, hq, true},  {DK, -1, hk, true}, {DV, -1, hk, true}};
  Checked c;
  const lin_status st = check_attention(s, v, 8, LSE, false, &c);
  if (st != LIN_SUCCESS) return st;
  if (c.nothing || (c.max_q == 0 && c.max_k == 0)) return LIN_SUCCESS;
  lin::AttnBwdArgs a{};
  a.s = attn_args(s, c);
  a.q = heads_ptr(v[0]);
  a.k = heads_ptr(v[1]);
  a.v = heads_ptr(v[2]);
  a.o = heads_ptr(v[3]);
  a.dout = heads_ptr(v[4]);
  a.lse = LSE;
  a.dq = heads_ptr(v[5]);
  a.dk = heads_ptr(v[6]);
  a.dv = heads_ptr(v[7]);
  // The query heads that share a key head as rows of one tile, where their
  // number divides it: never more tiles, fewer where sequences end inside one,
  // and fewer tokens of a tile behind a causal mask (us: nine sequences of up
  // to 997, 12 heads over 6, 64.4 -> 59.9; 8192 tokens, 16 over 4, 632 -> 627;
  // 16 sequences of one query on 2048 keys, 32 over 8, 252 -> 149).
  const int group = a.s.group, turn = lin::kAttnBwdBox;
  if (group <= turn && (group & (group - 1)) == 0 && c.max_q * group <= 65535LL * 128) {
    while ((1 << a.shift) < group) ++a.shift;
  }
  const int64_t tq = ((c.max_q << a.shift) + 127) / 128, tk = (c.max_k + 127) / 128;
  const int64_t hq_tiles = s->heads_q >> a.shift;
  lin::AttnBwdMaps maps;
  const View& q = v[0].extent ? v[0] : v[1];   // (an empty side's maps are never used)
  const View& k = v[1].extent ? v[1] : v[0];
  const View& dout = v[4].extent ? v[4] : k;
  const int heads = 1 << a.shift;
  const bool ok = encode_view(&maps.q, q, s->dim, turn / heads, heads) &&
                  encode_view(&maps.k, k, s->dim, turn) &&
                  encode_view(&maps.v, v[2].extent ? v[2] : q, s->dim, turn) &&
                  encode_view(&maps.dout, dout, s->dim, turn / heads, heads);
  if (!ok) return cuda_fail(cudaErrorInvalidValue);
  const int sms = sm_count(c.dev);
  a.q_parts = lin::attn_parts(tq * hq_tiles * s->sequences, c.max_k, sms);
  a.k_parts = lin::attn_parts(tk * s->heads_kv * s->sequences, c.max_q * (int64_t)a.s.group, sms);
  // workspace: the parts' sums, delta [heads][tokens], then the largest dO
  // norms of the query tiles
  if (a.q_parts > 1) a.q_part_rows = (int32_t)(s->sequences * c.max_q);
  if (a.k_parts > 1) a.k_part_rows = (int32_t)(s->sequences * c.max_k);
  const uint64_t dq = (uint64_t)a.q_parts * a.q_part_rows * s->heads_q * s->dim;
  const uint64_t dk = (uint64_t)a.k_parts * a.k_part_rows * s->heads_kv * s->dim;
  const uint64_t delta = (uint64_t)s->heads_q * (uint64_t)s->tokens_q;
  const uint64_t norms = (uint64_t)s->sequences * (uint64_t)hq_tiles * (uint64_t)tq;
  const size_t bytes = (size_t)std::max<uint64_t>(16, (dq + 2 * dk + delta + norms) * 4);
  float* ws = static_cast<float*>(take_stream_workspace(c.dev, bytes, stream));
  if (!ws) return LIN_ERROR_CUDA;
  a.dq_part = ws;
  a.dk_part = ws + dq;
  a.dv_part = a.dk_part + dk;
  a.delta = a.dv_part + dk;
  a.norm = a.delta + delta;
  a.norms = (int64_t)norms;
  int kernels = 0;
  cudaError_t e = lin::launch_attn_bwd(s->dtype == LIN_BFLOAT16, maps, a, (int)s->heads_kv,
                                       (int)s->sequences, &kernels, stream);
  const cudaError_t ef = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = ef;
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info(kernels, bytes);
  return LIN_SUCCESS;
}

}  // namespace
}  // namespace lin_detail

extern "C" {

lin_status lin_attention(const lin_attention_shape* shape, const lin_heads* Q, const lin_heads* K,
                         const lin_heads* V, const lin_heads* O, float* LSE,
                         lin_stream_t stream) {
  return lin_detail::attention(shape, Q, K, V, O, LSE, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_attention_backward(const lin_attention_shape* shape, const lin_heads* Q,
                                  const lin_heads* K, const lin_heads* V, const lin_heads* O,
                                  const float* LSE, const lin_heads* DO, const lin_heads* DQ,
                                  const lin_heads* DK, const lin_heads* DV, lin_stream_t stream) {
  return lin_detail::attention_backward(shape, Q, K, V, O, LSE, DO, DQ, DK, DV,
                                        reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
