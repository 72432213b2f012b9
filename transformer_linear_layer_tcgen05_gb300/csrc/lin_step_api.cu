// lin_step_api.cu -- the entry points of include/lin.h around attention and
// the loss: norms and rotation of the query and key heads, distillation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "lin.h"
#include "lin_distill.h"
#include "lin_heads.h"
#include "lin_internal.h"
#include "lin_rope.h"

namespace lin_detail {

namespace {

// A dense buffer of a call: `align` bytes, `out` if the call writes it.
struct Buffer {
  const void* p;
  uint64_t bytes;
  uint32_t align;
  bool out;
};

// Presence and alignment, then that no output meets another buffer.
lin_status check_buffers(const Buffer* b, int n) {
  for (int i = 0; i < n; ++i)
    if (b[i].bytes && !b[i].p) return LIN_ERROR_INVALID_VALUE;
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(b[i].p) % b[i].align != 0) return LIN_ERROR_MISALIGNED;
  for (int i = 0; i < n; ++i)
    for (int k = 0; k < n; ++k)
      if (k != i && b[i].out && overlaps(b[i].p, b[i].bytes, b[k].p, b[k].bytes))
        return LIN_ERROR_ALIASING;
  return LIN_SUCCESS;
}

lin_status check_on_device(const Buffer* b, int n, int dev, SeenRange* seen) {
  for (int i = 0; i < n; ++i)
    if (b[i].bytes) {
      const lin_status st = check_buffer(b[i].p, b[i].bytes, dev, seen);
      if (st != LIN_SUCCESS) return st;
    }
  return LIN_SUCCESS;
}

// Both directions: DX, DWQ and DWK are null in the forward one, where Q, K
// and V are written.
lin_status qk_norm_rope(const lin_qk_norm_rope_shape* s, const float* X, const float* WQ,
                        const float* WK, const float* COS, const float* SIN,
                        const int32_t* positions, const lin_heads* Q, const lin_heads* K,
                        const lin_heads* V, bool backward, float* DX, float* DWQ, float* DWK,
                        cudaStream_t stream) {
  set_last_launch_info(0, 0);
  if (!s || !Q || !K || !V) return LIN_ERROR_INVALID_VALUE;
  if (s->dtype != LIN_BINARY16 && s->dtype != LIN_BFLOAT16) return LIN_ERROR_INVALID_VALUE;
  if (s->tokens < 0 || s->heads_q < 1 || s->heads_kv < 1 || s->dim < 1 || s->rot < 0 ||
      s->rot > s->dim || !(s->eps >= 0.0f) || std::isinf(s->eps) ||
      (s->rot > 0 && s->table_rows < 1))
    return LIN_ERROR_INVALID_VALUE;
  if (s->tokens > kMaxExtent || s->heads_q > 65536 || s->heads_kv > 65536 || s->dim % 8 != 0 ||
      s->dim > 256 || s->rot % 8 != 0 || s->table_rows > kMaxExtent)
    return LIN_ERROR_UNSUPPORTED_SHAPE;
  const int64_t heads = s->heads_q + 2 * s->heads_kv;
  // (a group of threads takes a few heads of one token: see the grid)
  if ((unsigned __int128)s->tokens * heads * s->dim >= ((unsigned __int128)1 << 40))
    return LIN_ERROR_UNSUPPORTED_SHAPE;
  View v[] = {{Q, s->tokens, s->heads_q, !backward},
              {K, s->tokens, s->heads_kv, !backward},
              {V, s->tokens, s->heads_kv, !backward}};
  for (View& w : v) {
    const lin_status st = check_view(w, s->dim);
    if (st != LIN_SUCCESS) return st;
  }
  const uint64_t t = (uint64_t)s->tokens, xb = t * heads * s->dim * 4, wb = (uint64_t)s->dim * 4;
  const uint64_t tb = s->rot ? (uint64_t)s->table_rows * s->rot * 2 : 0;
  Buffer b[] = {{X, xb, 16, false},      {WQ, wb, 16, false},
                {WK, wb, 16, false},     {COS, tb, 16, false},
                {SIN, tb, 16, false},    {positions, positions ? t * 4 : 0, 4, false},
                {DX, backward ? xb : 0, 16, true}, {DWQ, backward ? wb : 0, 4, true},
                {DWK, backward ? wb : 0, 4, true}};
  const int nb = (int)(sizeof(b) / sizeof(b[0]));
  lin_status st = check_buffers(b, nb);
  if (st != LIN_SUCCESS) return st;
  for (int i = 0; i < 3; ++i) {
    for (const Buffer& o : b)
      if ((v[i].out || o.out) && overlaps(v[i].t->data, v[i].extent, o.p, o.bytes))
        return LIN_ERROR_ALIASING;
    for (int k = 0; k < 3; ++k)
      if (k != i && v[i].out && views_overlap(v[i], v[k], s->dim)) return LIN_ERROR_ALIASING;
  }
  int dev = 0;
  int* word = nullptr;
  if ((st = current_device(&dev, &word)) != LIN_SUCCESS) return st;
  SeenRange seen;
  if ((st = check_on_device(b, nb, dev, &seen)) != LIN_SUCCESS) return st;
  for (const View& w : v)
    if (w.extent && (st = check_buffer(w.t->data, w.extent, dev, &seen)) != LIN_SUCCESS) return st;
  if (s->tokens == 0) {   // no rows: the weights' gradients are sums of nothing
    cudaError_t e = cudaSuccess;
    if (backward) e = cudaMemsetAsync(DWQ, 0, wb, stream);
    if (backward && e == cudaSuccess) e = cudaMemsetAsync(DWK, 0, wb, stream);
    return e == cudaSuccess ? LIN_SUCCESS : cuda_fail(e);
  }
  lin::RopeArgs a{};
  a.x = X;
  a.wq = WQ;
  a.wk = WK;
  a.cos = COS;
  a.sin = SIN;
  a.pos = positions;
  a.tokens = s->tokens;
  a.table_rows = s->table_rows;
  a.hq = (int32_t)s->heads_q;
  a.hk = (int32_t)s->heads_kv;
  a.dim = (int32_t)s->dim;
  a.rot = (int32_t)s->rot;
  a.eps = s->eps;
  a.status = word;
  a.q = heads_ptr(v[0]);
  a.k = heads_ptr(v[1]);
  a.v = heads_ptr(v[2]);
  const bool bf16 = s->dtype == LIN_BFLOAT16, inter = s->interleaved != 0;
  if (!backward) {
    const cudaError_t e = lin::launch_qk_norm_rope(a, inter, bf16, stream);
    if (e != cudaSuccess) return cuda_fail(e);
    set_last_launch_info(1, 0);
    return LIN_SUCCESS;
  }
  a.dx = DX;
  a.dwq = DWQ;
  a.dwk = DWK;
  const int ctas = lin::qk_norm_rope_bwd_ctas(a, sm_count(dev));
  const size_t bytes = (size_t)ctas * (size_t)s->dim * 4;
  a.partial = static_cast<float*>(take_stream_workspace(dev, bytes, stream));
  if (!a.partial) return LIN_ERROR_CUDA;
  cudaError_t e = lin::launch_qk_norm_rope_bwd(a, inter, bf16, ctas, stream);
  const cudaError_t ef = cudaFreeAsync(a.partial, stream);
  if (e == cudaSuccess) e = ef;
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info(2, bytes);
  return LIN_SUCCESS;
}

lin_status distill_topk(const float* LOGITS, int64_t ld, const int32_t* ids, const float* teacher,
                        float* DLOGITS, int64_t ldd, float* losses, float* loss_sum, int64_t M,
                        int64_t V, int64_t K, float tau, float inv_norm, cudaStream_t stream) {
  set_last_launch_info(0, 0);
  if (M < 0 || V < 0 || K < 0 || !loss_sum) return LIN_ERROR_INVALID_VALUE;
  if (!(tau > 0.0f) || std::isinf(tau)) return LIN_ERROR_INVALID_VALUE;
  if (M > 1 && (ld < V || (DLOGITS && ldd < V))) return LIN_ERROR_INVALID_VALUE;
  if (M > kMaxExtent / 8 || V > kMaxExtent - 65536 || K > 1024 || ld >= (1LL << 40) ||
      ldd >= (1LL << 40))
    return LIN_ERROR_UNSUPPORTED_SHAPE;
  if (M <= 1) ld = ldd = V;   // (the stride of one row is not looked at)
  const uint64_t rows = (uint64_t)M;
  auto extent = [&](int64_t stride) {
    return M > 0 && V > 0 ? ((rows - 1) * (uint64_t)stride + (uint64_t)V) * 4 : 0;
  };
  const bool in_place = DLOGITS == LOGITS;
  if (in_place && DLOGITS && ld != ldd) return LIN_ERROR_ALIASING;
  Buffer b[] = {{LOGITS, extent(ld), 4, false},
                {ids, rows * (uint64_t)K * 4, 4, false},
                {teacher, rows * (uint64_t)K * 4, 4, false},
                {losses, rows * 4, 4, true},
                {loss_sum, 4, 4, true},
                {DLOGITS, DLOGITS && !in_place ? extent(ldd) : 0, 4, true}};
  const int nb = (int)(sizeof(b) / sizeof(b[0]));
  lin_status st = check_buffers(b, nb);
  if (st != LIN_SUCCESS) return st;
  if (in_place && DLOGITS)   // the logits are written too
    for (int i = 1; i < nb; ++i)
      if (overlaps(DLOGITS, extent(ld), b[i].p, b[i].bytes)) return LIN_ERROR_ALIASING;
  int dev = 0;
  int* word = nullptr;
  if ((st = current_device(&dev, &word)) != LIN_SUCCESS) return st;
  SeenRange seen;
  if ((st = check_on_device(b, nb, dev, &seen)) != LIN_SUCCESS) return st;
  if (M == 0 || V == 0) {   // no rows, or no entry that a row could list
    cudaError_t e = cudaMemsetAsync(loss_sum, 0, 4, stream);
    if (e == cudaSuccess && M > 0) e = cudaMemsetAsync(losses, 0, rows * 4, stream);
    return e == cudaSuccess ? LIN_SUCCESS : cuda_fail(e);
  }
  lin::DistillArgs a{LOGITS, ids, teacher, DLOGITS, losses, M, V, ld, ldd, (int32_t)K, tau,
                     inv_norm, wait_limit_ns(), word, 1, 1, 0, 1};
  const cudaError_t e = lin::launch_distill(a, loss_sum, sm_count(dev), stream);
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info(2, 0);
  return LIN_SUCCESS;
}

}  // namespace
}  // namespace lin_detail

extern "C" {

lin_status lin_qk_norm_rope(const lin_qk_norm_rope_shape* shape, const float* X, const float* WQ,
                            const float* WK, const float* COS, const float* SIN,
                            const int32_t* positions, const lin_heads* Q, const lin_heads* K,
                            const lin_heads* V, lin_stream_t stream) {
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, Q, K, V, false, nullptr,
                                  nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_qk_norm_rope_backward(const lin_qk_norm_rope_shape* shape, const float* X,
                                     const float* WQ, const float* WK, const float* COS,
                                     const float* SIN, const int32_t* positions,
                                     const lin_heads* DQ, const lin_heads* DK, const lin_heads* DV,
                                     float* DX, float* DWQ, float* DWK, lin_stream_t stream) {
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, DQ, DK, DV, true, DX, DWQ,
                                  DWK, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_distill_topk(const float* LOGITS, int64_t ld, const int32_t* ids,
                            const float* teacher, float* DLOGITS, int64_t ldd, float* losses,
                            float* loss_sum, int64_t M, int64_t V, int64_t K, float temperature,
                            float inv_norm, lin_stream_t stream) {
  return lin_detail::distill_topk(LOGITS, ld, ids, teacher, DLOGITS, ldd, losses, loss_sum, M, V,
                                  K, temperature, inv_norm,
                                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
