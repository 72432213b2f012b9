// lin_step_api.cu -- the entry points of include/lin.h around attention, the
// loss and the weights: norms and rotation of the query and key heads, norms
// around a block, distillation, the AdamW step.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "lin.h"
#include "lin_adamw.h"
#include "lin_distill.h"
#include "lin_heads.h"
#include "lin_internal.h"
#include "lin_norms.h"
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

// Tensors of one AdamW call, and host memory for what it keeps of them: on the
// stack for a few, else from the heap (null if there is none).
constexpr int64_t kMaxTensors = 1 << 20;
template <typename T>
struct Scratch {
  alignas(T) unsigned char few[64 * sizeof(T)];
  T* p;
  explicit Scratch(size_t n) : p(reinterpret_cast<T*>(few)) {
    if (n > 64) p = static_cast<T*>(std::malloc(n * sizeof(T)));
  }
  ~Scratch() {
    if (p != reinterpret_cast<T*>(few)) std::free(p);
  }
  Scratch(const Scratch&) = delete;
};

// Whether a call by axes gathers its tokens' angles by a kernel of its own,
// once for all heads, instead of pair by pair for every two heads. us, gathered
// and not, pairs dealt to three axes in turn: 576 tokens of 12 + 2 x 12 heads of
// 64 5.1 and 4.5, the gradient 9.3 and 8.8; 1280 tokens 6.2 and 6.2, 11.5 and
// 12.1; 16184 tokens of 32 + 2 x 8 of 128 96 and 128, 172 and 213.
bool gather_angles(uint64_t entries) { return entries >= (3u << 20); }

// Both directions: DX, DWQ and DWK are null in the forward one, where Q, K
// and V are written. axes > 0: positions [axes][tokens] and each pair's axis.
lin_status qk_norm_rope(const lin_qk_norm_rope_shape* s, const float* X, const float* WQ,
                        const float* WK, const float* COS, const float* SIN,
                        const int32_t* positions, int64_t axes, const int32_t* pair_axis,
                        const lin_heads* Q, const lin_heads* K, const lin_heads* V, bool backward,
                        float* DX, float* DWQ, float* DWK, cudaStream_t stream) {
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
  const uint64_t pb = axes > 0 ? (s->rot ? (uint64_t)axes * t * 4 : 0) : positions ? t * 4 : 0;
  Buffer b[] = {{X, xb, 16, false},      {WQ, wb, 16, false},
                {WK, wb, 16, false},     {COS, tb, 16, false},
                {SIN, tb, 16, false},    {positions, pb, 4, false},
                {pair_axis, axes > 0 ? (uint64_t)s->rot * 2 : 0, 16, false},
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
  a.axis = axes > 0 && s->rot ? pair_axis : nullptr;
  a.axes = (int32_t)axes;
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
  a.dx = DX;
  a.dwq = DWQ;
  a.dwk = DWK;
  const int ctas = backward ? lin::qk_norm_rope_bwd_ctas(a, sm_count(dev)) : 0;
  const bool gather = a.axis && gather_angles(t * heads * s->dim);
  // workspace: the angles by token (16-byte units), the partial sums
  const size_t angles = gather ? (size_t)t * (size_t)s->rot * 4 : 0;
  const size_t bytes = angles + (size_t)ctas * (size_t)s->dim * 4;
  float* ws = nullptr;
  if (bytes) {
    ws = static_cast<float*>(take_stream_workspace(dev, bytes, stream));
    if (!ws) return LIN_ERROR_CUDA;
  }
  a.partial = ws + angles / 4;
  cudaError_t e = gather ? lin::launch_gather_angles(a, ws, stream) : cudaSuccess;
  if (e == cudaSuccess)
    e = backward ? lin::launch_qk_norm_rope_bwd(a, inter, bf16, ctas, stream)
                 : lin::launch_qk_norm_rope(a, inter, bf16, stream);
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info((gather ? 1 : 0) + (backward ? 2 : 1), bytes);
  return LIN_SUCCESS;
}

lin_status check_axes(int64_t axes) {
  set_last_launch_info(0, 0);
  return axes < 1 ? LIN_ERROR_INVALID_VALUE
         : axes > lin::kMostAxes ? LIN_ERROR_UNSUPPORTED_SHAPE : LIN_SUCCESS;
}

// Both directions: X is the residual stream (forward) or its new value H
// (gradient).
lin_status block_norms(const lin_block_norms_shape* s, const float* X, const void* Y,
                       const float* GATE, const float* W_POST, const float* W_PRE, float* H,
                       void* N, bool backward, const float* DH, const void* DN, float* DX, void* DY,
                       float* DGATE, float* DW_POST, float* DW_PRE, cudaStream_t stream) {
  set_last_launch_info(0, 0);
  if (!s) return LIN_ERROR_INVALID_VALUE;
  if (s->dtype != LIN_BINARY16 && s->dtype != LIN_BFLOAT16 && s->dtype != LIN_BINARY32)
    return LIN_ERROR_INVALID_VALUE;
  if (s->gate < LIN_GATE_NONE || s->gate > LIN_GATE_FULL || s->tokens < 0 || s->width < 0 ||
      !std::isfinite(s->residual_scale) || !std::isfinite(s->block_scale) || !(s->eps >= 0.0f) ||
      std::isinf(s->eps))
    return LIN_ERROR_INVALID_VALUE;
  if (s->tokens > kMaxExtent || s->width % 4 != 0 || s->width > lin::kNormMostWidth ||
      s->tokens * s->width >= (1LL << 40))
    return LIN_ERROR_UNSUPPORTED_SHAPE;
  if (s->width == 0 || (s->tokens == 0 && !backward)) return LIN_SUCCESS;
  int dev = 0;
  int* word = nullptr;
  SeenRange seen;
  lin_status st;
  if (s->tokens == 0) {
    // The weights' gradients are sums of nothing (of the tensors of tokens,
    // which have no entries, nothing is looked at).
    const uint64_t wb = (uint64_t)s->width * 4;
    float* const sums[] = {DW_POST, DW_PRE, s->gate == LIN_GATE_CHANNEL ? DGATE : nullptr};
    Buffer b[3];
    for (int i = 0; i < 3; ++i) b[i] = Buffer{sums[i], sums[i] ? wb : 0, 16, true};
    if ((st = check_buffers(b, 3)) != LIN_SUCCESS || (st = current_device(&dev, &word)) != LIN_SUCCESS ||
        (st = check_on_device(b, 3, dev, &seen)) != LIN_SUCCESS)
      return st;
    cudaError_t e = cudaSuccess;
    for (float* p : sums)
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, wb, stream);
    return e == cudaSuccess ? LIN_SUCCESS : cuda_fail(e);
  }
  // What goes together: the block's output with its gate, its norm and their
  // gradients; the norm behind with its weight's gradient.
  const bool gated = s->gate != LIN_GATE_NONE, by_channel = s->gate == LIN_GATE_CHANNEL;
  if (gated != (GATE != nullptr)) return LIN_ERROR_INVALID_VALUE;
  if (!Y && (gated || W_POST)) return LIN_ERROR_INVALID_VALUE;
  if (!backward) {
    if (!X || (!H && !N) || (N != nullptr) != (W_PRE != nullptr)) return LIN_ERROR_INVALID_VALUE;
  } else {
    if (!DX || (!DH && !DN) || (DN != nullptr) != (W_PRE != nullptr) ||
        (DN != nullptr) != (DW_PRE != nullptr) || (W_POST != nullptr) != (DW_POST != nullptr) ||
        gated != (DGATE != nullptr) || (Y != nullptr) != (DY != nullptr) || (DN && !X))
      return LIN_ERROR_INVALID_VALUE;
  }
  const uint64_t n = (uint64_t)s->tokens * (uint64_t)s->width, wb = (uint64_t)s->width * 4;
  const uint64_t fb = n * 4, yb = n * (s->dtype == LIN_BINARY32 ? 4 : 2);
  const uint64_t gb = by_channel ? wb : s->gate == LIN_GATE_TOKEN ? (uint64_t)s->tokens * 4 : fb;
  const uint32_t ga = s->gate == LIN_GATE_TOKEN ? 4 : 16, ya = s->dtype == LIN_BINARY32 ? 16 : 8;
  auto has = [](const void* p, uint64_t bytes) { return p ? bytes : 0; };
  // (in place: H over X, DX over DH)
  const bool h_in_x = !backward && H == X, dx_in_dh = backward && DX == DH;
  Buffer b[] = {{X, h_in_x ? 0 : backward && !DN ? 0 : has(X, fb), 16, false},
                {Y, has(Y, yb), ya, false},
                {GATE, has(GATE, gb), ga, false},
                {W_POST, has(W_POST, wb), 16, false},
                {W_PRE, has(W_PRE, wb), 16, false},
                {DH, dx_in_dh ? 0 : has(DH, fb), 16, false},
                {DN, has(DN, yb), ya, false},
                {H, has(H, fb), 16, true},
                {N, has(N, yb), ya, true},
                {DX, has(DX, fb), 16, true},
                {DY, has(DY, yb), ya, true},
                {DGATE, has(DGATE, gb), ga, true},
                {DW_POST, has(DW_POST, wb), 16, true},
                {DW_PRE, has(DW_PRE, wb), 16, true}};
  const int nb = (int)(sizeof(b) / sizeof(b[0]));
  if ((st = check_buffers(b, nb)) != LIN_SUCCESS || (st = current_device(&dev, &word)) != LIN_SUCCESS ||
      (st = check_on_device(b, nb, dev, &seen)) != LIN_SUCCESS)
    return st;
  lin::NormsArgs a{};
  a.x = X;
  a.y = Y;
  a.gate = GATE;
  a.w_post = W_POST;
  a.w_pre = W_PRE;
  a.h = H;
  a.n = N;
  a.dh = DH;
  a.dn = DN;
  a.dx = DX;
  a.dy = DY;
  a.dgate = DGATE;
  a.dw_post = DW_POST;
  a.dw_pre = DW_PRE;
  a.tokens = s->tokens;
  a.width = (int32_t)s->width;
  a.form = s->gate;
  a.dtype = s->dtype;
  a.residual_scale = s->residual_scale;
  a.block_scale = s->block_scale;
  a.eps = s->eps;
  a.status = word;
  if (!backward) {
    const cudaError_t e = lin::launch_block_norms(a, sm_count(dev), stream);
    if (e != cudaSuccess) return cuda_fail(e);
    set_last_launch_info(1, 0);
    return LIN_SUCCESS;
  }
  a.kinds = (DN != nullptr) + (W_POST != nullptr) + by_channel;
  const int ctas = lin::block_norms_bwd_ctas(a, sm_count(dev));
  const size_t bytes = (size_t)ctas * (size_t)a.kinds * wb;
  if (bytes) {
    a.partial = static_cast<float*>(take_stream_workspace(dev, bytes, stream));
    if (!a.partial) return LIN_ERROR_CUDA;
  }
  cudaError_t e = lin::launch_block_norms_bwd(a, sm_count(dev), ctas, stream);
  if (bytes) {
    const cudaError_t ef = cudaFreeAsync(a.partial, stream);
    if (e == cudaSuccess) e = ef;
  }
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launch_info(bytes ? 2 : 1, bytes);
  return LIN_SUCCESS;
}

lin_status adamw(const lin_adamw_step* s, const lin_adamw_tensor* tensors, int64_t count,
                 cudaStream_t stream) {
  set_last_launch_info(0, 0);
  if (!s || count < 0 || (count > 0 && !tensors)) return LIN_ERROR_INVALID_VALUE;
  if (s->state_bits != 32 && s->state_bits != 8) return LIN_ERROR_INVALID_VALUE;
  auto share = [](double b) { return b >= 0.0 && b < 1.0; };
  if (!share(s->beta1) || !share(s->beta2) || !(s->eps >= 0.0) || std::isinf(s->eps) ||
      !std::isfinite(s->weight_decay) || (!s->step_device && s->step < 1) ||
      (!s->lr_device && !std::isfinite(s->lr)))
    return LIN_ERROR_INVALID_VALUE;
  const bool bits8 = s->state_bits == 8;
  // Each tensor's buffers, kind by kind (p, g, m, v, scales, copies): presence and
  // alignment, then that no written one meets another of the call.
  struct Range {
    uintptr_t at, end;
    bool out;
  };
  auto misaligned = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (misaligned(s->lr_device, 4) || misaligned(s->step_device, 4) || misaligned(s->grad_scale, 4))
    return LIN_ERROR_MISALIGNED;
  if (count > kMaxTensors) return LIN_ERROR_UNSUPPORTED_SHAPE;
  constexpr int kKinds = 8;   // (the last: the values on the device)
  const size_t most = (size_t)std::max<int64_t>(count, 3);
  Scratch<Range> ranges(most * kKinds);
  Scratch<lin::AdamwTensor> list((size_t)count);
  Scratch<uint32_t> first((size_t)count);
  if (!ranges.p || !list.p || !first.p) return LIN_ERROR_CUDA;
  size_t held[kKinds] = {};
  int64_t used = 0, blocks = 0;
  auto add = [&](int kind, const void* p, uint64_t bytes, bool out) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p && bytes) ranges.p[kind * most + held[kind]++] = Range{at, at + bytes, out};
  };
  add(7, s->lr_device, 4, false);
  add(7, s->step_device, 4, false);
  add(7, s->grad_scale, 4, false);
  const uint64_t state = bits8 ? 1 : 4;
  for (int64_t i = 0; i < count; ++i) {
    const lin_adamw_tensor& t = tensors[i];
    if (t.n < 0) return LIN_ERROR_INVALID_VALUE;
    if (t.n == 0) continue;
    if (t.n >= (1LL << 39)) return LIN_ERROR_UNSUPPORTED_SHAPE;
    if (!t.p || !t.g || !t.m || !t.v || (bits8 && (!t.m_scale || !t.v_scale))) return LIN_ERROR_INVALID_VALUE;
    const uintptr_t f = 4, c = bits8 ? 1 : 4;
    if (misaligned(t.p, f) || misaligned(t.g, f) || misaligned(t.m, c) || misaligned(t.v, c) ||
        (bits8 && (misaligned(t.m_scale, f) || misaligned(t.v_scale, f))) || misaligned(t.w16, 2))
      return LIN_ERROR_MISALIGNED;
    const int64_t nb = (t.n + lin::kAdamwBlock - 1) / lin::kAdamwBlock;
    const uint64_t n = (uint64_t)t.n;
    add(0, t.p, n * 4, true);
    add(1, t.g, n * 4, false);
    add(2, t.m, n * state, true);
    add(3, t.v, n * state, true);
    if (bits8) {
      add(4, t.m_scale, (uint64_t)nb * 4, true);
      add(5, t.v_scale, (uint64_t)nb * 4, true);
    }
    add(6, t.w16, n * 2, true);
    const uintptr_t wide = bits8 ? 8 : 32;
    lin::AdamwTensor& to = list.p[used];
    to.p = t.p;
    to.g = t.g;
    to.m = t.m;
    to.v = t.v;
    to.m_scale = t.m_scale;
    to.v_scale = t.v_scale;
    to.w16 = t.w16;
    to.n = t.n;
    to.wide = !misaligned(t.p, 32) && !misaligned(t.g, 32) && !misaligned(t.m, wide) &&
              !misaligned(t.v, wide) && !misaligned(t.w16, 16);
    ++used;
  }
  // In the order of their addresses neighbours tell. Tensors mostly come in that
  // order, kind by kind from buffers of their own: then each kind's neighbours
  // and the kinds' extents do (128 tensors of four kinds: sorting took 5 us).
  auto meet = [](const Range* r, size_t n) {
    uintptr_t end = 0, written_end = 0;   // behind everything, and what is written, so far
    for (size_t i = 0; i < n; ++i) {
      if (r[i].at < (r[i].out ? end : written_end)) return true;
      end = std::max(end, r[i].end);
      if (r[i].out) written_end = std::max(written_end, r[i].end);
    }
    return false;
  };
  auto before = [](const Range& a, const Range& b) { return a.at < b.at; };
  bool ordered = true;
  Range extents[kKinds];
  size_t kinds = 0, nr = 0;
  for (int k = 0; k < kKinds; ++k) {
    Range* r = ranges.p + k * most;
    if (held[k] == 0) continue;
    ordered = ordered && std::is_sorted(r, r + held[k], before);
    Range all = r[0];
    for (size_t i = 1; i < held[k]; ++i) all = Range{std::min(all.at, r[i].at), std::max(all.end, r[i].end), all.out};
    extents[kinds++] = all;
    if (ranges.p + nr != r) std::copy(r, r + held[k], ranges.p + nr);   // (down)
    nr += held[k];
  }
  std::sort(extents, extents + kinds, before);
  if (ordered && !meet(extents, kinds)) {
    size_t at = 0;
    for (int k = 0; k < kKinds; at += held[k++])
      if (meet(ranges.p + at, held[k])) return LIN_ERROR_ALIASING;
  } else {
    std::sort(ranges.p, ranges.p + nr, before);
    if (meet(ranges.p, nr)) return LIN_ERROR_ALIASING;
  }
  if (used == 0) return LIN_SUCCESS;
  int dev = 0;
  int* word = nullptr;
  lin_status st = current_device(&dev, &word);
  if (st != LIN_SUCCESS) return st;
  SeenRange seen;   // (neighbours share an allocation)
  for (size_t i = 0; i < nr; ++i) {
    const Range& r = ranges.p[i];
    if ((st = check_buffer(reinterpret_cast<const void*>(r.at), r.end - r.at, dev, &seen)) != LIN_SUCCESS)
      return st;
  }
  lin::AdamwArgs a{};
  a.beta1 = (float)s->beta1;
  a.beta1_rest = (float)(1.0 - s->beta1);
  a.beta2 = (float)s->beta2;
  a.beta2_rest = (float)(1.0 - s->beta2);
  // (Above zero it stays so, and of float32's normal numbers: where there has been
  // no gradient the kernel's 0 / eps would be 0 / 0, or 0 times an infinite
  // reciprocal. The root of a v above zero is 2^-75 or more, beside which this is
  // nothing.)
  a.eps = s->eps > 0.0 ? std::max((float)s->eps, 0x1p-126f) : 0.0f;
  const double t = (double)std::max<int64_t>(s->step, 1);
  const double c1 = 1.0 / -std::expm1(t * std::log(s->beta1));
  const double c2 = 1.0 / std::sqrt(-std::expm1(t * std::log(s->beta2)));
  a.keep = (float)(1.0 - s->lr * s->weight_decay);
  // (a device learning rate: the kernel multiplies the step's factor by it)
  a.rate = (float)(s->lr_device || s->step_device ? c1 : s->lr * c1);
  a.root = (float)c2;
  a.lr = s->lr_device;
  a.step = s->step_device;
  a.lr_value = (float)s->lr;
  a.decay = (float)s->weight_decay;
  a.log_beta1 = (float)std::log(s->beta1);
  a.log_beta2 = (float)std::log(s->beta2);
  a.grad_scale = s->grad_scale;
  a.status = word;
  int kernels = 0;
  for (int64_t i = 0; i < used;) {
    // as many tensors as a launch's parameters hold, and fewer than 2^31 blocks
    int n = 0;
    blocks = 0;
    while (i + n < used && n < lin::kAdamwMost) {
      const int64_t nb = (list.p[i + n].n + lin::kAdamwBlock - 1) / lin::kAdamwBlock;
      if (blocks + nb >= (1LL << 31) && n > 0) break;
      first.p[i + n] = (uint32_t)blocks;
      blocks += nb;
      ++n;
    }
    a.tensors = n;
    a.blocks = (uint32_t)blocks;
    const cudaError_t e = lin::launch_adamw(a, list.p + i, first.p + i, bits8, sm_count(dev), stream);
    if (e != cudaSuccess) return cuda_fail(e);
    ++kernels;
    i += n;
  }
  set_last_launch_info(kernels, 0);
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
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, 0, nullptr, Q, K, V, false,
                                  nullptr, nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_qk_norm_rope_backward(const lin_qk_norm_rope_shape* shape, const float* X,
                                     const float* WQ, const float* WK, const float* COS,
                                     const float* SIN, const int32_t* positions,
                                     const lin_heads* DQ, const lin_heads* DK, const lin_heads* DV,
                                     float* DX, float* DWQ, float* DWK, lin_stream_t stream) {
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, 0, nullptr, DQ, DK, DV,
                                  true, DX, DWQ, DWK, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_qk_norm_rope_axes(const lin_qk_norm_rope_shape* shape, int64_t axes, const float* X,
                                 const float* WQ, const float* WK, const float* COS,
                                 const float* SIN, const int32_t* positions,
                                 const int32_t* pair_axis, const lin_heads* Q, const lin_heads* K,
                                 const lin_heads* V, lin_stream_t stream) {
  const lin_status st = lin_detail::check_axes(axes);
  if (st != LIN_SUCCESS) return st;
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, axes, pair_axis, Q, K, V,
                                  false, nullptr, nullptr, nullptr,
                                  reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_qk_norm_rope_axes_backward(const lin_qk_norm_rope_shape* shape, int64_t axes,
                                          const float* X, const float* WQ, const float* WK,
                                          const float* COS, const float* SIN,
                                          const int32_t* positions, const int32_t* pair_axis,
                                          const lin_heads* DQ, const lin_heads* DK,
                                          const lin_heads* DV, float* DX, float* DWQ, float* DWK,
                                          lin_stream_t stream) {
  const lin_status st = lin_detail::check_axes(axes);
  if (st != LIN_SUCCESS) return st;
  return lin_detail::qk_norm_rope(shape, X, WQ, WK, COS, SIN, positions, axes, pair_axis, DQ, DK,
                                  DV, true, DX, DWQ, DWK, reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_block_norms(const lin_block_norms_shape* shape, const float* X, const void* Y,
                           const float* GATE, const float* W_POST, const float* W_PRE, float* H,
                           void* N, lin_stream_t stream) {
  return lin_detail::block_norms(shape, X, Y, GATE, W_POST, W_PRE, H, N, false, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, nullptr, nullptr,
                                 reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_block_norms_backward(const lin_block_norms_shape* shape, const float* H,
                                    const void* Y, const float* GATE, const float* W_POST,
                                    const float* W_PRE, const float* DH, const void* DN, float* DX,
                                    void* DY, float* DGATE, float* DW_POST, float* DW_PRE,
                                    lin_stream_t stream) {
  return lin_detail::block_norms(shape, H, Y, GATE, W_POST, W_PRE, nullptr, nullptr, true, DH, DN,
                                 DX, DY, DGATE, DW_POST, DW_PRE,
                                 reinterpret_cast<cudaStream_t>(stream));
}

lin_status lin_adamw(const lin_adamw_step* step, const lin_adamw_tensor* tensors, int64_t count,
                     lin_stream_t stream) {
  return lin_detail::adamw(step, tensors, count, reinterpret_cast<cudaStream_t>(stream));
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
