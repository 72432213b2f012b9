// lin_heads.h -- host checks of [tokens, heads, dim] tensors (lin_heads) that
// the entry points over them share.
#pragma once

#include <algorithm>
#include <cstdint>

#include "lin.h"
#include "lin_attn.h"
#include "lin_internal.h"

namespace lin_detail {

constexpr int64_t kMaxExtent = 0x7fffffffLL;

// One [tokens][heads][dim] tensor of a call.
struct View {
  const lin_heads* t;
  int64_t tokens, heads;
  bool out;
  // strides with those of an extent of one (which are never used) set to
  // something valid
  int64_t ts, hs;
  uint64_t extent;   // bytes from the first to behind the last entry
};

inline lin_status check_view(View& v, int64_t dim) {
  if (v.tokens == 0) {
    v.ts = v.hs = dim;
    v.extent = 0;
    return LIN_SUCCESS;
  }
  if (!v.t->data) return LIN_ERROR_INVALID_VALUE;
  v.hs = v.heads > 1 ? v.t->head_stride : dim;
  v.ts = v.tokens > 1 ? v.t->token_stride : std::max(dim, v.hs * v.heads);
  // no entry may be at two places of the tensor: the larger stride steps
  // over the smaller one's whole extent
  const bool head_inner = v.heads == 1 || (v.tokens > 1 && v.hs <= v.ts) || v.tokens == 1;
  const int64_t small = head_inner ? v.hs : v.ts, large = head_inner ? v.ts : v.hs;
  const int64_t inner = head_inner ? v.heads : v.tokens;
  if (small < dim || large < dim) return LIN_ERROR_INVALID_VALUE;
  if (v.hs % 8 != 0 || v.ts % 8 != 0) return LIN_ERROR_MISALIGNED;
  // (the tensor maps hold byte strides below 2^40)
  if (v.hs >= (1LL << 39) || v.ts >= (1LL << 39)) return LIN_ERROR_UNSUPPORTED_SHAPE;
  if (large < (inner - 1) * small + dim) return LIN_ERROR_INVALID_VALUE;
  if ((reinterpret_cast<uintptr_t>(v.t->data) & 15u) != 0) return LIN_ERROR_MISALIGNED;
  const unsigned __int128 ext =
      (unsigned __int128)(v.tokens - 1) * v.ts + (unsigned __int128)(v.heads - 1) * v.hs + dim;
  if (ext >> 61) return LIN_ERROR_UNSUPPORTED_SHAPE;
  v.extent = (uint64_t)ext * 2;
  return LIN_SUCCESS;
}

// Whether two views share an entry. Views whose ranges of memory meet may
// still be disjoint: the q, k and v heads of one buffer, whichever way its
// tokens and heads lie. Exact for equal strides (those of an extent of one
// count as any); views of other strides share an entry unless each token's
// heads of either lie within a row of the other's.
inline bool views_overlap(const View& a, const View& b, int64_t dim) {
  if (!overlaps(a.t->data, a.extent, b.t->data, b.extent)) return false;
  const int64_t ra = (a.heads - 1) * a.hs + dim, rb = (b.heads - 1) * b.hs + dim;
  // b's first entry from a's, in entries
  const int64_t d = (static_cast<const char*>(b.t->data) - static_cast<const char*>(a.t->data)) / 2;
  if (a.tokens > 1 && b.tokens > 1 && a.ts == b.ts && ra <= a.ts && rb <= a.ts) {
    const int64_t r = ((d % a.ts) + a.ts) % a.ts;   // b's row starts r entries into one of a's
    if (r >= ra && a.ts - r >= rb) return false;
  }
  if ((a.tokens > 1 && b.tokens > 1 && a.ts != b.ts) || (a.heads > 1 && b.heads > 1 && a.hs != b.hs))
    return true;
  // A head of b lies d + i ts + j hs from one of a, for the differences i of
  // their tokens and j of their heads: fewer than dim entries away, they meet.
  const int64_t ts = a.tokens > 1 ? a.ts : b.ts, hs = a.heads > 1 ? a.hs : b.hs;
  const int64_t i_lo = 1 - a.tokens, i_hi = b.tokens - 1;
  for (int64_t j = 1 - a.heads; j < b.heads; ++j) {
    const int64_t r = d + j * hs;
    const int64_t near = -r / ts;   // (toward zero: one of the two nearest is it or beside it)
    for (int64_t i = near - 1; i <= near + 1; ++i) {
      const int64_t at = r + std::min(std::max(i, i_lo), i_hi) * ts;
      if (at > -dim && at < dim) return true;
    }
  }
  return false;
}

inline lin::HeadsPtr heads_ptr(const View& v) {
  return lin::HeadsPtr{static_cast<uint16_t*>(v.t->data), v.ts, v.hs};
}

}  // namespace lin_detail
