// lin_attn_bwd.cuh -- attention backward from Q, K, V, O, each row's
// log-sum-exp L and dO, recomputing the probabilities:
//   P = 2^(c S - L log2 e), S = Q K^T, c = scale log2 e
//   delta_i = sum_d dO_id O_id (= sum_j P_ij dP_ij),  dP = dO V^T,
//   dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// in two kernels whose sums have a fixed order (no atomics): the first owns a
// tile of 128 queries and runs over the keys for dQ (three products a tile;
// it also leaves delta for the second), the second owns 128 keys of one key
// head and runs over the queries of every query head that shares it for dK
// and dV (four products a tile).
//
// The element-wise results that feed a product (dS, P^T, dS^T) are written as
// 16-bit operands into tensor memory over the f32 tile that they were made
// from. In binary16 their range is short (P of a long row is below 2^-14, and
// dS scales with dO, which a mean over many tokens makes small), so they are
// scaled by powers of two that are taken out again in f32 at the end: P by
// 2^8, dS so that the rows of dO count as having a norm near 2^4 (per row
// for dQ, where a row of dS meets only its own row of dQ; by the largest row
// norm that a key tile meets for dK: dS is off by up to 2^-29 of that norm).
//
// These roundings, one of each operand, are a choice: the tensor cores take both
// operands in one type, and dS in two parts would be two of the five products
// twice. dQ and dK are off by 4.2e-4 of their size in binary16 and 2.7e-3 in
// bfloat16, where sums of an f32 dS, rounded to that type at the end alone, are by
// 2.1e-4 and 1.7e-3.
//
// The streamed side comes in tiles of 64 rows, which take turns between two
// streams: each has its own S and dP in tensor memory and a warpgroup of its
// own, a thread to a row, so that one stream's element-wise work and the
// latencies between the roles pass while the tensor cores work for the other.
// S of a stream's next tile is issued behind the product that reads this
// tile's P (or behind its reading, in the dQ kernel), dP of the next behind
// the use of dS. One thread issues all of them, and its own steps count: a
// wait takes it some 100 cycles even for a barrier that is long complete, so
// a turn has as few as it can (one barrier for the pair of streamed tiles
// instead of one each: 703 -> 651 us at 8192 tokens; two issuing threads: 641
// for heads of 128, but 472 -> 509 for heads of 64). The CTA's own operands
// (Q and dO, or K and V) are in tensor memory beside the accumulators, which
// spares shared memory the reading of them; dK and dV of more than 64 entries
// leave no room for that.
//
// What bounds it. 8192 causal tokens, 16 heads of 128: 618-623 us, 1105 TF/s
// of the five products that the gradient needs and 1550 of the seven that the
// two kernels execute, 0.80 of the cuBLAS burst rate under the same power
// limit as the forward kernel. One kernel of five products would have to add
// dQ up over the key tiles: with atomics the order of the sums changes, and
// adds in a fixed order were not tried. Heads of 64, same lengths: 466 us,
// 0.53 of that rate: the element-wise work of a turn and the latencies between
// the roles. Short calls: 512 tokens, 12 heads 19 us, two kernels of four to
// eight turns each behind one another: the second needs no more of the first
// than delta and the norms of dO, but waits for its end.
//
// Where there are fewer tiles than SMs the other side is cut into parts, a
// CTA each, whose f32 sums a third kernel adds in order.
//
// SCORES: P is that of z = cap tanh(scale s / cap) - slope |distance| over each
// query's own range of keys, and dS has the cap's derivative as a factor. Each
// kernel runs over the tiles that its rows' ranges meet: the first from its
// rows' own, the second from what the first leaves for each of its tiles.
#pragma once

#include "lin_attn.cuh"

#include <algorithm>
#include <type_traits>

namespace lin {

namespace {

constexpr float kPShift = 8.0f;     // P^T is scaled by 2^8
constexpr int kNormExp = 4;         // dO rows count as having a norm near 2^4
constexpr int kRowWarps = 8;        // the two streams' warpgroups
constexpr int kDkvThreads = 384;
constexpr int kTailWarp = 10;       // of the dK, dV kernel: zeroes rows that take no part
constexpr int kStatsWarp = 11;      // of the dK, dV kernel: rows' statistics
constexpr int kTurn = 64;           // rows of a streamed tile
// (of a tile's extent, beside the key behind its last) some row without a key
// holds what a product with zero would not remove
constexpr int kBadFlag = 1 << 30;

// Shared memory and barriers of both kernels. A stage of the ring holds the
// streamed pair of tiles: A (K in the dQ kernel, Q in the other) and B (V, dO).
// OWN: the CTA's own operands are two tiles of 128 rows in shared memory.
template <int DP, int N_, int SUMS, bool OWN, int ROW_FLOATS>
struct BwdCfg {
  static constexpr int N = N_;                   // stages
  static constexpr bool kOwnSmem = OWN;
  using Tile = AttnTile<DP, kTurn>;
  static constexpr uint32_t TILE = Tile::BYTES;
  static constexpr int OWN_READY = 0;            // the CTA's own operands
  static constexpr int FULL = 1, EMPTY = FULL + N;
  static constexpr int TAIL = EMPTY + N;         // the stage, cut at the sequence's end
  // of each stream: S complete, dP complete, S read (dQ) or P^T written (dK,
  // dV), dS written
  static constexpr int S_FULL = TAIL + N, DP_FULL = S_FULL + 2;
  static constexpr int S_DONE = DP_FULL + 2, DS_READY = S_DONE + 2;
  static constexpr int SUM_READY = DS_READY + 2; // (dQ) the streams' sums of P dP
  static constexpr int OUT_FULL = SUM_READY + 1; // the sums complete (every product is)
  static constexpr int BARS = OUT_FULL + 1;
  static __device__ __forceinline__ uint32_t arrivals(int i) {
    // (a lane of each warp of rows: 8 warps, 4 of a stream)
    return i == SUM_READY || (i == OWN_READY && !OWN) ? 8 : i >= S_DONE && i < SUM_READY ? 4 : 1;
  }
  static __device__ __forceinline__ bool streamed_full(int i) { return i >= FULL && i < EMPTY; }
  static constexpr uint32_t OFF_TMEM = BARS * 8, OFF_ABORT = OFF_TMEM + 4;
  static constexpr uint32_t OFF_RED = 448;       // 16 floats
  static_assert(OFF_ABORT + 4 <= OFF_RED, "barrier region");
  static constexpr uint32_t OFF_OWN = 0;         // (tiles first: they want 1024-byte bases)
  static constexpr uint32_t OFF_A = OWN ? 2 * AttnTile<DP>::BYTES : 0;
  static constexpr uint32_t OFF_B = OFF_A + N * TILE;
  // dK, dV: [N][kTurn] floats -L log2 e + 8, then [N][kTurn] -a delta; dQ:
  // the rows' sums of dO O and dO^2, by halves
  static constexpr uint32_t OFF_ROWS = OFF_B + N * TILE;
  static constexpr uint32_t OFF_CTL = OFF_ROWS + ROW_FLOATS * 4;
  static constexpr uint32_t SMEM = OFF_CTL + 512;
  static_assert(SMEM <= 232448, "shared memory");
  // tensor memory: S of the two streams, dP of them (P^T and dS over them),
  // the sums (DP columns each), the CTA's own two operands
  static constexpr uint32_t S_COL = 0, DP_COL = 2 * kTurn, OUT_COL = 4 * kTurn;
  static constexpr uint32_t OWN_COL = OUT_COL + SUMS * DP;
  static_assert(OWN_COL + (OWN ? 0 : DP) <= 512, "tensor memory");
};
template <int DP>
using DqCfg = BwdCfg<DP, 6, 1, false, 4 * 128>;
// (a form of the scores: four more values of each row, two of each tile)
constexpr int dkv_stages(int dp, bool scores) { return dp == 64 ? 6 : scores ? 4 : 5; }
constexpr int dkv_rows(int dp, bool scores) {
  return dkv_stages(dp, scores) * ((scores ? 6 : 2) * kTurn + (scores ? 4 : 0));
}
template <int DP, bool SCORES>
using DkvCfg = BwdCfg<DP, dkv_stages(DP, SCORES), 2, (DP > 64), dkv_rows(DP, SCORES)>;

// The CTA's shared memory, which the tiles' swizzle wants at a multiple of
// 1024 bytes (it begins there: the kernels have no other shared memory). At
// any other place the kernel would compute nonsense: reported, never run.
__device__ __forceinline__ bool smem_aligned(const void* p, int* status) {
  if ((smem_u32(p) & 1023u) == 0) return true;
  if (threadIdx.x == 0) report_check(status, CHK_BUFFER, smem_u32(p));
  return false;
}

// Columns of packed results and operands into tensor memory.
template <int N>
__device__ __forceinline__ void tmem_put(uint32_t col, const uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 24 || N == 32, "columns");
  if constexpr (N == 32) {
    tmem_st_32x32b_x32(col, r);
  } else {
    tmem_st_32x32b_x16(col, reinterpret_cast<const uint32_t(&)[16]>(r));
    if constexpr (N == 24)
      tmem_st_32x32b_x8(col + 16, reinterpret_cast<const uint32_t(&)[8]>(r[16]));
  }
}

// 2^e as a float, e held to where 2^e and 2^-e are normal.
__device__ __forceinline__ float pow2i(int e) {
  return __int_as_float((min(max(e, -120), 120) + 127) << 23);
}
// The exponent e that brings a norm near 2^kNormExp when multiplied by 2^e;
// 0 for a norm of zero or one that is no number.
__device__ __forceinline__ int norm_exponent(float norm) {
  const int bits = __float_as_int(norm);
  const int ex = (bits >> 23) & 255;
  return ex == 0 || ex == 255 ? 0 : min(max(kNormExp - (ex - 127), -100), 100);
}

// Where a thread's row of a gradient goes: to the 16-bit tensor, or, as one
// of several parts, in f32 to [part][row][head][dim] (`rows` to a part, this
// one at `row_at`, which without parts may wrap and is not used).
struct HeadGrad {
  uint16_t* row;
  float* part_row;
  __device__ __forceinline__ HeadGrad(const HeadsPtr& t, float* parts_base, int parts, int part,
                                      int rows, uint32_t row_at, int heads, int dim,
                                      int64_t token, int h)
      : row(t.p + token * t.token_stride + (int64_t)h * t.head_stride),
        part_row(parts > 1 ? parts_base + ((part * rows + row_at) * heads + h) * dim : nullptr) {}
  // Checked build: the row inside its part.
  __device__ __forceinline__ bool ok(int* status, int rows, uint32_t row_at) const {
    return !part_row || dcheck(row_at < (uint32_t)rows, status, CHK_PART, row_at);
  }
  // N columns from c0 on, times `back` (zeros if there is nothing), those
  // below dim.
  template <bool BF16, int N>
  __device__ __forceinline__ void put(const uint32_t (&o)[N], bool any, float back, int c0,
                                      int dim) const {
#pragma unroll
    for (int g = 0; g < N / 8; ++g) {
      const int col = c0 + g * 8;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = any ? __uint_as_float(o[g * 8 + e]) * back : 0.0f;
      if (col >= dim) continue;
      if (part_row) {
        *reinterpret_cast<float4*>(part_row + col) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(part_row + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        store16(row + col, pack16<BF16>(v[0], v[1]), pack16<BF16>(v[2], v[3]),
                pack16<BF16>(v[4], v[5]), pack16<BF16>(v[6], v[7]));
      }
    }
  }
};

}  // namespace

// ---------------------------------------------------------------- dQ

template <int DP, bool BF16, int FORM>
__global__ void __launch_bounds__(kAttnThreads, 1)
    lin_attn_dq_kernel(const __grid_constant__ AttnBwdMaps maps,
                       const __grid_constant__ AttnBwdArgs args) {
  using C = DqCfg<DP>;
  constexpr bool SCORES = FORM != kNoForm;
  constexpr bool CAPPED = SCORES && (FORM & kCap), BIASED = SCORES && (FORM & kBias);
  static_assert(!C::kOwnSmem && C::OFF_OWN == 0, "own operands in tensor memory");
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = args.s;
  // rows i << shift | head of the CTA
  const int shift = args.shift, h0 = (int)blockIdx.x << shift;
  const PartOf at = part_of(blockIdx.z, args.q_parts);
  const int b = at.b, part = at.part;
  const int qt = gridDim.y - 1 - blockIdx.y;   // longest rows of a causal mask first
  const int r0 = qt * 128;
  const SeqRange sq = seq_range(a.cu_q, b, a.tokens_q, a.max_q);
  const int rows = sq.len << shift;
  const int64_t norm_at = ((int64_t)b * gridDim.x + blockIdx.x) * gridDim.y + qt;
  auto norm_ok = [&] {   // (checked build)
    return dcheck(norm_at >= 0 && norm_at < args.norms, a.status, CHK_STATS, norm_at);
  };
  // the keys that the tile's rows see, for the dK, dV kernel
  auto leave_extent = [&](const KeyRange& r) {
    if (SCORES && args.extents && threadIdx.x == 0 && part == 0 && norm_ok())
      args.extents[norm_at] = make_int2(r.lo, r.hi);
  };
  if (r0 >= rows) {   // (the whole CTA)
    if (threadIdx.x == 0 && part == 0 && norm_ok()) args.norm[norm_at] = 0.0f;
    leave_extent(KeyRange{INT_MAX, 0});
    return;
  }
  const SeqRange sk = seq_range(a.cu_k, b, a.tokens_k, a.max_k);
  // this part's key tiles: j0 .. j0 + n - 1 (one or two stay together: see delta)
  int tiles, j0, n;
  bool few;
  auto share = [&](int lo, int hi) {   // of the keys lo .. hi - 1
    const int from = lo / kTurn;
    tiles = hi > 0 ? (hi + kTurn - 1) / kTurn - from : 0;
    few = tiles <= 2;
    j0 = few ? 0 : at.begin(tiles);
    n = few ? (part == 0 ? tiles : 0) : at.end(tiles) - j0;
    j0 += from;
  };
  if constexpr (!SCORES) {
    const int last = min(r0 + 127, rows - 1) >> shift;
    share(0, a.causal ? min(sk.len, last + sk.len - sq.len + 1) : sk.len);
  }
  const int hk = h0 / a.group;

  if (!smem_aligned(smem_raw, a.status)) return;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* const ctl_gen = smem_raw + C::OFF_CTL;
  auto bar = [&](int slot) { return base + C::OFF_CTL + (uint32_t)slot * 8u; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = reinterpret_cast<volatile int*>(ctl_gen + C::OFF_ABORT);
  const WaitCtl ctl{a.timeout_ns, abort, a.status};
  auto k_tile = [&](int s) { return base + C::OFF_A + (uint32_t)s * C::TILE; };
  auto v_tile = [&](int s) { return base + C::OFF_B + (uint32_t)s * C::TILE; };

  if (warp == kAttnMmaWarp) {
    tmem_alloc(base + C::OFF_CTL + C::OFF_TMEM, 512);
    tmem_relinquish_alloc_permit();
  }
  if (tid == 0) *abort = 0;
  if (tid < C::BARS) {
    mbar_init(bar(tid), C::arrivals(tid));
    fence_barrier_init();
  }
  // the keys of this thread's row (row warps), and of all rows
  KeyRange mine{0, 0};
  int* const extents = reinterpret_cast<int*>(ctl_gen + C::OFF_RED) + 8;
  bool* const bad_rows = reinterpret_cast<bool*>(ctl_gen + C::OFF_RED + 16);   // 8, of the row warps
  if constexpr (SCORES) {
    if (warp < kRowWarps) {
      const int i = (r0 + (tid & 127)) >> shift;
      if (i < sq.len && q_row_ok(a, sq.start + i, h0)) mine = key_range(args.scores, a.causal, sq, sk, i);
      const KeyRange all = warp_extent(mine);
      if (lane == 0 && warp < 4) {
        extents[2 * warp] = all.lo;
        extents[2 * warp + 1] = all.hi;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_launch_dependents();   // (the dK, dV kernel waits for this grid's end before it reads)
  if constexpr (SCORES) {
    const KeyRange all = join_extents(extents, 4);
    share(all.lo, all.hi);   // (no key: nothing, whatever lo is)
  }
  // (an allocation of all 512 columns begins at column 0)
  constexpr uint32_t tmem = 0;
  constexpr uint32_t kQ = C::OWN_COL, kDo = kQ + DP / 2;   // Q and dO

  const int k_left = sk.len - (j0 + n - 1) * kTurn;   // keys of the last tile (kTurn or more: all)
  if (warp == kAttnCopyWarp) {
    if (lane == 0 && n > 0) {
      int issued = 0;
      RingAt<C::N> r;
      for (int j = 0; j < n; ++j, ++issued) {
        if (j >= C::N && !attn_wait(bar(C::EMPTY + r.s), r.parity ^ 1, ctl)) break;
        mbar_arrive_expect_tx(bar(C::FULL + r.s), 2 * C::TILE);
        if (stage_ok(a, r.s, C::N) && k_row_ok(a, sk.start + (j0 + j) * kTurn, hk)) {
          load_tile<DP, kTurn>(k_tile(r.s), &maps.k, hk, sk.start + (j0 + j) * kTurn,
                               bar(C::FULL + r.s));
          load_tile<DP, kTurn>(v_tile(r.s), &maps.v, hk, sk.start + (j0 + j) * kTurn,
                               bar(C::FULL + r.s));
        }
        r.next();
      }
      if (*abort) {   // no copy may still be in flight when the CTA ends
        for (int j = max(0, issued - C::N); j < issued; ++j)
          attn_wait(bar(C::FULL + j % C::N), (j / C::N) & 1, ctl, false);
      }
    }
    __syncwarp();
    if (n > 0 && k_left < kTurn) {   // cut the last K tile at the sequence's end (dS K runs over it)
      const int s = (n - 1) % C::N;
      if (warp_attn_wait(bar(C::FULL + s), ((n - 1) / C::N) & 1, ctl)) {
        if (dcheck(k_left > 0, a.status, CHK_BUFFER, k_left))
          zero_rows<DP, kTurn>(k_tile(s), k_left, kTurn, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::TAIL));
      }
    }
  } else if (warp == kAttnMmaWarp) {
    if (n > 0 && elect_one()) {   // one thread issues every product
      const uint64_t k_desc = C::Tile::k_major(k_tile(0)), v_desc = C::Tile::k_major(v_tile(0));
      const uint64_t kt_desc = C::Tile::mn_major(k_tile(0));
      constexpr uint64_t STAGE = C::Tile::UNITS;
      RingAt<C::N> r, next;   // stages of tile j, and of the next S and dP
      int nj = 0;             // tile of `next`
      auto scores = [&](int t) -> bool {   // S = Q K^T of the next tile
        if (!attn_wait(bar(C::FULL + next.s), next.parity, ctl) ||
            (++nj == n && k_left < kTurn && !attn_wait(bar(C::TAIL), 0, ctl)))
          return false;
        if (!stage_ok(a, next.s, C::N)) return false;
        umma_entries_tmem<DP, kTurn, BF16>(C::S_COL + t * kTurn, kQ, k_desc + next.s * STAGE);
        umma_commit(bar(C::S_FULL + t));
        return true;
      };
      auto dprobs = [&](int t) {   // dP = dO V^T of that tile
        umma_entries_tmem<DP, kTurn, BF16>(C::DP_COL + t * kTurn, kDo, v_desc + next.s * STAGE);
        umma_commit(bar(C::DP_FULL + t));
        next.next();
      };
      bool ok = attn_wait(bar(C::OWN_READY), 0, ctl);
      tc_fence_after_sync();
      for (int t = 0; t < 2 && t < n && ok; ++t) {
        ok = scores(t);
        if (ok) dprobs(t);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int t = j & 1, u = (j >> 1) & 1;
        if (j + 2 < n) {
          ok = attn_wait(bar(C::S_DONE + t), u, ctl);
          tc_fence_after_sync();
          ok = ok && scores(t);
        }
        ok = ok && attn_wait(bar(C::DS_READY + t), u, ctl);
        if (!ok) break;
        tc_fence_after_sync();
        umma_tokens<DP, BF16, kTurn / 16>(C::OUT_COL, C::DP_COL + t * kTurn, kt_desc + r.s * STAGE,
                                          0, j == 0);
        umma_commit(bar(C::EMPTY + r.s));
        r.next();
        if (j + 2 < n) dprobs(t);
      }
      // (also on the way out: tensor memory must be idle at the end)
      umma_commit(bar(C::OUT_FULL));
      attn_wait(bar(C::OUT_FULL), 0, ctl, false);
    }
    __syncwarp();
  } else if (warp < kRowWarps) {
    const int half = warp >> 2, row = tid & 127;
    const int i = (r0 + row) >> shift, h = h0 + (row & ((1 << shift) - 1));
    const int64_t token = sq.start + (i < sq.len ? i : 0);
    const bool live = i < sq.len && q_row_ok(a, token, h);
    const float c = a.scale * kLog2E;
    // The row's Q and dO into tensor memory; delta and the norm of dO on the
    // way: each of the row's two threads has half of the entries.
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    float dsum = 0.0f, nsum = 0.0f;
    const float lse = live ? args.lse[(int64_t)h * a.tokens_q + token] : -INFINITY;
    {
      auto row_of = [&](const HeadsPtr& t) {
        return live ? t.p + token * t.token_stride + (int64_t)h * t.head_stride : nullptr;
      };
      uint32_t x[DP / 4], y[DP / 4], z[DP / 4];
      load_row_part<DP, 2>(x, row_of(args.q), half, a.dim);
      load_row_part<DP, 2>(y, row_of(args.dout), half, a.dim);
      load_row_part<DP, 2>(z, row_of(args.o), half, a.dim);
      tmem_put<DP / 4>(tmem + lanes + kQ + half * (DP / 4), x);
      tmem_put<DP / 4>(tmem + lanes + kDo + half * (DP / 4), y);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::OWN_READY));
#pragma unroll
      for (int e = 0; e < DP / 4; ++e) {
        const float2 u = unpack16<BF16>(z[e]), v = unpack16<BF16>(y[e]);
        dsum = fmaf(u.x, v.x, fmaf(u.y, v.y, dsum));
        nsum = fmaf(v.x, v.x, fmaf(v.y, v.y, nsum));
      }
      if constexpr (SCORES) {
        // A row without a key has P = dS = 0, which the second kernel's products
        // over the queries multiply with its Q and dO: nothing, unless one of
        // these is no finite number, or so large that S or dP might not be. Such
        // rows, and only such, are zeroed there (all rows without keys, by a warp
        // between the copies and the products: nine sequences of up to 997 with
        // one row in twenty 47 -> 72 us).
        bool bad = false;
        if (__any_sync(0xffffffffu, live && mine.hi == 0)) {
          // (binary16: its largest products are far below float32's end; bfloat16: 2^15)
          constexpr uint32_t big = BF16 ? 0x4700u : 0x7c00u;
#pragma unroll
          for (int e = 0; e < DP / 4; ++e)
            bad |= (x[e] & 0x7fffu) >= big || ((x[e] >> 16) & 0x7fffu) >= big ||
                   (y[e] & 0x7fffu) >= big || ((y[e] >> 16) & 0x7fffu) >= big;
        }
        bad = __any_sync(0xffffffffu, bad && live && mine.hi == 0);
        if (lane == 0) bad_rows[warp] = bad;
      }
    }
    float* red = reinterpret_cast<float*>(smem_raw + C::OFF_ROWS);   // 4 x 128 floats
    red[half * 128 + row] = dsum;
    red[256 + half * 128 + row] = nsum;
    named_bar_sync(1, 256);
    float delta = red[row] + red[128 + row];
    const float norm = sqrtf(red[256 + row] + red[384 + row]);
    float* red2 = reinterpret_cast<float*>(ctl_gen + C::OFF_RED);
    if (half == 0) {
      if (live && (tiles == 0 || !few) && part == 0) args.delta[(int64_t)h * a.tokens_q + token] = delta;
      // (rows without a key, L = -inf, do not count, whatever their dO holds;
      // nor do NaN)
      float big = lse == -INFINITY ? 0.0f : norm;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      if (lane == 0) red2[warp] = big;
    }
    named_bar_sync(1, 256);
    if (tid == 0 && part == 0 && norm_ok())
      args.norm[norm_at] = fmaxf(fmaxf(red2[0], red2[1]), fmaxf(red2[2], red2[3]));
    if (SCORES && tid == 0) {
      bool bad = false;
      for (int w = 0; w < kRowWarps; ++w) bad |= bad_rows[w];
      const KeyRange all = join_extents(extents, 4);
      leave_extent(KeyRange{all.lo, all.hi | (bad ? kBadFlag : 0)});
    }
    const int ne = norm_exponent(norm);
    const float amp = pow2i(ne);
    float nd = -delta * amp;
    // a row without a key (L = -inf) has no probabilities
    float nl = lse == -INFINITY ? -INFINITY : -lse * kLog2E;
    // the last key that this row sees, and the first
    const int lim = SCORES ? mine.hi - 1
                    : live ? (a.causal ? min(sk.len - 1, i + sk.len - sq.len) : sk.len - 1)
                           : -1;
    const int low = SCORES ? mine.lo : 0;
    const ScoreTurn turned(args.scores, a.scale);
    const float slope = BIASED && live ? args.scores.slopes[h] * kLog2E : 0.0f;
    if (CAPPED) nl += turned.top;
    const uint32_t s_col = tmem + lanes + C::S_COL + half * kTurn;
    const uint32_t dp_col = tmem + lanes + C::DP_COL + half * kTurn;
    if (few && n == 1 && half == 1) {   // (no tile: nothing to the row's sums below)
      red[128 + row] = 0.0f;
      red[384 + row] = 0.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::SUM_READY));
    }
    bool ok = true;
    for (int j = half; j < n; j += 2) {   // the warpgroup's stream
      const int u = (j >> 1) & 1;
      // (of the row's keys in this tile; what a branch goes by is at hand when S comes)
      const int last_j = lim - (j0 + j) * kTurn, first_j = low - (j0 + j) * kTurn;
      const bool cut = CAPPED && __any_sync(0xffffffffu, last_j < kTurn - 1 || first_j > 0);
      ok = warp_attn_wait(bar(C::S_FULL + half), u, ctl);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t p[2][32], d[2][32];
      tmem_ld_32x32b_x32(s_col, p[0]);
      tmem_ld_32x32b_x32(s_col + 32, p[1]);
      tmem_wait_ld_x32(p[0]);
      tmem_wait_ld_x32(p[1]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::S_DONE + half));
      const float f = CAPPED ? -turned.twice : c;
      const float2 cc = make_float2(f, f), ll = make_float2(nl, nl);
      // P of two scores (capped: of their r)
      auto probability = [&](float2 x, float2 far) {
        x = fma2(x, cc, ll);
        if (BIASED)
          x = make_float2(fmaf(-slope, fabsf(far.x), x.x), fmaf(-slope, fabsf(far.y), x.y));
        return make_float2(ex2_approx(x.x), ex2_approx(x.y));
      };
      const float here = (float)(i + sk.len - sq.len - (j0 + j) * kTurn);   // (a bias)
      // All of the row's keys are in the streams' first tiles (few): delta is at
      // hand as the sum of P dP itself. It replaces the sum of dO O, whose O has
      // been rounded to 16 bits: with few keys that rounding is no longer small
      // against dP - delta (at one key the difference is zero).
      auto sum_delta = [&]() -> bool {
        float sd = 0.0f, sp = 0.0f;
        const int lim_h = lim - (SCORES ? j0 + half : half) * kTurn;
        const int low_h = SCORES ? low - (j0 + half) * kTurn : 0;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e <= lim_h && (!SCORES || q * 32 + e >= low_h)) {
              float x = __uint_as_float(p[q][e]);
              if (SCORES) x = probability(make_float2(x, x), make_float2(here - (q * 32 + e), 0.0f)).x;
              sd = fmaf(x, __uint_as_float(d[q][e]), sd);
              sp += x;
            }
        red[half * 128 + row] = sd;
        red[256 + half * 128 + row] = sp;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::SUM_READY));
        if (!warp_attn_wait(bar(C::SUM_READY), 0, ctl)) return false;
        sp = red[256 + row] + red[384 + row];
        delta = sp > 0.0f ? (red[row] + red[128 + row]) / sp : 0.0f;
        nd = -delta * amp;
        if (half == 0 && live) args.delta[(int64_t)h * a.tokens_q + token] = delta;
        return true;
      };
      auto take_dp = [&]() -> bool {
        if (!warp_attn_wait(bar(C::DP_FULL + half), u, ctl)) return false;
        tc_fence_after_sync();
        tmem_ld_32x32b_x32(dp_col, d[0]);
        tmem_ld_32x32b_x32(dp_col + 32, d[1]);
        tmem_wait_ld_x32(d[0]);
        tmem_wait_ld_x32(d[1]);
        return true;
      };
      if constexpr (SCORES) {
        // r of the scores (hidden ones zeroed: four share a reciprocal, and a row's
        // results do not go by what its mask hides), and from it P times the
        // cap's derivative
        auto rests = [&] {
          if (cut) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (q * 32 + e > last_j || q * 32 + e < first_j) p[q][e] = 0u;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 4) turned.rest4(&p[q][e]);
        };
        auto probabilities = [&] {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float2 far = make_float2(here - (float)(q * 32), here - (float)(q * 32 + 1));
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 r = make_float2(__uint_as_float(p[q][e]), __uint_as_float(p[q][e + 1]));
              float2 x = probability(r, far);
              if constexpr (BIASED) far = add2(far, make_float2(-2.0f, -2.0f));
              if constexpr (CAPPED) x = ScoreTurn::times_slope(x, r);
              p[q][e] = __float_as_uint(x.x);
              p[q][e + 1] = __float_as_uint(x.y);
            }
          }
        };
        if constexpr (CAPPED) rests();
        if (few) {
          ok = take_dp() && sum_delta();
          if (!ok) break;
          probabilities();
        } else {
          probabilities();
          ok = take_dp();
          if (!ok) break;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(p[q][e]), __uint_as_float(p[q][e + 1])), cc, ll);
            p[q][e] = __float_as_uint(ex2_approx(x.x));
            p[q][e + 1] = __float_as_uint(ex2_approx(x.y));
          }
      }
      if constexpr (!SCORES) {
        ok = take_dp();
        if (ok && few) ok = sum_delta();
        if (!ok) break;
      }
      const float2 aa = make_float2(amp, amp), dd = make_float2(nd, nd);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(d[q][e]), __uint_as_float(d[q][e + 1])), aa, dd);
          const float2 y = mul2(make_float2(__uint_as_float(p[q][e]), __uint_as_float(p[q][e + 1])), x);
          d[q][e] = __float_as_uint(y.x);
          d[q][e + 1] = __float_as_uint(y.y);
        }
      if constexpr (SCORES) {
        const int low_j = low - (j0 + j) * kTurn;
        if (__any_sync(0xffffffffu, low_j > 0)) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e < low_j) d[q][e] = 0u;
        }
      }
      const int lim_j = lim - (j0 + j) * kTurn;
      if (__any_sync(0xffffffffu, lim_j < kTurn - 1)) {   // masked keys, whatever their dP holds
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e > lim_j) d[q][e] = 0u;
      }
      uint32_t w[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        w[e] = pack16<BF16>(__uint_as_float(d[e >> 4][(2 * e) & 31]),
                            __uint_as_float(d[e >> 4][(2 * e + 1) & 31]));
      tmem_st_32x32b_x32(dp_col, w);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::DS_READY + half));
    }
    if (ok && n > 0) {
      ok = warp_attn_wait(bar(C::OUT_FULL), 0, ctl);
      tc_fence_after_sync();
    }
    if (ok) {
      const float back = a.scale * pow2i(-ne);
      const HeadGrad out(args.dq, args.dq_part, args.q_parts, part, args.q_part_rows,
                         (uint32_t)b * a.max_q + i, a.heads_q, a.dim, token, h);
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        const int c0 = half * (DP / 2) + q * 16;
        uint32_t o[16];
        if (n > 0) {
          tmem_ld_32x32b_x16(tmem + lanes + C::OUT_COL + c0, o);
          tmem_wait_ld_x16(o);
        }
        const bool put = live && out.ok(a.status, args.q_part_rows, (uint32_t)b * a.max_q + i);
        out.put<BF16>(o, n > 0, back, c0, put ? a.dim : 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kAttnMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dK, dV

template <int DP, bool BF16, int FORM>
__global__ void __launch_bounds__(kDkvThreads, 1)
    lin_attn_dkv_kernel(const __grid_constant__ AttnBwdMaps maps,
                        const __grid_constant__ AttnBwdArgs args) {
  constexpr bool SCORES = FORM != kNoForm;
  constexpr bool CAPPED = SCORES && (FORM & kCap), BIASED = SCORES && (FORM & kBias);
  using C = DkvCfg<DP, SCORES>;
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = args.s;
  const int hk = blockIdx.x;
  const PartOf at = part_of(blockIdx.z, args.k_parts);
  const int b = at.b, part = at.part;
  const int k0 = blockIdx.y * 128;   // a causal mask's first keys meet the most queries
  const SeqRange sk = seq_range(a.cu_k, b, a.tokens_k, a.max_k);
  if (k0 >= sk.len) {   // (the whole CTA)
    // The grid's end has to stand for the dQ kernel's too, for whatever waits
    // for it next, even where no CTA of it has a key. One that waits is enough
    // (nine sequences of up to 997: 63.7 us a call; if all do, they keep the
    // others from starting: 64.6).
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0) pdl_wait();
    return;
  }
  const SeqRange sq = seq_range(a.cu_q, b, a.tokens_q, a.max_q);
  // Rows i << shift | head of the group (shift 0: the heads one after another),
  // in tiles t0 .. t1 - 1 of each pass over them.
  const int shift = args.shift;
  const int off = sk.len - sq.len;   // causal: query i sees the keys up to i + off
  const int rows = sq.len << shift;
  int t1 = (rows + kTurn - 1) / kTurn;
  int t0 = a.causal ? min((max(k0 - off, 0) << shift) / kTurn, t1) : 0;
  const bool ranged = SCORES && args.extents != nullptr;
  bool holes = false;   // (in some tile of the sequence) rows to be zeroed: see kBadFlag
  float met = 0.0f;     // (ranges) the largest row norm of dO of the tiles that see one of these keys
  if (ranged) {
    // the first and the last tile of 128 rows that see one of these keys
    pdl_wait();
    const int tiles = ((a.max_q << shift) + 127) / 128;
    const int heads = a.group >> shift;   // (tiles of them)
    const int64_t ext = ((int64_t)b * gridDim.x + hk) * tiles * heads;
    int lo = INT_MAX, hi = -1, bad = 0, big = 0;
    for (int k = threadIdx.x & 31; k < tiles * heads; k += 32) {
      const int i = k % tiles;
      if (!dcheck(ext + k < args.norms, a.status, CHK_STATS, k)) continue;
      const int2 e = args.extents[ext + k];
      const int norm = __float_as_int(args.norm[ext + k]);   // (not negative: ordered as it is)
      bad |= e.y & kBadFlag;
      if (e.x < k0 + 128 && (e.y & ~kBadFlag) > k0) {
        lo = min(lo, i);
        hi = max(hi, i);
        big = max(big, norm);
      }
    }
    holes = __any_sync(0xffffffffu, bad);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    met = __int_as_float(__reduce_max_sync(0xffffffffu, big));
    t1 = min(t1, 2 * hi + 2);
    t0 = min(max(t0, lo < INT_MAX ? 2 * lo : 0), t1);
  }
  const int per = t1 - t0;
  // this part's turns (of all passes' tiles): from .. from + n - 1
  const int passes = a.group >> shift;
  const int from = at.begin(per * passes), n = at.end(per * passes) - from;
  const int tile0 = from > 0 ? from % per : 0;           // the first turn's tile of its pass
  const int q_left = rows - (t1 - 1) * kTurn;            // rows of the last tile
  // rows of the first tile that see no key at all (more queries than keys)
  const int q_none = a.causal ? (max(-off, 0) << shift) - t0 * kTurn : 0;
  const bool cut_rows = holes || q_left < kTurn || q_none > 0;
  const int h0 = hk * a.group;

  if (!smem_aligned(smem_raw, a.status)) return;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* const ctl_gen = smem_raw + C::OFF_CTL;
  auto bar = [&](int slot) { return base + C::OFF_CTL + (uint32_t)slot * 8u; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = reinterpret_cast<volatile int*>(ctl_gen + C::OFF_ABORT);
  const WaitCtl ctl{a.timeout_ns, abort, a.status};
  auto q_tile = [&](int s) { return base + C::OFF_A + (uint32_t)s * C::TILE; };
  auto do_tile = [&](int s) { return base + C::OFF_B + (uint32_t)s * C::TILE; };
  auto lse_rows = [&](int s) { return reinterpret_cast<float*>(smem_raw + C::OFF_ROWS) + s * kTurn; };
  auto delta_rows = [&](int s) { return lse_rows(C::N + s); };
  // (a form of the scores) the rows' places among the keys, slopes, first keys
  // and those behind their last, and a tile's largest first and smallest end
  auto place_rows = [&](int s) { return lse_rows(2 * C::N + s); };
  auto slope_rows = [&](int s) { return lse_rows(3 * C::N + s); };
  auto first_rows = [&](int s) { return reinterpret_cast<int*>(lse_rows(4 * C::N + s)); };
  auto end_rows = [&](int s) { return reinterpret_cast<int*>(lse_rows(5 * C::N + s)); };
  auto tile_keys = [&](int s) { return reinterpret_cast<int*>(lse_rows(6 * C::N)) + 4 * s; };

  if (warp == kAttnMmaWarp) {
    tmem_alloc(base + C::OFF_CTL + C::OFF_TMEM, 512);
    tmem_relinquish_alloc_permit();
  }
  if (tid == 0) *abort = 0;
  if (tid < C::BARS) {
    // (a stage has the copy's arrival and the statistics')
    mbar_init(bar(tid), C::streamed_full(tid) ? 2 : C::arrivals(tid));
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // (an allocation of all 512 columns begins at column 0)
  constexpr uint32_t tmem = 0;
  constexpr uint32_t kK = C::OWN_COL, kV = kK + DP / 2;   // K and V (heads of up to 64)
  const uint32_t k_own = base + C::OFF_OWN, v_own = k_own + AttnTile<DP>::BYTES;   // (of 128)
  // The exponent of dS's scale, from the largest row norm of dO that this tile
  // of keys meets, in tiles of 128 rows: behind a causal mask from the one of
  // its first turn on (the rows before it may be larger by more than binary16
  // spans), with ranges of keys of the tiles that see one of its keys (other
  // documents' may be as much larger). By each warp that wants it, once the dQ
  // kernel, which leaves the norms and delta, is done; the copies and the first
  // products do not wait for that.
  auto scale_exponent = [&]() -> int {
    if (ranged) return norm_exponent(met);
    pdl_wait();
    const int tiles = ((a.max_q << shift) + 127) / 128;
    const float* nm = args.norm + ((int64_t)b * gridDim.x + hk) * tiles * passes;
    float big = 0.0f;
    for (int p = 0; p < passes; ++p, nm += tiles)
      for (int i = t0 * kTurn / 128 + lane; i < tiles; i += 32)
        if (dcheck(nm + i < args.norm + args.norms, a.status, CHK_STATS, nm + i - args.norm))
          big = fmaxf(big, nm[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    return norm_exponent(big);
  };
  // scale of dP and delta: dS then carries 2^ne, P's 2^8 taken back
  auto ds_scale = [&](int ne) { return pow2i(ne) * pow2i(-(int)kPShift); };

  if (warp == kAttnCopyWarp) {
    if (n > 0) {
      if (C::kOwnSmem && lane == 0) {
        mbar_arrive_expect_tx(bar(C::OWN_READY), 2 * AttnTile<DP>::BYTES);
#pragma unroll
        for (int r = 0; r < 128; r += kTurn)
#pragma unroll
          for (int s = 0; s < AttnTile<DP>::SUB; ++s) {
            const uint32_t at = s * AttnTile<DP>::SUB_BYTES + r * 128;
            tma_load_3d(k_own + at, &maps.k, s * 64, hk, sk.start + k0 + r, bar(C::OWN_READY));
            tma_load_3d(v_own + at, &maps.v, s * 64, hk, sk.start + k0 + r, bar(C::OWN_READY));
          }
      }
      if (lane == 0) {
        int issued = 0;
        RingAt<C::N> r;
        int h = h0 + from / per, tile = tile0;   // of this turn (n > 0: per > 0)
        for (int it = 0; it < n; ++it, ++issued) {
          const int z = sq.start + ((t0 + tile) * kTurn >> shift);
          if (it >= C::N && !attn_wait(bar(C::EMPTY + r.s), r.parity ^ 1, ctl)) break;
          mbar_arrive_expect_tx(bar(C::FULL + r.s), 2 * C::TILE);
          if (stage_ok(a, r.s, C::N) && q_row_ok(a, z, h + (1 << shift) - 1)) {
            load_tile<DP, kTurn>(q_tile(r.s), &maps.q, h, z, bar(C::FULL + r.s));
            load_tile<DP, kTurn>(do_tile(r.s), &maps.dout, h, z, bar(C::FULL + r.s));
          }
          r.next();
          if (++tile == per) {
            tile = 0;
            ++h;
          }
        }
        if (*abort) {   // no copy may still be in flight when the CTA ends
          if (C::kOwnSmem) attn_wait(bar(C::OWN_READY), 0, ctl, false);
          for (int it = max(0, issued - C::N); it < issued; ++it)
            attn_wait(bar(C::FULL + it % C::N), (it / C::N) & 1, ctl, false);
        }
      }
    }
  } else if (!SCORES && warp == kStatsWarp) {
    // The rows' statistics of each turn, in the form that the element-wise
    // warps add: rows behind the sequence's end and rows without a key have
    // P = 0. A warp of its own, which has the next turn's on their way while it
    // waits for a stage: with these loads between its copies the copying warp
    // took longer for a turn than the products (3000 cycles; 757 us at 8192
    // tokens).
    constexpr int N = kTurn / 32;
    const float damp = ds_scale(scale_exponent());
    RingAt<C::N> r;
    int h = n > 0 ? h0 + from / per : 0, tile = tile0;
    float lse[N], delta[N];
    auto load = [&]() {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int r = (t0 + tile) * kTurn + e * 32 + lane, i = r >> shift;
        const int hr = h + (r & ((1 << shift) - 1));
        const int64_t at = (int64_t)hr * a.tokens_q + sq.start + i;
        const bool in = i < sq.len && q_row_ok(a, sq.start + i, hr);
        lse[e] = in ? args.lse[at] : -INFINITY;
        delta[e] = in ? args.delta[at] : 0.0f;
      }
      if (++tile == per) {
        tile = 0;
        ++h;
      }
    };
    if (n > 0) load();
    for (int it = 0; it < n; ++it) {
      float nl[N], nd[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        nl[e] = lse[e] == -INFINITY ? -INFINITY : fmaf(-lse[e], kLog2E, kPShift);
        nd[e] = delta[e] * -damp;
      }
      if (it + 1 < n) load();
      if (it >= C::N && !warp_attn_wait(bar(C::EMPTY + r.s), r.parity ^ 1, ctl)) break;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        lse_rows(r.s)[e * 32 + lane] = nl[e];
        delta_rows(r.s)[e * 32 + lane] = nd[e];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::FULL + r.s));
      r.next();
    }
  } else if (SCORES && warp == kStatsWarp) {
    // The same with a form of the scores: each row's place among the keys and
    // slope, its range of keys, and what all of a tile's rows see.
    constexpr int N = kTurn / 32;
    const float damp = ds_scale(scale_exponent());
    const ScoreTurn turned(args.scores, a.scale);
    int h = n > 0 ? h0 + from / per : 0, tile = tile0;   // of the next loads
    struct Rows {
      float lse[N], delta[N], slope[N];
      KeyRange keys[N];
      int i[N];   // (-1: no row)
    } ahead[2];
    auto load = [&](Rows& to) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int row = (t0 + tile) * kTurn + e * 32 + lane, i = row >> shift;
        const int hr = h + (row & ((1 << shift) - 1));
        const int64_t at = (int64_t)hr * a.tokens_q + sq.start + i;
        const bool in = i < sq.len && q_row_ok(a, sq.start + i, hr);
        to.lse[e] = in ? args.lse[at] : -INFINITY;
        to.delta[e] = in ? args.delta[at] : 0.0f;
        to.slope[e] = BIASED && in ? args.scores.slopes[hr] : 0.0f;
        to.keys[e] = in ? load_keys(args.scores, sq, sk, i) : KeyRange{0, 0};
        to.i[e] = in ? i : -1;
      }
      if (++tile == per) {
        tile = 0;
        ++h;
      }
    };
    if (n > 0) load(ahead[0]);
    if (n > 1) load(ahead[1]);
    RingAt<C::N> r;
    bool ok = true;
    for (int it = 0; it < n && ok; it += 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (it + k >= n || !ok) break;
        Rows& rows = ahead[k];
        float nl[N], nd[N];
        KeyRange keys[N];
        int first = 0, end = INT_MAX;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          // (rows behind the end and rows without a key have P = 0 already)
          keys[e] = rows.i[e] < 0 ? KeyRange{0, 0} : held_keys(rows.keys[e], a.causal, sq, sk, rows.i[e]);
          // (a capped score is a line in r: its constant with the rest of P's exponent)
          nl[e] = rows.lse[e] == -INFINITY
                      ? -INFINITY
                      : fmaf(-rows.lse[e], kLog2E, CAPPED ? kPShift + turned.top : kPShift);
          // (a row without a key: whatever its dO held)
          nd[e] = rows.lse[e] == -INFINITY ? 0.0f : rows.delta[e] * -damp;
          if (keys[e].hi > 0) {
            first = max(first, keys[e].lo);
            end = min(end, keys[e].hi);
          }
        }
        first = __reduce_max_sync(0xffffffffu, first);
        end = __reduce_min_sync(0xffffffffu, end);
        if (it + k >= C::N) ok = warp_attn_wait(bar(C::EMPTY + r.s), r.parity ^ 1, ctl);
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          lse_rows(r.s)[e * 32 + lane] = nl[e];
          delta_rows(r.s)[e * 32 + lane] = nd[e];
          if constexpr (BIASED) {
            place_rows(r.s)[e * 32 + lane] = (float)(rows.i[e] + off);
            slope_rows(r.s)[e * 32 + lane] = rows.slope[e] * kLog2E;
          }
          first_rows(r.s)[e * 32 + lane] = keys[e].lo;
          end_rows(r.s)[e * 32 + lane] = keys[e].hi;
        }
        if (lane == 0) {
          tile_keys(r.s)[0] = first;
          tile_keys(r.s)[1] = end;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::FULL + r.s));
        r.next();
        if (it + k + 2 < n) load(rows);
      }
    }
  } else if (warp == kTailWarp) {
    // Where the last query tile of a head is cut by the sequence's end, or its
    // first one begins with rows without a key, this warp hands every stage on
    // to the products (a phase that nobody waited for would not be told from
    // the one before it), those tiles with such rows zeroed: they enter the
    // products that run over the queries.
    if (n > 0 && cut_rows) {
      int tile = tile0;
      RingAt<C::N> r;
      for (int it = 0; it < n; ++it) {
        if (!warp_attn_wait(bar(C::FULL + r.s), r.parity, ctl)) break;
        // (holes: the rows without a key, by the ranges that came with the stage)
        uint32_t none[2] = {0u, 0u};
        if (holes) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            none[e] = __ballot_sync(0xffffffffu, end_rows(r.s)[e * 32 + lane] == 0);
        }
        if (none[0] | none[1]) {
          constexpr int UNITS = C::Tile::SUB * 8;   // 16-byte units of a row
#pragma unroll
          for (int e = 0; e < 2; ++e)
            for (uint32_t left = none[e]; left; left &= left - 1) {
              const uint32_t at = (uint32_t)(e * 32 + __ffs((int)left) - 1) * 128u +
                                  (uint32_t)(lane % UNITS / 8) * C::Tile::SUB_BYTES + (lane & 7) * 16u;
              if (lane < 2 * UNITS) st_shared_v4((lane < UNITS ? q_tile(r.s) : do_tile(r.s)) + at, 0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
        }
        if (tile == 0 && q_none > 0 && stage_ok(a, r.s, C::N) &&
            dcheck(q_none < kTurn, a.status, CHK_BUFFER, q_none)) {
          zero_rows<DP, kTurn>(q_tile(r.s), 0, q_none, lane);
          zero_rows<DP, kTurn>(do_tile(r.s), 0, q_none, lane);
          fence_proxy_async_smem();
        }
        if (++tile == per) {
          tile = 0;
          if (q_left < kTurn && dcheck(q_left > 0, a.status, CHK_BUFFER, q_left)) {
            zero_rows<DP, kTurn>(q_tile(r.s), q_left, kTurn, lane);
            zero_rows<DP, kTurn>(do_tile(r.s), q_left, kTurn, lane);
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::TAIL + r.s));
        r.next();
      }
    }
  } else if (warp == kAttnMmaWarp) {
    if (n > 0 && elect_one()) {   // one thread issues every product
      const uint64_t q_desc = C::Tile::k_major(q_tile(0)), do_desc = C::Tile::k_major(do_tile(0));
      const uint64_t qt_desc = C::Tile::mn_major(q_tile(0));
      const uint64_t dot_desc = C::Tile::mn_major(do_tile(0));
      constexpr uint64_t STAGE = C::Tile::UNITS;
      const int ready = cut_rows ? C::TAIL : C::FULL;
      RingAt<C::N> r, next;   // stages of turn it, and of the next S^T and dP^T
      auto own = [&](uint32_t d, uint32_t col, uint32_t tile, uint64_t other) {
        if constexpr (C::kOwnSmem)
          umma_entries<DP, BF16, kTurn>(d, AttnTile<DP>::k_major(tile), other);
        else
          umma_entries_tmem<DP, kTurn, BF16>(d, col, other);
      };
      auto scores = [&](int t) -> bool {   // S^T = K Q^T of the next turn
        if (!attn_wait(bar(ready + next.s), next.parity, ctl)) return false;
        if (!stage_ok(a, next.s, C::N)) return false;
        own(C::S_COL + t * kTurn, kK, k_own, q_desc + next.s * STAGE);
        umma_commit(bar(C::S_FULL + t));
        return true;
      };
      auto dprobs = [&](int t) {   // dP^T = V dO^T of that turn
        own(C::DP_COL + t * kTurn, kV, v_own, do_desc + next.s * STAGE);
        umma_commit(bar(C::DP_FULL + t));
        next.next();
      };
      bool ok = attn_wait(bar(C::OWN_READY), 0, ctl);
      tc_fence_after_sync();
      for (int t = 0; t < 2 && t < n && ok; ++t) {
        ok = scores(t);
        if (ok) dprobs(t);
      }
      for (int it = 0; it < n && ok; ++it) {
        const int t = it & 1, u = (it >> 1) & 1;
        ok = attn_wait(bar(C::S_DONE + t), u, ctl);
        if (!ok) break;
        tc_fence_after_sync();
        umma_tokens<DP, BF16, kTurn / 16>(C::OUT_COL, C::S_COL + t * kTurn, dot_desc + r.s * STAGE,
                                          0, it == 0);   // dV += P^T dO
        if (it + 2 < n) ok = scores(t);
        ok = ok && attn_wait(bar(C::DS_READY + t), u, ctl);
        if (!ok) break;
        tc_fence_after_sync();
        umma_tokens<DP, BF16, kTurn / 16>(C::OUT_COL + DP, C::DP_COL + t * kTurn,
                                          qt_desc + r.s * STAGE, 0, it == 0);   // dK += dS^T Q
        umma_commit(bar(C::EMPTY + r.s));
        r.next();
        if (it + 2 < n) dprobs(t);
      }
      // (also on the way out: tensor memory must be idle at the end)
      umma_commit(bar(C::OUT_FULL));
      attn_wait(bar(C::OUT_FULL), 0, ctl, false);
    }
    __syncwarp();
  } else if (warp < kRowWarps) {
    const int half = warp >> 2, row = tid & 127;
    const int key = k0 + row;
    const bool live = key < sk.len && k_row_ok(a, (int64_t)sk.start + key, hk);
    const float c = a.scale * kLog2E;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + C::S_COL + half * kTurn;
    const uint32_t dp_col = tmem + lanes + C::DP_COL + half * kTurn;
    if constexpr (!C::kOwnSmem) {   // the row's K and V into tensor memory, half by each thread
      auto row_of = [&](const HeadsPtr& t) {
        return live ? t.p + (int64_t)(sk.start + key) * t.token_stride + (int64_t)hk * t.head_stride
                    : nullptr;
      };
      uint32_t x[DP / 4], y[DP / 4];
      load_row_part<DP, 2>(x, row_of(args.k), half, a.dim);
      load_row_part<DP, 2>(y, row_of(args.v), half, a.dim);
      tmem_put<DP / 4>(tmem + lanes + kK + half * (DP / 4), x);
      tmem_put<DP / 4>(tmem + lanes + kV + half * (DP / 4), y);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::OWN_READY));
    }
    const int ne = scale_exponent();
    const float damp = ds_scale(ne);
    const ScoreTurn turned(args.scores, a.scale);
    const float my_key = (float)key;
    constexpr int NQ = kTurn / 32;   // groups of 32 columns of a thread
    bool ok = true;
    int tile = per > 0 ? (tile0 + half) % per : 0;   // of its pass
    const int from_row = max(key - off, 0) << shift;
    RingAt<C::N> r;
    if (half) r.next();
    for (int it = half; it < n; it += 2) {   // the warpgroup's stream
      const int u = (it >> 1) & 1;
      const int i0 = (t0 + tile) * kTurn;
      for (tile += 2; tile >= per;) tile -= per;
      const float4* nl = reinterpret_cast<const float4*>(lse_rows(r.s));
      const float4* nd = reinterpret_cast<const float4*>(delta_rows(r.s));
      ok = warp_attn_wait(bar(C::S_FULL + half), u, ctl);
      if (!ok) break;
      // (the stage was full before S was formed)
      ok = warp_attn_wait(bar(C::FULL + r.s), r.parity, ctl);
      if (!ok) break;
      const int at_stage = r.s;
      r.next();
      r.next();
      tc_fence_after_sync();
      uint32_t p[NQ][32], d[NQ][32], w[NQ * 16];
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_ld_32x32b_x32(s_col + q * 32, p[q]);
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_wait_ld_x32(p[q]);
      const float f = CAPPED ? -turned.twice : c;
      const float2 cc = make_float2(f, f), pp = make_float2(damp, damp);
      bool cut;
      int first = 0;
      if constexpr (SCORES) {
        const int* bounds = tile_keys(at_stage);
        const bool cut_first = bounds[0] > k0, cut_end = bounds[1] < min(k0 + 128, sk.len);
        cut = cut_first || cut_end;
        if constexpr (CAPPED) {   // r
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = turned.rest(make_float2(__uint_as_float(p[q][e]), __uint_as_float(p[q][e + 1])));
              p[q][e] = __float_as_uint(x.x);
              p[q][e + 1] = __float_as_uint(x.y);
            }
        }
        // what leaves no probability, whatever else is added (of a cap's r: -2^80
        // at its smallest, times a slope of -0)
        const uint32_t out = __float_as_uint(CAPPED ? 1e30f : -INFINITY);
        auto leave_out = [&](const int* rows, auto outside) {
          const int4* at = reinterpret_cast<const int4*>(rows);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int4 b = at[q * 8 + e];
              uint32_t* x = &p[q][e * 4];
              if (outside(b.x)) x[0] = out;
              if (outside(b.y)) x[1] = out;
              if (outside(b.z)) x[2] = out;
              if (outside(b.w)) x[3] = out;
            }
        };
        if (cut_first) leave_out(first_rows(at_stage), [&](int b) { return key < b; });
        if (cut_end) leave_out(end_rows(at_stage), [&](int b) { return key >= b; });
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 l = nl[q * 8 + e];
            uint32_t* x = &p[q][e * 4];
            const float2 ru = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
            const float2 rv = make_float2(__uint_as_float(x[2]), __uint_as_float(x[3]));
            float2 u = fma2(ru, cc, make_float2(l.x, l.y));
            float2 v = fma2(rv, cc, make_float2(l.z, l.w));
            if constexpr (BIASED) {
              const float4 at = reinterpret_cast<const float4*>(place_rows(at_stage))[q * 8 + e];
              const float4 sl = reinterpret_cast<const float4*>(slope_rows(at_stage))[q * 8 + e];
              u = make_float2(fmaf(-sl.x, fabsf(at.x - my_key), u.x), fmaf(-sl.y, fabsf(at.y - my_key), u.y));
              v = make_float2(fmaf(-sl.z, fabsf(at.z - my_key), v.x), fmaf(-sl.w, fabsf(at.w - my_key), v.y));
            }
            u = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            v = make_float2(ex2_approx(v.x), ex2_approx(v.y));
            w[q * 16 + e * 2] = pack16<BF16>(u.x, u.y);
            w[q * 16 + e * 2 + 1] = pack16<BF16>(v.x, v.y);
            if constexpr (CAPPED) {   // (P itself is not wanted any more)
              u = ScoreTurn::times_slope(u, ru);
              v = ScoreTurn::times_slope(v, rv);
            }
            x[0] = __float_as_uint(u.x);
            x[1] = __float_as_uint(u.y);
            x[2] = __float_as_uint(v.x);
            x[3] = __float_as_uint(v.y);
          }
      } else {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 r = nl[q * 8 + e];
            uint32_t* x = &p[q][e * 4];
            const float2 u = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), cc,
                                  make_float2(r.x, r.y));
            const float2 v = fma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), cc,
                                  make_float2(r.z, r.w));
            x[0] = __float_as_uint(ex2_approx(u.x));
            x[1] = __float_as_uint(ex2_approx(u.y));
            x[2] = __float_as_uint(ex2_approx(v.x));
            x[3] = __float_as_uint(ex2_approx(v.y));
          }
        // causal: the key meets the queries from key - off on, the rows from_row on
        first = from_row - i0;
        cut = a.causal && __any_sync(0xffffffffu, first > 0);
        if (cut) {
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e < first) p[q][e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < NQ * 16; ++e)
          w[e] = pack16<BF16>(__uint_as_float(p[e >> 4][(2 * e) & 31]),
                              __uint_as_float(p[e >> 4][(2 * e + 1) & 31]));
      }
      tmem_put<NQ * 16>(s_col, w);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::S_DONE + half));
      ok = warp_attn_wait(bar(C::DP_FULL + half), u, ctl);
      if (!ok) break;
      tc_fence_after_sync();
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_ld_32x32b_x32(dp_col + q * 32, d[q]);
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_wait_ld_x32(d[q]);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 r = nd[q * 8 + e];
          uint32_t* x = &d[q][e * 4];
          const uint32_t* y = &p[q][e * 4];
          const float2 u = mul2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                                fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), pp,
                                     make_float2(r.x, r.y)));
          const float2 v = mul2(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                                fma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), pp,
                                     make_float2(r.z, r.w)));
          x[0] = __float_as_uint(u.x);
          x[1] = __float_as_uint(u.y);
          x[2] = __float_as_uint(v.x);
          x[3] = __float_as_uint(v.y);
        }
      if (SCORES && cut) {   // masked keys, whatever their dP holds
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (__uint_as_float(p[q][e]) == 0.0f) d[q][e] = 0u;   // (of either sign: see `out`)
      } else if (cut) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e < first) d[q][e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < NQ * 16; ++e)
        w[e] = pack16<BF16>(__uint_as_float(d[e >> 4][(2 * e) & 31]),
                            __uint_as_float(d[e >> 4][(2 * e + 1) & 31]));
      tmem_put<NQ * 16>(dp_col, w);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::DS_READY + half));
    }
    if (ok && n > 0) {
      ok = warp_attn_wait(bar(C::OUT_FULL), 0, ctl);
      tc_fence_after_sync();
    }
    if (ok) {   // the first half's threads write dV, the others dK
      const float back = half == 0 ? pow2i(-(int)kPShift) : a.scale * pow2i(-ne);
      const HeadGrad out(half == 0 ? args.dv : args.dk, half == 0 ? args.dv_part : args.dk_part,
                         args.k_parts, part, args.k_part_rows, (uint32_t)b * a.max_k + key,
                         a.heads_q / a.group, a.dim, (int64_t)sk.start + (live ? key : 0), hk);
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + C::OUT_COL + half * DP + q * 32, o);
          tmem_wait_ld_x32(o);
        }
        const bool put = live && out.ok(a.status, args.k_part_rows, (uint32_t)b * a.max_k + key);
        out.put<BF16>(o, n > 0, back, q * 32, put ? a.dim : 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kAttnMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// The two kernels of the arguments' head size and type.
template <int FORM>
cudaError_t launch_attn_bwd(bool bf16, const AttnBwdMaps& maps, const AttnBwdArgs& args,
                            int heads_kv, int sequences, int* kernels, cudaStream_t stream) {
  const unsigned tq = (unsigned)(((args.s.max_q << args.shift) + 127) / 128);
  const unsigned tk = (unsigned)((args.s.max_k + 127) / 128);
  const unsigned hq = (unsigned)(heads_kv * args.s.group), hk = (unsigned)heads_kv;
  const unsigned seqs = (unsigned)sequences;
  *kernels = 0;
  auto go = [&](auto kernel, uint32_t smem, dim3 grid, int threads, bool dependent) {
    if (grid.x == 0 || grid.y == 0 || grid.z == 0) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ++*kernels;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, maps, args);
  };
  auto both = [&](auto dq, uint32_t dq_smem, auto dkv, uint32_t dkv_smem) {
    const cudaError_t e = go(dq, dq_smem, dim3(hq >> args.shift, tq, seqs * args.q_parts),
                             kAttnThreads, false);
    if (e != cudaSuccess) return e;
    return go(dkv, dkv_smem, dim3(hk, tk, seqs * args.k_parts), kDkvThreads, tq > 0);
  };
  auto dims = [&](auto type) {
    constexpr bool B = decltype(type)::value;
    auto size = [&](auto entries) {
      constexpr int DP = decltype(entries)::value;
      return both(lin_attn_dq_kernel<DP, B, FORM>, DqCfg<DP>::SMEM,
                  lin_attn_dkv_kernel<DP, B, FORM>, DkvCfg<DP, FORM != kNoForm>::SMEM);
    };
    return args.s.dim <= 64   ? size(std::integral_constant<int, 64>{})
           : args.s.dim <= 96 ? size(std::integral_constant<int, 96>{})
                              : size(std::integral_constant<int, 128>{});
  };
  return bf16 ? dims(std::true_type{}) : dims(std::false_type{});
}

}  // namespace lin
