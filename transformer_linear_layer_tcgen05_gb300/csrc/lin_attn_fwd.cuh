// lin_attn_fwd.cuh -- attention forward: O = softmax(scale Q K^T) V and each
// row's log-sum-exp.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// for each tile of 128 keys S = Q K^T goes to tensor memory, the row's thread
// takes p = 2^(c s - c m) (c = scale log2 e), writes it back as 16-bit P over
// S, and O += P V accumulates in tensor memory. When a row's maximum grows by
// more than 8 in base-2 units the row's l and O are scaled down to the new
// one; below that the old maximum stays in place (p then reaches 2^8, well
// inside both 16-bit types' range) and O is left alone: the quotient O / l
// does not depend on it.
//
// A CTA runs two tiles of 128 queries of one head (one, where even so every
// CTA has an SM to itself) against the same keys: 128 threads per tile (one
// per row) take turns on the exponentials while the tensor cores work for the
// other tile, and each K, V tile is read once for 256 queries. The products
// of one thread execute in issue order, so S of the next tile is issued right
// behind the P V that reads P out of the same columns; heads of up to 64
// leave columns for P of its own, and S of the next tile then comes ahead of
// it (8192 tokens, 16 heads: 148 -> 139 us; both tiles' S ahead of either P V
// brings their exponentials into step: 146). Heads vary fastest over the grid
// and the causal mask's longest query tiles come first. Where there are fewer
// CTAs than SMs the keys are cut into parts, a CTA each, whose results a
// second kernel joins by their log-sum-exps.
//
// What bounds it. 8192 causal tokens, 32 heads of 128: 329-333 us, 1650-1670
// TF/s, 0.85-0.86 of the cuBLAS burst rate, with the clock pulled down to
// 1.75-1.87 GHz by the power limit: instructions cost time there even where
// no unit is full. 2^x by a polynomial in place of every eighth to second one
// of the special-function unit's: 360-406 us; two threads a row: 388; a
// thread of its own for each tile's products: 377 (the two tiles' products
// then alternate, and each waits for both). Heads of 64, 8192 tokens: 138 us,
// 0.51 of that rate: the rows' own work (about 1100 cycles a tile of each
// warp, half of it the 128 exponentials) comes to twice the products'; what
// the power limit rules out at 128 was not measured there. Short calls: 512
// tokens, 12 heads 8.3-8.5 us of which four tiles' turns are some 5, in which one
// warpgroup takes all exponentials of a row while the other has no rows.
//
// P is rounded to the tensors' 16 bits for its product: the tensor cores take both
// operands in one type, and P in two parts would be the product twice. It costs
// O less than its own rounding does (512 tokens, binary16: 2.4e-4 off instead of
// the 2.1e-4 of an f32 P; 8192, bfloat16: 2.1e-3 instead of 1.7e-3).
//
// SCORES: the row's thread turns its scores into z = cap tanh(scale s / cap) -
// slope |distance| (in base-2 units) before the maximum, and masks by its own
// range of keys; the CTA runs over the key tiles from the first to the last that
// its rows' ranges meet. 8192 causal tokens, 32 heads over 8 of 128: cap 50 462 us,
// bias 415, both 584; documents 126, with the cap 167; a window of 1024 keys 140
// and 176. The row's own work bounds these: no unit is full, and a tile's way from
// S to P is longer than the products behind it.
#pragma once

#include "lin_attn.cuh"

#include <type_traits>

namespace lin {

namespace {

// Three warpgroups: the two tiles' rows, and the copying and issuing warps
// (two of the third's stay idle: registers are handed over by whole
// warpgroups). A thread that holds a row of S wants more than the 168
// registers of an even share; without the hand-over the loop spilled and the
// 8192-token case took 578 us instead of 348.
constexpr int kFwdThreads = 384;
constexpr int kFwdRegsRow = 208, kFwdRegsIssue = 88;
static_assert(2 * kFwdRegsRow + kFwdRegsIssue <= 3 * 168, "registers of the launch");
template <int DP>
struct FwdCfg {
  static constexpr int NKV = DP <= 64 ? 3 : 2;   // stages of the K and of the V ring
  static constexpr uint32_t TILE = AttnTile<DP>::BYTES;
  // barrier slots
  static constexpr int Q_FULL = 0;               // 2
  static constexpr int K_FULL = 2;
  static constexpr int K_EMPTY = K_FULL + NKV;
  static constexpr int V_FULL = K_EMPTY + NKV;
  static constexpr int V_EMPTY = V_FULL + NKV;
  static constexpr int S_FULL = V_EMPTY + NKV;   // 2
  static constexpr int P_READY = S_FULL + 2;     // 2 x 2: first and second half of the keys
  static constexpr int S_TAKEN = P_READY + 4;    // 2
  static constexpr int O_FULL = S_TAKEN + 2;     // 2
  static constexpr int TAIL = O_FULL + 2;        // the last V tile is cut at the sequence's end
  static constexpr int DRAIN = TAIL + 1;         // every product of the CTA is done
  static constexpr int BARS = DRAIN + 1;
  static constexpr uint32_t OFF_TMEM = BARS * 8, OFF_ABORT = OFF_TMEM + 4;
  static constexpr uint32_t OFF_EXTENTS = 512;   // 16 ints: the warps' keys
  static constexpr uint32_t OFF_MEET = 640;      // a barrier: two threads to a row
  static_assert(OFF_ABORT + 4 <= OFF_EXTENTS, "barrier region");
  static constexpr uint32_t OFF_Q = 1024;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NKV * TILE;
  static constexpr uint32_t SMEM = OFF_V + NKV * TILE + 1024;   // + alignment of the base
  static_assert(SMEM <= 232448, "shared memory");
  // P has columns of its own where the 512 hold them, and S of the next tile
  // is then computed while the rows work on this one's
  static constexpr bool AHEAD = DP == 64;
  // tensor memory columns: S (and P over it) of the two tiles, O, P
  static constexpr uint32_t S_COL = 0, O_COL = 256;
  static constexpr uint32_t p_col(int t) { return AHEAD ? 384 + t * 64 : S_COL + t * 128; }
  static_assert(O_COL >= S_COL + 256 && O_COL + 2 * DP <= (AHEAD ? 384u : 512u), "tensor memory");
};

// Key tiles that the queries [i0, i0 + n) of a sequence need.
__device__ __forceinline__ int fwd_key_tiles(int i0, int n, int lq, int lk, int causal) {
  if (i0 >= lq) return 0;
  const int last = min(i0 + n, lq) - 1;
  const int hi = causal ? min(lk, last + lk - lq + 1) : lk;
  return hi > 0 ? (hi + 127) / 128 : 0;
}

}  // namespace

// TILES of 128 rows to a CTA. PACKED: a row is query i of one of the `pack`
// query heads that share a key head, tile_q queries of them all to a tile.
// (These are the compiler's parameters: read from the arguments, the rows of
// a CTA cost the longest problems 2 %, 347 -> 353 us.)
template <int DP, bool BF16, int TILES, bool PACKED, int FORM>
__global__ void __launch_bounds__(kFwdThreads, 1)
    lin_attn_fwd_kernel(const __grid_constant__ AttnFwdMaps maps,
                        const __grid_constant__ AttnFwdArgs args) {
  using C = FwdCfg<DP>;
  constexpr bool SCORES = FORM != kNoForm;
  constexpr bool CAPPED = SCORES && (FORM & kCap), BIASED = SCORES && (FORM & kBias);
  // Two threads to a row, one of each warpgroup, where the second one has no
  // tile: each turns half of the scores, and they meet for the maximum. (Ranges
  // alone have the sums, bit by bit, of the causal mask that they may be.)
  constexpr bool SPLIT = TILES == 1 && (CAPPED || BIASED);
  constexpr int NQ = SPLIT ? 2 : 4;   // groups of 32 columns of a thread
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = args.s;
  const int pack = PACKED ? args.pack : 1, tile_q = PACKED ? args.tile_q : 128;
  const int h0 = (int)blockIdx.x * pack;   // the first head of the CTA
  // Parts only where every CTA has an SM to itself: one tile to each. (The rows
  // ask for parts in either form: compiled without it the one of two tiles takes
  // 140.9 us instead of 137.8 at 8192 tokens, 16 heads of 64.)
  const int parts = args.parts;
  const PartOf at = part_of(blockIdx.z, TILES == 1 ? parts : 1);
  const int b = at.b;
  // longest rows of a causal mask first
  const int i0 = (int)(gridDim.y - 1 - blockIdx.y) * (TILES * tile_q);
  const SeqRange sq = seq_range(a.cu_q, b, a.tokens_q, a.max_q);
  if (i0 >= sq.len) return;   // (the whole CTA)
  const SeqRange sk = seq_range(a.cu_k, b, a.tokens_k, a.max_k);
  // key tiles of the two query tiles, and of them those of this part, from j0 on
  // (b0, b1: those of them before a tile's own first, a form's ranges)
  int all0 = 0, all1 = 0, from = 0, j0, n0, n1, n, b0 = 0, b1 = 0;
  auto share = [&] {
    const int all = max(max(all0, all1) - from, 0);
    j0 = from + at.begin(all);
    const int j1 = from + at.end(all);
    n0 = max(min(all0, j1) - j0, 0);
    n1 = max(min(all1, j1) - j0, 0);
    n = max(n0, n1);
  };
  if constexpr (!SCORES) {
    all0 = fwd_key_tiles(i0, tile_q, sq.len, sk.len, a.causal);
    all1 = TILES > 1 ? fwd_key_tiles(i0 + tile_q, tile_q, sq.len, sk.len, a.causal) : 0;
    share();
  }
  const int hk = h0 / a.group;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gen = smem_raw + (base - smem_u32(smem_raw));
  auto bar = [&](int slot) { return base + (uint32_t)slot * 8u; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = reinterpret_cast<volatile int*>(gen + C::OFF_ABORT);
  const WaitCtl ctl{a.timeout_ns, abort, a.status};

  if (warp == kAttnMmaWarp) {
    tmem_alloc(base + C::OFF_TMEM, 512);
    tmem_relinquish_alloc_permit();
  }
  if (tid == 0) *abort = 0;
  if (tid < C::BARS) {
    mbar_init(bar(tid), SPLIT && tid == C::S_TAKEN              ? 8
                        : tid >= C::P_READY && tid < C::O_FULL ? 4
                                                               : 1);
    if (SPLIT && tid == 0) mbar_init(base + C::OFF_MEET, 8);
    fence_barrier_init();
  }
  // the keys of this thread's row, and of each warp's rows
  KeyRange mine{0, 0};
  int* const extents = reinterpret_cast<int*>(gen + C::OFF_EXTENTS);
  if constexpr (SCORES) {
    if (warp < 8) {
      const int turn = PACKED ? (tid & 127) / pack : tid & 127;
      const int i = i0 + (SPLIT ? 0 : (warp >> 2) * tile_q) + turn;
      if (i < sq.len && (warp < 4 || TILES > 1 || SPLIT) && (!PACKED || turn < tile_q) &&
          q_row_ok(a, sq.start + i, h0))
        mine = key_range(args.scores, a.causal, sq, sk, i);
      const KeyRange all = warp_extent(mine);
      if (lane == 0) {
        extents[2 * warp] = all.lo;
        extents[2 * warp + 1] = all.hi;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if constexpr (SCORES) {
    const KeyRange t0 = join_extents(extents, 4);
    const KeyRange t1 = TILES > 1 ? join_extents(extents + 8, 4) : KeyRange{INT_MAX, 0};
    from = min(t0.lo, t1.lo) / 128;   // (INT_MAX without a key: there are no tiles then)
    all0 = (t0.hi + 127) / 128;
    all1 = (t1.hi + 127) / 128;
    share();
    b0 = max(t0.lo / 128 - j0, 0);
    b1 = max(t1.lo / 128 - j0, 0);
    if (b0 >= n0) n0 = b0 = 0;   // (none in this part)
    if (b1 >= n1) n1 = b1 = 0;
  }
  // (an allocation of all 512 columns begins at column 0)
  constexpr uint32_t tmem = 0;

  const int v_left = sk.len - (j0 + n - 1) * 128;   // keys of the last tile (128 or more: all)
  if (warp >= 8) {
    setmaxnreg_dec<kFwdRegsIssue>();
    if (warp == kAttnCopyWarp) {
      if (lane == 0 && n > 0) {
        const int z = sq.start + i0;
        const uint32_t q_bytes = PACKED ? AttnTile<DP>::SUB * (uint32_t)(pack * tile_q) * 128u : C::TILE;
        int k_issued = 0, v_issued = 0;
        bool second = false;
        if (n0 > 0) {   // (the first rows of a causal mask may see no key at all)
          mbar_arrive_expect_tx(bar(C::Q_FULL), q_bytes);
          if (dcheck(q_bytes <= C::TILE, a.status, CHK_BUFFER, q_bytes) && q_row_ok(a, z, h0 + pack - 1))
            load_tile<DP, 128>(base + C::OFF_Q, &maps.q, h0, z, bar(C::Q_FULL));
        }
        for (int j = 0; j < n; ++j) {
          const int s = j % C::NKV, round = j / C::NKV;
          if (round > 0 && !attn_wait(bar(C::K_EMPTY + s), (round - 1) & 1, ctl)) break;
          mbar_arrive_expect_tx(bar(C::K_FULL + s), C::TILE);
          if (stage_ok(a, s, C::NKV) && k_row_ok(a, sk.start + (j0 + j) * 128, hk))
            load_tile<DP, 128>(base + C::OFF_K + s * C::TILE, &maps.k, hk,
                               sk.start + (j0 + j) * 128, bar(C::K_FULL + s));
          ++k_issued;
          if (j == 0 && n1 > 0) {
            mbar_arrive_expect_tx(bar(C::Q_FULL + 1), q_bytes);
            if (q_row_ok(a, z + tile_q, h0 + pack - 1))
              load_tile<DP, 128>(base + C::OFF_Q + C::TILE, &maps.q, h0, z + tile_q, bar(C::Q_FULL + 1));
            second = true;
          }
          if (round > 0 && !attn_wait(bar(C::V_EMPTY + s), (round - 1) & 1, ctl)) break;
          mbar_arrive_expect_tx(bar(C::V_FULL + s), C::TILE);
          if (stage_ok(a, s, C::NKV))
            load_tile<DP, 128>(base + C::OFF_V + s * C::TILE, &maps.v, hk,
                               sk.start + (j0 + j) * 128, bar(C::V_FULL + s));
          ++v_issued;
        }
        // no copy may still be in flight when the CTA ends (after a wait that
        // ran out; otherwise all of these have completed)
        if (*abort) {
          if (n0 > 0) attn_wait(bar(C::Q_FULL), 0, ctl, false);
          if (second) attn_wait(bar(C::Q_FULL + 1), 0, ctl, false);
          for (int j = max(0, k_issued - C::NKV); j < k_issued; ++j)
            attn_wait(bar(C::K_FULL + j % C::NKV), (j / C::NKV) & 1, ctl, false);
          for (int j = max(0, v_issued - C::NKV); j < v_issued; ++j)
            attn_wait(bar(C::V_FULL + j % C::NKV), (j / C::NKV) & 1, ctl, false);
        }
      }
      __syncwarp();
      if (n > 0 && v_left < 128) {   // cut the last V tile at the sequence's end
        const int s = (n - 1) % C::NKV;
        if (warp_wait_phase<kAttnNapNs>(bar(C::V_FULL + s), ((n - 1) / C::NKV) & 1, ctl)) {
          if (dcheck(v_left > 0, a.status, CHK_BUFFER, v_left))
            zero_rows<DP, 128>(base + C::OFF_V + s * C::TILE, v_left, 128, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::TAIL));
        }
      }
    } else if (warp == kAttnMmaWarp) {
      if (n > 0 && elect_one()) {   // one thread issues every product
        const uint64_t q_desc = AttnTile<DP>::k_major(base + C::OFF_Q);
        const uint64_t k_desc = AttnTile<DP>::k_major(base + C::OFF_K);
        const uint64_t v_desc = AttnTile<DP>::mn_major(base + C::OFF_V);
        auto scores = [&](int t, int s) {   // S_t = Q_t K^T, K in stage s
          if (!stage_ok(a, s, C::NKV)) return;
          umma_entries<DP, BF16>(C::S_COL + t * 128, q_desc + t * AttnTile<DP>::UNITS,
                                 k_desc + s * AttnTile<DP>::UNITS);
          umma_commit(bar(C::S_FULL + t));
        };
        // A tile's first scores: its queries' copy is waited for here, once for
        // each tile that has keys, wherever among the key tiles it begins (copies
        // complete in no order, so no other wait stands for this one).
        auto first_scores = [&](int t, int s) -> bool {
          if (!attn_wait(bar(C::Q_FULL + t), 0, ctl)) return false;
          scores(t, s);
          return true;
        };
        bool ok = attn_wait(bar(C::K_FULL), 0, ctl);
        for (int t = 0; t < 2 && ok; ++t)
          if ((t ? n1 : n0) > 0 && (t ? b1 : b0) == 0) ok = first_scores(t, 0);
        if (ok) umma_commit(bar(C::K_EMPTY));
        int s = 0, s1 = 1 % C::NKV;           // stages of tiles j and j + 1
        uint32_t round = 0, round1 = C::NKV == 1;
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) ok = attn_wait(bar(C::K_FULL + s1), round1 & 1, ctl);
          if (C::AHEAD && ok && j + 1 < n0 && j + 1 >= b0) {
            if (j < b0) {
              ok = first_scores(0, s1);
            } else {
              ok = attn_wait(bar(C::S_TAKEN), (j - b0) & 1, ctl);
              tc_fence_after_sync();
              if (ok) scores(0, s1);
            }
          }
          ok = ok && attn_wait(bar(C::V_FULL + s), round & 1, ctl);
          if (ok && j + 1 == n && v_left < 128) ok = attn_wait(bar(C::TAIL), 0, ctl);
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : n0, bt = t ? b1 : b0;
            if (j >= nt || !ok) continue;
            if (j < bt) {   // (its first scores; ahead, the first tile's are out already)
              if (j + 1 == bt && (!C::AHEAD || t == 1)) ok = first_scores(t, s1);
              continue;
            }
            if (C::AHEAD && t == 1 && j + 1 < nt) {
              ok = attn_wait(bar(C::S_TAKEN + 1), (j - bt) & 1, ctl);
              tc_fence_after_sync();
              if (!ok) break;
              scores(1, s1);
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              ok = ok && attn_wait(bar(C::P_READY + 2 * t + half), (j - bt) & 1, ctl);
              // (split: both threads of a row may have scaled their half of O)
              if (SPLIT && half == 0) ok = ok && attn_wait(bar(C::P_READY + 1), (j - bt) & 1, ctl);
              if (!ok || !stage_ok(a, s, C::NKV)) break;
              tc_fence_after_sync();
              umma_tokens<DP, BF16, 4>(C::O_COL + t * DP, C::p_col(t) + half * 32,
                                       v_desc + s * AttnTile<DP>::UNITS, half * 4,
                                       j == bt && half == 0);
            }
            if (!ok) break;
            if (!C::AHEAD && j + 1 < nt)
              scores(t, s1);
            else   // (ahead: for every tile)
              umma_commit(bar(C::O_FULL + t));
          }
          if (!ok) break;
          umma_commit(bar(C::V_EMPTY + s));
          if (j + 1 < n) umma_commit(bar(C::K_EMPTY + s1));
          s = s1;
          round = round1;
          if (++s1 == C::NKV) {
            s1 = 0;
            ++round1;
          }
        }
        // tensor memory stays allocated until every issued product has finished
        umma_commit(bar(C::DRAIN));
        attn_wait(bar(C::DRAIN), 0, ctl, false);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kFwdRegsRow>();
    const int t = SPLIT ? 0 : warp >> 2, row = tid & 127;
    const int half = SPLIT ? warp >> 2 : 0, col0 = half * 64;   // (split) the thread's columns
    const int nk = t ? n1 : n0, bt = t ? b1 : b0;
    const int turn = PACKED ? row / pack : row;
    const int h = PACKED ? h0 + row - turn * pack : h0;
    const int i = i0 + t * tile_q + turn;   // query of the sequence
    // (packed: the last rows of a tile may be nobody's)
    const bool live = i < sq.len && t < TILES && (!PACKED || turn < tile_q);
    const ScoreTurn turned(args.scores, a.scale);
    // the factor to base-2 units (capped scores are in them already), and the
    // bias of a key's distance, before that factor
    const float c = CAPPED ? 1.0f : a.scale * kLog2E;
    const float slope = BIASED && live ? args.scores.slopes[h] * kLog2E / c : 0.0f;
    // the last key that this row may see, and the first
    const int lim = SCORES ? mine.hi - 1
                    : live ? (a.causal ? min(sk.len - 1, i + sk.len - sq.len) : sk.len - 1)
                           : -1;
    const int low = SCORES ? mine.lo : 0;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes per warp, lane field at bit 16
    const uint32_t s_col = tmem + lanes + C::S_COL + t * 128 + col0;
    const uint32_t p_col = tmem + lanes + C::p_col(t) + half * 32;
    const uint32_t o_col = tmem + lanes + C::O_COL + t * DP;
    // (A row that sees no key at all, which with ranges keeps its scores, has a
    // maximum that nothing exceeds: it never asks for a new one. What is in its
    // place may be nobody's, and whatever was in memory.)
    float m = SCORES && lim < 0 ? INFINITY : -INFINITY, l = 0.0f;
    bool ok = true;
    // (split) what the row's two threads tell each other, in two places in turn
    // (the second tile's queries have none here)
    volatile float* const told = reinterpret_cast<volatile float*>(gen + C::OFF_Q + C::TILE);
    auto meet = [&](int at, float mine_is, float* other) -> bool {
      volatile float* to = told + (at & 1) * 256;
      to[half * 128 + row] = mine_is;
      tc_fence_before_sync();   // (either's P may come over what the other has read of S)
      __syncwarp();
      if (lane == 0) mbar_arrive(base + C::OFF_MEET);
      if (!warp_wait_phase<kAttnNapNs>(base + C::OFF_MEET, at & 1, ctl)) return false;
      tc_fence_after_sync();
      *other = to[(half ^ 1) * 128 + row];
      return true;
    };
    for (int j = bt; j < nk; ++j) {
      ok = warp_wait_phase<kAttnNapNs>(bar(C::S_FULL + t), (j - bt) & 1, ctl);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t s[NQ][32];
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_ld_32x32b_x32(s_col + q * 32, s[q]);
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_wait_ld_x32(s[q]);
      if constexpr (C::AHEAD) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::S_TAKEN + t));
      }
      const int lim_j = lim - (j0 + j) * 128 - col0;
      if constexpr (SCORES) {
        // (a row without a key cuts no tile: its sums are dropped at the end)
        const int low_j = low - (j0 + j) * 128 - col0;
        const bool cut_end = __any_sync(0xffffffffu, lim >= 0 && lim_j < NQ * 32 - 1);
        const bool cut_first = __any_sync(0xffffffffu, lim >= 0 && low_j > 0);
        auto leave_out = [&](int q, uint32_t value) {   // of 32 keys
          if (!__any_sync(0xffffffffu, lim >= 0 && (lim_j < q * 32 + 31 || low_j > q * 32))) return;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e > lim_j || q * 32 + e < low_j) s[q][e] = value;
        };
        if constexpr (CAPPED) {
          // Where the mask cuts the tile, by groups of 32 keys: those that no row of
          // the warp sees are left as they are, and hidden ones of the others
          // zeroed. The way goes by the row's own largest score of the group or the
          // tile: a row's results do not go by what other rows hold, nor by what the
          // mask hides. (NaN is passed over: each way gives NaN.)
          auto two = [&](int q, int e) -> float2 {
            return make_float2(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
          };
          auto put = [&](int q, int e, float2 y) {
            s[q][e] = __float_as_uint(y.x);
            s[q][e + 1] = __float_as_uint(y.y);
          };
          auto by_rest = [&](int q) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              turned.rest4(&s[q][e]);
              put(q, e, turned.score(two(q, e)));
              put(q, e + 2, turned.score(two(q, e + 2)));
            }
          };
          auto cap = [&](auto first_group, auto groups) {
            constexpr int Q0 = decltype(first_group)::value, Q1 = Q0 + decltype(groups)::value;
            float big[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = Q0; q < Q1; ++q)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float& b = big[e / 2 & 3];
                b = max3(b, fabsf(__uint_as_float(s[q][e])), fabsf(__uint_as_float(s[q][e + 1])));
              }
            big[0] = max3(fmaxf(big[0], big[1]), big[2], big[3]);
            auto by_terms = [&](const auto& terms) {
#pragma unroll
              for (int q = Q0; q < Q1; ++q)
#pragma unroll
                for (int e = 0; e < 32; e += 2) put(q, e, ScoreTurn::by_terms(terms, two(q, e)));
            };
            if (big[0] <= args.scores.few_up_to) {
              by_terms(args.scores.few);
            } else if (big[0] <= args.scores.up_to) {
              by_terms(args.scores.terms);
            } else {
#pragma unroll
              for (int q = Q0; q < Q1; ++q) by_rest(q);
            }
            __syncwarp();
          };
          auto group = [&](auto q) {
            constexpr int Q = decltype(q)::value;
            if (!__any_sync(0xffffffffu, lim_j >= Q * 32 && low_j <= Q * 32 + 31)) return;
            leave_out(Q, 0u);
            cap(q, std::integral_constant<int, 1>{});
          };
          if constexpr (SPLIT) {   // (short calls: little code rather than few instructions)
            if (cut_end || cut_first) {
#pragma unroll
              for (int q = 0; q < NQ; ++q) leave_out(q, 0u);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) by_rest(q);
          } else if (cut_end || cut_first) {
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            group(std::integral_constant<int, 3>{});
          } else {
            cap(std::integral_constant<int, 0>{}, std::integral_constant<int, 4>{});
          }
        }
        if constexpr (BIASED) {   // (in the scores' own units: c comes later)
          const float here = (float)(i + sk.len - sq.len - (j0 + j) * 128 - col0);
          const float2 sl = make_float2(-slope, -slope);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            float2 far = make_float2(here - (float)(q * 32), here - (float)(q * 32 + 1));
            if (a.causal) {   // what is not hidden lies behind the query: no sign to drop
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 x = fma2(far, sl, make_float2(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])));
                s[q][e] = __float_as_uint(x.x);
                s[q][e + 1] = __float_as_uint(x.y);
                far = add2(far, make_float2(-2.0f, -2.0f));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                s[q][e] = __float_as_uint(fmaf(-slope, fabsf(far.x), __uint_as_float(s[q][e])));
                s[q][e + 1] = __float_as_uint(fmaf(-slope, fabsf(far.y), __uint_as_float(s[q][e + 1])));
                far = add2(far, make_float2(-2.0f, -2.0f));
              }
            }
          }
        }
        if (cut_end || cut_first) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) leave_out(q, 0xff800000u);   // -inf
        }
      } else if (__any_sync(0xffffffffu, lim_j < 127)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e > lim_j) s[q][e] = 0xff800000u;   // -inf
      }
      float mx[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
        for (int e = 1; e < 31; e += 2)
          mx[q] = max3(mx[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
        mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
      }
      float top = SPLIT ? fmaxf(mx[0], mx[1]) : fmaxf(max3(mx[0], mx[1], mx[NQ - 2]), mx[NQ - 1]);
      if constexpr (SPLIT) {
        float other;
        ok = meet(j - bt, top, &other);
        if (!ok) break;
        top = fmaxf(top, other);
      }
      // (a row without a key so far has m = -inf: the difference is inf)
      const bool grow = top > m && !((top - m) * c <= 8.0f);
      if (C::AHEAD && j > bt) {   // P V of the tiles so far: O may change, and P
        ok = warp_wait_phase<kAttnNapNs>(bar(C::O_FULL + t), (j - bt - 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after_sync();
      }
      if (__any_sync(0xffffffffu, grow)) {
        // (Capped and biased scores: only rows that ask for it take it, so that a
        // row's results do not go by what other rows of its warp hold. More warps
        // then have a row that asks: bias 408 -> 415 us at 8192 tokens, cap 460 ->
        // 462. Ranges alone have the sums, bit by bit, of the mask that they may be.)
        const float to = CAPPED || BIASED ? (grow ? top : m) : fmaxf(m, top);
        const float alpha = (CAPPED || BIASED ? grow : to > m) ? ex2_approx((m - to) * c) : 1.0f;
        m = to;
        if (j > bt) {   // P V of the tiles so far is complete (not ahead: S came behind it)
          l *= alpha;
#pragma unroll
          for (int q = 0; q < DP / 32; ++q) {
            if (SPLIT && (q & 1) != half) continue;
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_col + q * 32, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x32(o_col + q * 32, o);
          }
        }
      }
      const float shift = m == -INFINITY ? 0.0f : -m * c;
      const float2 cc = make_float2(c, c), sh = make_float2(shift, shift);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int q = 0; q < NQ / 2; ++q) {   // the product may start on the first half
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int k = q * 64 + 2 * e;
          float2 x = make_float2(__uint_as_float(s[k >> 5][k & 31]),
                                 __uint_as_float(s[k >> 5][(k & 31) + 1]));
          x = fma2(x, cc, sh);
          x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          sum[e & 1] = add2(sum[e & 1], x);
          p[e] = pack16<BF16>(x.x, x.y);
        }
        tmem_st_32x32b_x32(p_col + q * 32, p);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::P_READY + 2 * t + (SPLIT ? half : q)));
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
    }
    if constexpr (SPLIT) {
      float other = 0.0f;
      ok = ok && meet(nk - bt, l, &other);
      l = half ? other + l : l + other;   // (both threads the same sum)
    }
    if (SCORES && lim < 0) l = 0.0f;   // (a row without a key, whatever it has summed)
    if (ok && nk > 0) {
      ok = warp_wait_phase<kAttnNapNs>(bar(C::O_FULL + t), C::AHEAD ? (nk - bt - 1) & 1 : 0, ctl);
      tc_fence_after_sync();
    }
    if (ok) {
      // a row without a key: O = 0 and a log-sum-exp of -inf
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // (NaN stays NaN)
      const int64_t token = sq.start + i;
      uint16_t* out = args.o.p + token * args.o.token_stride + (int64_t)h * args.o.head_stride;
      // among the parts' rows (unsigned: without parts it may wrap, unused)
      const uint32_t row_at = (uint32_t)b * a.max_q + i;
      float* part_row = args.o_part + ((at.part * args.part_rows + row_at) * a.heads_q + h) * a.dim;
      float* lse = parts > 1
                       ? args.lse_part + (at.part * a.heads_q + h) * args.part_rows + row_at
                       : args.lse + (int64_t)h * a.tokens_q + token;
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        if (SPLIT && (q & 1) != half) continue;
        uint32_t o[32];
        if (nk > 0) {   // (uniform over the warp)
          tmem_ld_32x32b_x32(o_col + q * 32, o);
          tmem_wait_ld_x32(o);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int col = q * 32 + g * 8;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(o[g * 8 + 2 * e]), y = __uint_as_float(o[g * 8 + 2 * e + 1]);
            w[e] = nk > 0 ? pack16<BF16>(l == 0.0f ? 0.0f : x * inv, l == 0.0f ? 0.0f : y * inv) : 0u;
          }
          if (!live || col >= a.dim || !q_row_ok(a, token, h)) continue;
          if (parts > 1 && !dcheck(row_at < (uint32_t)args.part_rows && at.part < parts, a.status,
                                    CHK_PART, row_at))
            continue;
          if (parts > 1) {   // in f32
            const float z = nk > 0 ? inv : 0.0f;
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
            if (l != 0.0f && nk > 0) {
              u = make_float4(__uint_as_float(o[g * 8]) * z, __uint_as_float(o[g * 8 + 1]) * z,
                              __uint_as_float(o[g * 8 + 2]) * z, __uint_as_float(o[g * 8 + 3]) * z);
              v = make_float4(__uint_as_float(o[g * 8 + 4]) * z, __uint_as_float(o[g * 8 + 5]) * z,
                              __uint_as_float(o[g * 8 + 6]) * z, __uint_as_float(o[g * 8 + 7]) * z);
            }
            float4* to = reinterpret_cast<float4*>(part_row + col);
            to[0] = u;
            to[1] = v;
          } else {
            store16(out + col, w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && half == 0 && q_row_ok(a, token, h))
        *lse = l == 0.0f ? -INFINITY : m * (CAPPED ? kLn2 : a.scale) + logf(l);
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

// The kernel of the arguments' head size, tiles and type.
template <int FORM>
cudaError_t launch_attn_fwd(bool bf16, const AttnFwdMaps& maps, const AttnFwdArgs& args,
                            int heads_kv, int sequences, cudaStream_t stream) {
  const unsigned heads = (unsigned)(heads_kv * args.s.group);
  const int rows = args.tiles * args.tile_q;
  const dim3 grid(heads / (unsigned)args.pack, (unsigned)((args.s.max_q + rows - 1) / rows),
                  (unsigned)sequences * (unsigned)args.parts);
  auto go = [&](auto kernel, uint32_t smem) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kFwdThreads, smem, stream>>>(maps, args);
    return cudaGetLastError();
  };
  auto types = [&](auto size) {
    constexpr int DP = decltype(size)::value;
    constexpr uint32_t smem = FwdCfg<DP>::SMEM;
    if (args.tiles == 1)
      return bf16 ? go(lin_attn_fwd_kernel<DP, true, 1, true, FORM>, smem)
                  : go(lin_attn_fwd_kernel<DP, false, 1, true, FORM>, smem);
    if (args.pack > 1 || FORM != kNoForm)
      return bf16 ? go(lin_attn_fwd_kernel<DP, true, 2, true, FORM>, smem)
                  : go(lin_attn_fwd_kernel<DP, false, 2, true, FORM>, smem);
    if constexpr (FORM == kNoForm)   // (a form's rows are dealt out at run time)
      return bf16 ? go(lin_attn_fwd_kernel<DP, true, 2, false, FORM>, smem)
                  : go(lin_attn_fwd_kernel<DP, false, 2, false, FORM>, smem);
    return cudaErrorInvalidValue;
  };
  // (heads of 65 to 96 entries: a quarter less of both products than 128; 4096
  // causal tokens, 16 heads of 96: 52.2 -> 49.1 us)
  return args.s.dim <= 64   ? types(std::integral_constant<int, 64>{})
         : args.s.dim <= 96 ? types(std::integral_constant<int, 96>{})
                            : types(std::integral_constant<int, 128>{});
}

}  // namespace lin
