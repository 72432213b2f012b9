// lin_attn_fwd.cu -- attention forward: O = softmax(scale Q K^T) V and each
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
  static_assert(OFF_ABORT + 4 <= 1024, "barrier region");
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
template <int DP, bool BF16, int TILES, bool PACKED>
__global__ void __launch_bounds__(kFwdThreads, 1)
    lin_attn_fwd_kernel(const __grid_constant__ AttnFwdMaps maps,
                        const __grid_constant__ AttnFwdArgs args) {
  using C = FwdCfg<DP>;
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
  const int all0 = fwd_key_tiles(i0, tile_q, sq.len, sk.len, a.causal);
  const int all1 = TILES > 1 ? fwd_key_tiles(i0 + tile_q, tile_q, sq.len, sk.len, a.causal) : 0;
  const int all = max(all0, all1);
  const int j0 = at.begin(all), j1 = at.end(all);
  const int n0 = max(min(all0, j1) - j0, 0), n1 = max(min(all1, j1) - j0, 0);
  const int n = max(n0, n1);
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
    mbar_init(bar(tid), tid >= C::P_READY && tid < C::O_FULL ? 4 : 1);
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
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
        bool ok = attn_wait(bar(C::K_FULL), 0, ctl);
        for (int t = 0; t < 2 && ok; ++t) {
          if ((t ? n1 : n0) == 0) continue;
          ok = attn_wait(bar(C::Q_FULL + t), 0, ctl);
          if (ok) scores(t, 0);
        }
        if (ok) umma_commit(bar(C::K_EMPTY));
        int s = 0, s1 = 1 % C::NKV;           // stages of tiles j and j + 1
        uint32_t round = 0, round1 = C::NKV == 1;
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) ok = attn_wait(bar(C::K_FULL + s1), round1 & 1, ctl);
          if (C::AHEAD && ok && j + 1 < n0) {
            ok = attn_wait(bar(C::S_TAKEN), j & 1, ctl);
            tc_fence_after_sync();
            if (ok) scores(0, s1);
          }
          ok = ok && attn_wait(bar(C::V_FULL + s), round & 1, ctl);
          if (ok && j + 1 == n && v_left < 128) ok = attn_wait(bar(C::TAIL), 0, ctl);
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : n0;
            if (j >= nt || !ok) continue;
            if (C::AHEAD && t == 1 && j + 1 < nt) {
              ok = attn_wait(bar(C::S_TAKEN + 1), j & 1, ctl);
              tc_fence_after_sync();
              if (!ok) break;
              scores(1, s1);
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              ok = ok && attn_wait(bar(C::P_READY + 2 * t + half), j & 1, ctl);
              if (!ok || !stage_ok(a, s, C::NKV)) break;
              tc_fence_after_sync();
              umma_tokens<DP, BF16, 4>(C::O_COL + t * DP, C::p_col(t) + half * 32,
                                       v_desc + s * AttnTile<DP>::UNITS, half * 4,
                                       j == 0 && half == 0);
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
    const int t = warp >> 2, row = tid & 127;
    const int nk = t ? n1 : n0;
    const int turn = PACKED ? row / pack : row;
    const int h = PACKED ? h0 + row - turn * pack : h0;
    const int i = i0 + t * tile_q + turn;   // query of the sequence
    // (packed: the last rows of a tile may be nobody's)
    const bool live = i < sq.len && t < TILES && (!PACKED || turn < tile_q);
    const float c = a.scale * kLog2E;
    // the last key that this row may see
    const int lim = live ? (a.causal ? min(sk.len - 1, i + sk.len - sq.len) : sk.len - 1) : -1;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes per warp, lane field at bit 16
    const uint32_t s_col = tmem + lanes + C::S_COL + t * 128;
    const uint32_t p_col = tmem + lanes + C::p_col(t);
    const uint32_t o_col = tmem + lanes + C::O_COL + t * DP;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < nk; ++j) {
      ok = warp_wait_phase<kAttnNapNs>(bar(C::S_FULL + t), j & 1, ctl);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t s[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(s_col + q * 32, s[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_wait_ld_x32(s[q]);
      if constexpr (C::AHEAD) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::S_TAKEN + t));
      }
      const int lim_j = lim - (j0 + j) * 128;
      if (__any_sync(0xffffffffu, lim_j < 127)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e > lim_j) s[q][e] = 0xff800000u;   // -inf
      }
      float mx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
        for (int e = 1; e < 31; e += 2)
          mx[q] = max3(mx[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
        mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
      }
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      // (a row without a key so far has m = -inf: the difference is inf)
      const bool grow = top > m && !((top - m) * c <= 8.0f);
      if (C::AHEAD && j > 0) {   // P V of the tiles so far: O may change, and P
        ok = warp_wait_phase<kAttnNapNs>(bar(C::O_FULL + t), (j - 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after_sync();
      }
      if (__any_sync(0xffffffffu, grow)) {
        const float to = fmaxf(m, top);
        const float alpha = to > m ? ex2_approx((m - to) * c) : 1.0f;
        m = to;
        if (j > 0) {   // P V of the tiles so far is complete (not ahead: S came behind it)
          l *= alpha;
#pragma unroll
          for (int q = 0; q < DP / 32; ++q) {
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
      for (int q = 0; q < 2; ++q) {   // the product may start on the first half
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
        if (lane == 0) mbar_arrive(bar(C::P_READY + 2 * t + q));
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
    }
    if (ok && nk > 0) {
      ok = warp_wait_phase<kAttnNapNs>(bar(C::O_FULL + t), C::AHEAD ? (nk - 1) & 1 : 0, ctl);
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
      if (live && q_row_ok(a, token, h)) *lse = l == 0.0f ? -INFINITY : m * a.scale + logf(l);
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

// O and the log-sum-exps from the parts': weights 2^(L_p - L) of their rows,
// added in order. A CTA per 32 rows of a sequence and head, eight entries to
// a thread.
template <bool BF16>
__global__ void __launch_bounds__(256)
    lin_attn_join_parts_kernel(const __grid_constant__ AttnFwdArgs args) {
  const AttnArgs& a = args.s;
  const int h = blockIdx.x;
  const SeqRange r = seq_range(a.cu_q, blockIdx.z, a.tokens_q, a.max_q);
  const int groups = a.dim / 8;
  pdl_wait();
  for (int k = threadIdx.x; k < 32 * groups; k += 256) {
    const int i = blockIdx.y * 32 + k / groups, col = k % groups * 8;
    if (i >= r.len) continue;
    const int64_t token = (int64_t)r.start + i;
    const int row_at = (int)blockIdx.z * a.max_q + i;
    if (!q_row_ok(a, token, h) || !dcheck(row_at < args.part_rows, a.status, CHK_PART, row_at)) continue;
    const float* ls = args.lse_part + h * args.part_rows + row_at;
    const int ls_step = a.heads_q * args.part_rows;
    float top = -INFINITY;
    for (int q = 0; q < args.parts; ++q) top = fmaxf(top, ls[q * ls_step]);
    const float shift = top == -INFINITY ? 0.0f : top;   // (a row without a key)
    const float* p = args.o_part + (row_at * a.heads_q + h) * a.dim + col;
    const int step = ls_step * a.dim;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    float total = 0.0f;
    for (int q = 0; q < args.parts; ++q) {
      const float w = ex2_approx((ls[q * ls_step] - shift) * kLog2E);
      const float4 u = __ldcs(reinterpret_cast<const float4*>(p + q * step));
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p + q * step) + 1);
      total += w;
      x = make_float4(fmaf(w, u.x, x.x), fmaf(w, u.y, x.y), fmaf(w, u.z, x.z), fmaf(w, u.w, x.w));
      y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    store16(args.o.p + token * args.o.token_stride + (int64_t)h * args.o.head_stride + col,
            pack16<BF16>(x.x * inv, x.y * inv), pack16<BF16>(x.z * inv, x.w * inv),
            pack16<BF16>(y.x * inv, y.y * inv), pack16<BF16>(y.z * inv, y.w * inv));
    if (col == 0) args.lse[(int64_t)h * a.tokens_q + token] = top + logf(total);
  }
}

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
      return bf16 ? go(lin_attn_fwd_kernel<DP, true, 1, true>, smem)
                  : go(lin_attn_fwd_kernel<DP, false, 1, true>, smem);
    if (args.pack > 1)
      return bf16 ? go(lin_attn_fwd_kernel<DP, true, 2, true>, smem)
                  : go(lin_attn_fwd_kernel<DP, false, 2, true>, smem);
    return bf16 ? go(lin_attn_fwd_kernel<DP, true, 2, false>, smem)
                : go(lin_attn_fwd_kernel<DP, false, 2, false>, smem);
  };
  // (heads of 65 to 96 entries: a quarter less of both products than 128; 4096
  // causal tokens, 16 heads of 96: 52.2 -> 49.1 us)
  const cudaError_t e = args.s.dim <= 64   ? types(std::integral_constant<int, 64>{})
                        : args.s.dim <= 96 ? types(std::integral_constant<int, 96>{})
                                           : types(std::integral_constant<int, 128>{});
  if (e != cudaSuccess || args.parts == 1) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(heads, (unsigned)((args.s.max_q + 31) / 32), (unsigned)sequences);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, lin_attn_join_parts_kernel<true>, args)
              : cudaLaunchKernelEx(&cfg, lin_attn_join_parts_kernel<false>, args);
}

}  // namespace lin
