// lin_attn_bwd.cu -- attention backward from Q, K, V, O, each row's
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
// norm that a key tile meets for dK).
//
// Eight warps do the element-wise part, two threads to a row, each half of
// the tile's columns. The products are issued so that the tensor cores have
// one while each element-wise phase runs: S of the next tile behind the use
// of this tile's P (or its reading, in the dQ kernel), dP of the next behind
// the use of this tile's dS.
#include "lin_attn.cuh"

namespace lin {

namespace {

constexpr float kPShift = 8.0f;     // P^T is scaled by 2^8
constexpr int kNormExp = 4;         // dO rows count as having a norm near 2^4
constexpr int kDkvThreads = kAttnThreads + 32;
constexpr int kTailWarp = 10;       // of the dK, dV kernel: cuts tiles at the sequence's end

// The streamed operands are two rings: A (K in the dQ kernel, Q in the other),
// whose tile enters the first and the last product of its turn, and B (V, dO).
// A's next tile is wanted early in a turn and its last one is still in use
// then, so with heads of 128, where shared memory holds five tiles beside the
// CTA's own two, A has three of them.
template <int DP>
struct BwdCfg {
  static constexpr int NA = DP == 64 ? 4 : 3, NB = DP == 64 ? 4 : 2;
  static constexpr uint32_t TILE = AttnTile<DP>::BYTES;
  static constexpr int OWN_FULL = 0;             // the CTA's own two tiles
  static constexpr int A_FULL = 1, A_EMPTY = A_FULL + NA;
  static constexpr int B_FULL = A_EMPTY + NA, B_EMPTY = B_FULL + NB;
  static constexpr int S_FULL = B_EMPTY + NB;    // S complete
  static constexpr int DP_FULL = S_FULL + 1;     // dP complete
  static constexpr int S_DONE = DP_FULL + 1;     // 2 halves: S read (dQ) / P^T written (dK, dV)
  static constexpr int DS_READY = S_DONE + 2;    // 2 halves: dS written
  static constexpr int A_TAIL = DS_READY + 2;    // the stage, cut at the sequence's end
  static constexpr int B_TAIL = A_TAIL + NA;
  static constexpr int OUT_FULL = B_TAIL + NB;   // the sums complete (every product is)
  static constexpr int BARS = OUT_FULL + 1;
  static constexpr bool by_half(int i) { return i >= S_DONE && i < A_TAIL; }
  static constexpr uint32_t OFF_TMEM = BARS * 8, OFF_ABORT = OFF_TMEM + 4;
  static constexpr uint32_t OFF_RED = 448;       // 16 floats
  static_assert(OFF_ABORT + 4 <= OFF_RED, "barrier region");
  static constexpr uint32_t OFF_OWN = 0;         // (tiles first: they want 1024-byte bases)
  static constexpr uint32_t OFF_A = 2 * TILE, OFF_B = OFF_A + NA * TILE;
  // [NA][128] floats: -L log2 e + 8; then [NB][128]: -a delta
  static constexpr uint32_t OFF_ROWS = OFF_B + NB * TILE;
  static constexpr uint32_t OFF_CTL = OFF_ROWS + (NA + NB) * 512;
  static constexpr uint32_t SMEM = OFF_CTL + 512;
  static_assert((NA + NB) * 512 >= 2048, "the dQ kernel's row sums");
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr uint32_t S_COL = 0, DP_COL = 128, OUT_COL = 256;   // sums: DP columns each
};

// The CTA's shared memory, which the tiles' swizzle wants at a multiple of
// 1024 bytes (it begins there: the kernels have no other shared memory). At
// any other place the kernel would compute nonsense: reported, never run.
__device__ __forceinline__ bool smem_aligned(const void* p, int* status) {
  if ((smem_u32(p) & 1023u) == 0) return true;
  if (threadIdx.x == 0) report_check(status, CHK_BUFFER, smem_u32(p));
  return false;
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

}  // namespace

// ---------------------------------------------------------------- dQ

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAttnThreads, 1)
    lin_attn_dq_kernel(const __grid_constant__ AttnBwdMaps maps,
                       const __grid_constant__ AttnBwdArgs args) {
  using C = BwdCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = args.s;
  const int h = blockIdx.x, b = blockIdx.z;
  const int qt = gridDim.y - 1 - blockIdx.y;   // longest rows of a causal mask first
  const int i0 = qt * 128;
  const SeqRange sq = seq_range(a.cu_q, b, a.tokens_q, a.max_q);
  const int64_t norm_at = ((int64_t)b * a.heads_q + h) * gridDim.y + qt;
  if (i0 >= sq.len) {   // (the whole CTA)
    if (threadIdx.x == 0) args.norm[norm_at] = 0.0f;
    return;
  }
  const SeqRange sk = seq_range(a.cu_k, b, a.tokens_k, a.max_k);
  const int last = min(i0 + 127, sq.len - 1);
  const int hi = a.causal ? min(sk.len, last + sk.len - sq.len + 1) : sk.len;
  const int n = hi > 0 ? (hi + 127) / 128 : 0;
  const int hk = h / a.group;

  if (!smem_aligned(smem_raw, a.status)) return;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* const ctl_gen = smem_raw + C::OFF_CTL;
  auto bar = [&](int slot) { return base + C::OFF_CTL + (uint32_t)slot * 8u; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = reinterpret_cast<volatile int*>(ctl_gen + C::OFF_ABORT);
  const WaitCtl ctl{a.timeout_ns, abort, a.status};
  const uint32_t q_tile = base + C::OFF_OWN, do_tile = q_tile + C::TILE;
  auto k_tile = [&](int s) { return base + C::OFF_A + (uint32_t)s * C::TILE; };
  auto v_tile = [&](int s) { return base + C::OFF_B + (uint32_t)s * C::TILE; };

  if (warp == kAttnMmaWarp) {
    tmem_alloc(base + C::OFF_CTL + C::OFF_TMEM, 512);
    tmem_relinquish_alloc_permit();
  }
  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < C::BARS; ++i)
      mbar_init(bar(i), C::by_half(i) ? 128 : 1);
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // (an allocation of all 512 columns begins at column 0)
  constexpr uint32_t tmem = 0;

  const int k_left = sk.len - (n - 1) * 128;   // keys of the last tile (128 or more: all)
  if (warp == kAttnCopyWarp) {
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(bar(C::OWN_FULL), 2 * C::TILE);
      load_tile<DP>(q_tile, &maps.q, h, sq.start + i0, bar(C::OWN_FULL));
      load_tile<DP>(do_tile, &maps.dout, h, sq.start + i0, bar(C::OWN_FULL));
      int a_issued = 0, b_issued = 0;
      for (int j = 0; j < n; ++j) {
        const int sa = j % C::NA, ra = j / C::NA, sb = j % C::NB, rb = j / C::NB;
        if (ra > 0 && !wait_phase(bar(C::A_EMPTY + sa), (ra - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar(C::A_FULL + sa), C::TILE);
        load_tile<DP>(k_tile(sa), &maps.k, hk, sk.start + j * 128, bar(C::A_FULL + sa));
        ++a_issued;
        if (rb > 0 && !wait_phase(bar(C::B_EMPTY + sb), (rb - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar(C::B_FULL + sb), C::TILE);
        load_tile<DP>(v_tile(sb), &maps.v, hk, sk.start + j * 128, bar(C::B_FULL + sb));
        ++b_issued;
      }
      if (*abort) {   // no copy may still be in flight when the CTA ends
        wait_phase(bar(C::OWN_FULL), 0, ctl, false);
        for (int j = max(0, a_issued - C::NA); j < a_issued; ++j)
          wait_phase(bar(C::A_FULL + j % C::NA), (j / C::NA) & 1, ctl, false);
        for (int j = max(0, b_issued - C::NB); j < b_issued; ++j)
          wait_phase(bar(C::B_FULL + j % C::NB), (j / C::NB) & 1, ctl, false);
      }
    }
    __syncwarp();
    if (n > 0 && k_left < 128) {   // cut the last K tile at the sequence's end (dS K runs over it)
      const int s = (n - 1) % C::NA;
      if (warp_wait_phase(bar(C::A_FULL + s), ((n - 1) / C::NA) & 1, ctl)) {
        zero_rows<DP>(k_tile(s), k_left, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::A_TAIL));
      }
    }
  } else if (warp == kAttnMmaWarp) {
    if (n > 0 && elect_one()) {   // one thread issues every product
      const uint64_t q_desc = AttnTile<DP>::k_major(q_tile), do_desc = AttnTile<DP>::k_major(do_tile);
      const uint64_t k_desc = AttnTile<DP>::k_major(k_tile(0)), v_desc = AttnTile<DP>::k_major(v_tile(0));
      const uint64_t kt_desc = AttnTile<DP>::mn_major(k_tile(0));
      constexpr uint64_t STAGE = AttnTile<DP>::UNITS;
      RingAt<C::NA> ka, kn;   // K of tile j, and of the next S
      RingAt<C::NB> vn;       // V of the next dP
      int kj = 0;             // tile of kn
      auto scores = [&]() -> bool {   // S = Q K^T of the next tile
        if (!wait_phase(bar(C::A_FULL + kn.s), kn.parity, ctl) ||
            (++kj == n && k_left < 128 && !wait_phase(bar(C::A_TAIL), 0, ctl)))
          return false;
        umma_entries<DP, BF16>(C::S_COL, q_desc, k_desc + kn.s * STAGE);
        umma_commit(bar(C::S_FULL));
        kn.next();
        return true;
      };
      auto dprobs = [&]() -> bool {   // dP = dO V^T of the next tile
        if (!wait_phase(bar(C::B_FULL + vn.s), vn.parity, ctl)) return false;
        umma_entries<DP, BF16>(C::DP_COL, do_desc, v_desc + vn.s * STAGE);
        umma_commit(bar(C::DP_FULL));
        umma_commit(bar(C::B_EMPTY + vn.s));
        vn.next();
        return true;
      };
      bool ok = wait_phase(bar(C::OWN_FULL), 0, ctl) && scores() && dprobs();
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) {
          ok = wait_phase(bar(C::S_DONE), j & 1, ctl) && wait_phase(bar(C::S_DONE + 1), j & 1, ctl);
          tc_fence_after_sync();
          ok = ok && scores();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && wait_phase(bar(C::DS_READY + half), j & 1, ctl);
          if (!ok) break;
          tc_fence_after_sync();
          umma_tokens<DP, BF16>(C::OUT_COL, C::DP_COL + half * 64, kt_desc + ka.s * STAGE, half,
                                j == 0 && half == 0);
        }
        if (!ok) break;
        umma_commit(bar(C::A_EMPTY + ka.s));
        ka.next();
        if (j + 1 < n) ok = dprobs();
      }
      // (also on the way out: tensor memory must be idle at the end)
      umma_commit(bar(C::OUT_FULL));
      wait_phase(bar(C::OUT_FULL), 0, ctl, false);
    }
    __syncwarp();
  } else {
    const int half = warp >> 2, row = tid & 127;
    const int i = i0 + row;
    const bool live = i < sq.len;
    const int64_t token = sq.start + (live ? i : 0);
    const float c = a.scale * kLog2E;
    // delta and the norm of dO's row: each of the row's two threads takes
    // every other group of eight entries
    float dsum = 0.0f, nsum = 0.0f;
    if (live) {
      const uint16_t* o = args.o.p + token * args.o.token_stride + (int64_t)h * args.o.head_stride;
      const uint16_t* g =
          args.dout.p + token * args.dout.token_stride + (int64_t)h * args.dout.head_stride;
#pragma unroll
      for (int e = 0; e < DP / 16; ++e) {
        const int col = e * 16 + half * 8;
        if (col < a.dim) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(o + col));
          const uint4 y = __ldg(reinterpret_cast<const uint4*>(g + col));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 u = unpack16<BF16>(xs[k]), v = unpack16<BF16>(ys[k]);
            dsum = fmaf(u.x, v.x, fmaf(u.y, v.y, dsum));
            nsum = fmaf(v.x, v.x, fmaf(v.y, v.y, nsum));
          }
        }
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
      if (live && n != 1) args.delta[(int64_t)h * a.tokens_q + token] = delta;
      float big = norm;   // (NaN rows do not count)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      if (lane == 0) red2[warp] = big;
    }
    named_bar_sync(1, 256);
    if (tid == 0)
      args.norm[norm_at] = fmaxf(fmaxf(red2[0], red2[1]), fmaxf(red2[2], red2[3]));
    const int ne = norm_exponent(norm);
    const float amp = pow2i(ne);
    float nd = -delta * amp;
    const float lse = live ? args.lse[(int64_t)h * a.tokens_q + token] : -INFINITY;
    // a row without a key (L = -inf) has no probabilities
    const float nl = lse == -INFINITY ? -INFINITY : -lse * kLog2E;
    // the last key that this row sees
    const int lim = live ? (a.causal ? min(sk.len - 1, i + sk.len - sq.len) : sk.len - 1) : -1;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + C::S_COL + half * 64;
    const uint32_t dp_col = tmem + lanes + C::DP_COL + half * 64;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = warp_wait_phase(bar(C::S_FULL), j & 1, ctl);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t p[2][32], d[2][32];
      tmem_ld_32x32b_x32(s_col, p[0]);
      tmem_ld_32x32b_x32(s_col + 32, p[1]);
      tmem_wait_ld_x32(p[0]);
      tmem_wait_ld_x32(p[1]);
      tc_fence_before_sync();
      mbar_arrive(bar(C::S_DONE + half));
      const float2 cc = make_float2(c, c), ll = make_float2(nl, nl);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(p[q][e]), __uint_as_float(p[q][e + 1])), cc, ll);
          p[q][e] = __float_as_uint(ex2_approx(x.x));
          p[q][e + 1] = __float_as_uint(ex2_approx(x.y));
        }
      ok = warp_wait_phase(bar(C::DP_FULL), j & 1, ctl);
      if (!ok) break;
      tc_fence_after_sync();
      tmem_ld_32x32b_x32(dp_col, d[0]);
      tmem_ld_32x32b_x32(dp_col + 32, d[1]);
      tmem_wait_ld_x32(d[0]);
      tmem_wait_ld_x32(d[1]);
      if (n == 1) {
        // All of the row's keys are in this tile, so delta is at hand as the
        // sum of P dP itself. It replaces the sum of dO O, whose O has been
        // rounded to 16 bits: with few keys that rounding is no longer small
        // against dP - delta (at one key the difference is zero).
        float sd = 0.0f, sp = 0.0f;
        const int lim_h = lim - half * 64;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e <= lim_h) {
              sd = fmaf(__uint_as_float(p[q][e]), __uint_as_float(d[q][e]), sd);
              sp += __uint_as_float(p[q][e]);
            }
        red[half * 128 + row] = sd;
        red[256 + half * 128 + row] = sp;
        named_bar_sync(1, 256);
        sp = red[256 + row] + red[384 + row];
        delta = sp > 0.0f ? (red[row] + red[128 + row]) / sp : 0.0f;
        nd = -delta * amp;
        if (half == 0 && live) args.delta[(int64_t)h * a.tokens_q + token] = delta;
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
      const int lim_j = lim - j * 128 - half * 64;
      if (__any_sync(0xffffffffu, lim_j < 63)) {   // masked keys, whatever their dP holds
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
      mbar_arrive(bar(C::DS_READY + half));
    }
    if (ok && n > 0) {
      ok = warp_wait_phase(bar(C::OUT_FULL), 0, ctl);
      tc_fence_after_sync();
    }
    if (ok) {
      const float back = a.scale * pow2i(-ne);
      uint16_t* out = args.dq.p + token * args.dq.token_stride + (int64_t)h * args.dq.head_stride;
#pragma unroll
      for (int q = 0; q < DP / 64; ++q) {
        const int c0 = half * (DP / 2) + q * 32;
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + C::OUT_COL + c0, o);
          tmem_wait_ld_x32(o);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = n > 0 ? pack16<BF16>(__uint_as_float(o[g * 8 + 2 * e]) * back,
                                        __uint_as_float(o[g * 8 + 2 * e + 1]) * back)
                         : 0u;
          const int col = c0 + g * 8;
          if (live && col < a.dim) store16(out + col, w[0], w[1], w[2], w[3]);
        }
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

template <int DP, bool BF16>
__global__ void __launch_bounds__(kDkvThreads, 1)
    lin_attn_dkv_kernel(const __grid_constant__ AttnBwdMaps maps,
                        const __grid_constant__ AttnBwdArgs args) {
  using C = BwdCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = args.s;
  const int hk = blockIdx.x, b = blockIdx.z;
  const int k0 = blockIdx.y * 128;   // a causal mask's first keys meet the most queries
  const SeqRange sk = seq_range(a.cu_k, b, a.tokens_k, a.max_k);
  if (k0 >= sk.len) return;   // (the whole CTA)
  const SeqRange sq = seq_range(a.cu_q, b, a.tokens_q, a.max_q);
  // query tiles t0 .. t1 - 1 of each head of the group
  const int off = sk.len - sq.len;   // causal: query i sees the keys up to i + off
  const int t1 = (sq.len + 127) / 128;
  const int t0 = a.causal ? min(max(k0 - off, 0) / 128, t1) : 0;
  const int per = t1 - t0;
  const int n = per * a.group;
  const int q_left = sq.len - (t1 - 1) * 128;   // queries of the last tile
  const int h0 = hk * a.group;

  if (!smem_aligned(smem_raw, a.status)) return;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* const ctl_gen = smem_raw + C::OFF_CTL;
  auto bar = [&](int slot) { return base + C::OFF_CTL + (uint32_t)slot * 8u; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = reinterpret_cast<volatile int*>(ctl_gen + C::OFF_ABORT);
  const WaitCtl ctl{a.timeout_ns, abort, a.status};
  const uint32_t k_tile = base + C::OFF_OWN, v_tile = k_tile + C::TILE;
  auto q_tile = [&](int s) { return base + C::OFF_A + (uint32_t)s * C::TILE; };
  auto do_tile = [&](int s) { return base + C::OFF_B + (uint32_t)s * C::TILE; };
  auto lse_rows = [&](int s) { return reinterpret_cast<float*>(smem_raw + C::OFF_ROWS) + s * 128; };
  auto delta_rows = [&](int s) { return lse_rows(C::NA + s); };

  if (warp == kAttnMmaWarp) {
    tmem_alloc(base + C::OFF_CTL + C::OFF_TMEM, 512);
    tmem_relinquish_alloc_permit();
  }
  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < C::BARS; ++i)
      mbar_init(bar(i), C::by_half(i) ? 128 : 1);
    fence_barrier_init();
  }
  // the largest row norm of dO that this tile meets (every tile of the
  // heads: the masked ones do no harm)
  float* red = reinterpret_cast<float*>(ctl_gen + C::OFF_RED);
  {
    const int tiles = (a.max_q + 127) / 128;
    const float* nm = args.norm + ((int64_t)b * a.heads_q + h0) * tiles;
    float big = 0.0f;
    for (int i = tid; i < tiles * a.group; i += kDkvThreads) big = fmaxf(big, nm[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) red[warp] = big;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // (an allocation of all 512 columns begins at column 0)
  constexpr uint32_t tmem = 0;
  float big = 0.0f;
#pragma unroll
  for (int w = 0; w < kDkvThreads / 32; ++w) big = fmaxf(big, red[w]);
  const int ne = norm_exponent(big);
  // scale of dP and delta: dS then carries 2^ne, P's 2^8 taken back
  const float damp = pow2i(ne) * pow2i(-(int)kPShift);

  if (warp == kAttnCopyWarp) {
    if (n > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(C::OWN_FULL), 2 * C::TILE);
        load_tile<DP>(k_tile, &maps.k, hk, sk.start + k0, bar(C::OWN_FULL));
        load_tile<DP>(v_tile, &maps.v, hk, sk.start + k0, bar(C::OWN_FULL));
      }
      int a_issued = 0, b_issued = 0;
      for (int it = 0; it < n; ++it) {
        const int sa = it % C::NA, ra = it / C::NA, sb = it % C::NB, rb = it / C::NB;
        const int h = h0 + it / per, i0 = (t0 + it % per) * 128;
        // the rows' statistics, in the form that the element-wise warps add:
        // rows behind the sequence's end and rows without a key have P = 0
        float nl[4], nd[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * 32 + lane;
          const int64_t at = (int64_t)h * a.tokens_q + sq.start + i;
          const float lse = i < sq.len ? args.lse[at] : -INFINITY;
          nl[e] = lse == -INFINITY ? -INFINITY : fmaf(-lse, kLog2E, kPShift);
          nd[e] = i < sq.len ? args.delta[at] * -damp : 0.0f;
        }
        if (ra > 0 && !lane0_wait_phase(bar(C::A_EMPTY + sa), (ra - 1) & 1, ctl, lane)) break;
        __syncwarp();   // (the stage's last readers are done for every lane)
#pragma unroll
        for (int e = 0; e < 4; ++e) lse_rows(sa)[e * 32 + lane] = nl[e];
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(C::A_FULL + sa), C::TILE);
          load_tile<DP>(q_tile(sa), &maps.q, h, sq.start + i0, bar(C::A_FULL + sa));
        }
        ++a_issued;
        if (rb > 0 && !lane0_wait_phase(bar(C::B_EMPTY + sb), (rb - 1) & 1, ctl, lane)) break;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) delta_rows(sb)[e * 32 + lane] = nd[e];
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(C::B_FULL + sb), C::TILE);
          load_tile<DP>(do_tile(sb), &maps.dout, h, sq.start + i0, bar(C::B_FULL + sb));
        }
        ++b_issued;
      }
      if (lane == 0 && *abort) {   // no copy may still be in flight when the CTA ends
        wait_phase(bar(C::OWN_FULL), 0, ctl, false);
        for (int it = max(0, a_issued - C::NA); it < a_issued; ++it)
          wait_phase(bar(C::A_FULL + it % C::NA), (it / C::NA) & 1, ctl, false);
        for (int it = max(0, b_issued - C::NB); it < b_issued; ++it)
          wait_phase(bar(C::B_FULL + it % C::NB), (it / C::NB) & 1, ctl, false);
      }
    }
  } else if (warp == kTailWarp) {
    // Where the last query tile of a head is cut by the sequence's end, this
    // warp hands every stage on to the products (a phase that nobody waited
    // for would not be told from the one before it), that tile with the rows
    // behind the end zeroed: they enter the products that run over the queries.
    if (n > 0 && q_left < 128) {
      int tile = 0;
      RingAt<C::NA> qa;
      RingAt<C::NB> da;
      for (int it = 0; it < n; ++it) {
        const bool cut = ++tile == per;
        if (cut) tile = 0;
        if (!warp_wait_phase(bar(C::A_FULL + qa.s), qa.parity, ctl)) break;
        if (cut) {
          zero_rows<DP>(q_tile(qa.s), q_left, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::A_TAIL + qa.s));
        if (!warp_wait_phase(bar(C::B_FULL + da.s), da.parity, ctl)) break;
        if (cut) {
          zero_rows<DP>(do_tile(da.s), q_left, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_TAIL + da.s));
        qa.next();
        da.next();
      }
    }
  } else if (warp == kAttnMmaWarp) {
    if (n > 0 && elect_one()) {   // one thread issues every product
      const uint64_t k_desc = AttnTile<DP>::k_major(k_tile), v_desc = AttnTile<DP>::k_major(v_tile);
      const uint64_t q_desc = AttnTile<DP>::k_major(q_tile(0)), do_desc = AttnTile<DP>::k_major(do_tile(0));
      const uint64_t qt_desc = AttnTile<DP>::mn_major(q_tile(0));
      const uint64_t dot_desc = AttnTile<DP>::mn_major(do_tile(0));
      constexpr uint64_t STAGE = AttnTile<DP>::UNITS;
      const int a_ready = q_left < 128 ? C::A_TAIL : C::A_FULL;
      const int b_ready = q_left < 128 ? C::B_TAIL : C::B_FULL;
      RingAt<C::NA> qa, qn;   // Q of tile it, and of the next S^T
      RingAt<C::NB> da, dn;   // dO of tile it, and of the next dP^T
      auto scores = [&]() -> bool {   // S^T = K Q^T of the next tile
        if (!wait_phase(bar(a_ready + qn.s), qn.parity, ctl)) return false;
        umma_entries<DP, BF16>(C::S_COL, k_desc, q_desc + qn.s * STAGE);
        umma_commit(bar(C::S_FULL));
        qn.next();
        return true;
      };
      auto dprobs = [&]() -> bool {   // dP^T = V dO^T of the next tile
        if (!wait_phase(bar(b_ready + dn.s), dn.parity, ctl)) return false;
        umma_entries<DP, BF16>(C::DP_COL, v_desc, do_desc + dn.s * STAGE);
        umma_commit(bar(C::DP_FULL));
        dn.next();
        return true;
      };
      bool ok = wait_phase(bar(C::OWN_FULL), 0, ctl) && scores() && dprobs();
      for (int it = 0; it < n && ok; ++it) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // dV += P^T dO
          ok = ok && wait_phase(bar(C::S_DONE + half), it & 1, ctl);
          if (!ok) break;
          tc_fence_after_sync();
          umma_tokens<DP, BF16>(C::OUT_COL, C::S_COL + half * 64, dot_desc + da.s * STAGE, half,
                                it == 0 && half == 0);
        }
        if (ok && it + 1 < n) ok = scores();
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // dK += dS^T Q
          ok = ok && wait_phase(bar(C::DS_READY + half), it & 1, ctl);
          if (!ok) break;
          tc_fence_after_sync();
          umma_tokens<DP, BF16>(C::OUT_COL + DP, C::DP_COL + half * 64, qt_desc + qa.s * STAGE, half,
                                it == 0 && half == 0);
        }
        if (!ok) break;
        // (dO's stage too: its rows' delta was read for dS)
        umma_commit(bar(C::A_EMPTY + qa.s));
        umma_commit(bar(C::B_EMPTY + da.s));
        qa.next();
        da.next();
        if (it + 1 < n) ok = dprobs();
      }
      // (also on the way out: tensor memory must be idle at the end)
      umma_commit(bar(C::OUT_FULL));
      wait_phase(bar(C::OUT_FULL), 0, ctl, false);
    }
    __syncwarp();
  } else {
    const int half = warp >> 2, row = tid & 127;
    const int key = k0 + row;
    const bool live = key < sk.len;
    const float c = a.scale * kLog2E;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + C::S_COL + half * 64;
    const uint32_t dp_col = tmem + lanes + C::DP_COL + half * 64;
    bool ok = true;
    int tile = 0;   // of its head
    RingAt<C::NA> qa;
    RingAt<C::NB> da;
    for (int it = 0; it < n; ++it) {
      const int i0 = (t0 + tile) * 128;
      if (++tile == per) tile = 0;
      const float4* nl = reinterpret_cast<const float4*>(lse_rows(qa.s) + half * 64);
      const float4* nd = reinterpret_cast<const float4*>(delta_rows(da.s) + half * 64);
      ok = warp_wait_phase(bar(C::S_FULL), it & 1, ctl);
      if (!ok) break;
      // (the rows' statistics came before the copies that the products waited for)
      ok = warp_wait_phase(bar(C::A_FULL + qa.s), qa.parity, ctl);
      if (!ok) break;
      qa.next();
      tc_fence_after_sync();
      uint32_t p[2][32], d[2][32], w[32];
      tmem_ld_32x32b_x32(s_col, p[0]);
      tmem_ld_32x32b_x32(s_col + 32, p[1]);
      tmem_wait_ld_x32(p[0]);
      tmem_wait_ld_x32(p[1]);
      const float2 cc = make_float2(c, c), pp = make_float2(damp, damp);
#pragma unroll
      for (int q = 0; q < 2; ++q)
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
      // causal: the key meets the queries from key - off on
      const int from = key - off - i0 - half * 64;
      const bool cut = a.causal && __any_sync(0xffffffffu, from > 0);
      if (cut) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e < from) p[q][e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e)
        w[e] = pack16<BF16>(__uint_as_float(p[e >> 4][(2 * e) & 31]),
                            __uint_as_float(p[e >> 4][(2 * e + 1) & 31]));
      tmem_st_32x32b_x32(s_col, w);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar(C::S_DONE + half));
      ok = warp_wait_phase(bar(C::DP_FULL), it & 1, ctl) &&
           warp_wait_phase(bar(C::B_FULL + da.s), da.parity, ctl);
      if (!ok) break;
      da.next();
      tc_fence_after_sync();
      tmem_ld_32x32b_x32(dp_col, d[0]);
      tmem_ld_32x32b_x32(dp_col + 32, d[1]);
      tmem_wait_ld_x32(d[0]);
      tmem_wait_ld_x32(d[1]);
#pragma unroll
      for (int q = 0; q < 2; ++q)
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
      if (cut) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e < from) d[q][e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e)
        w[e] = pack16<BF16>(__uint_as_float(d[e >> 4][(2 * e) & 31]),
                            __uint_as_float(d[e >> 4][(2 * e + 1) & 31]));
      tmem_st_32x32b_x32(dp_col, w);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar(C::DS_READY + half));
    }
    if (ok && n > 0) {
      ok = warp_wait_phase(bar(C::OUT_FULL), 0, ctl);
      tc_fence_after_sync();
    }
    if (ok) {   // the first half's threads write dV, the others dK
      const float back = half == 0 ? pow2i(-(int)kPShift) : a.scale * pow2i(-ne);
      const HeadsPtr& g = half == 0 ? args.dv : args.dk;
      uint16_t* out = g.p + (int64_t)(sk.start + (live ? key : 0)) * g.token_stride +
                      (int64_t)hk * g.head_stride;
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + C::OUT_COL + half * DP + q * 32, o);
          tmem_wait_ld_x32(o);
        }
#pragma unroll
        for (int e8 = 0; e8 < 4; ++e8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = n > 0 ? pack16<BF16>(__uint_as_float(o[e8 * 8 + 2 * e]) * back,
                                        __uint_as_float(o[e8 * 8 + 2 * e + 1]) * back)
                         : 0u;
          const int col = q * 32 + e8 * 8;
          if (live && col < a.dim) store16(out + col, w[0], w[1], w[2], w[3]);
        }
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

cudaError_t launch_attn_bwd(bool bf16, const AttnBwdMaps& maps, const AttnBwdArgs& args,
                            int heads_kv, int sequences, cudaStream_t stream) {
  const unsigned tq = (unsigned)((args.s.max_q + 127) / 128);
  const unsigned tk = (unsigned)((args.s.max_k + 127) / 128);
  auto go = [&](auto kernel, uint32_t smem, dim3 grid, int threads) {
    if (grid.x == 0 || grid.y == 0 || grid.z == 0) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads, smem, stream>>>(maps, args);
    return cudaGetLastError();
  };
  auto both = [&](auto dq, auto dkv, uint32_t smem) {
    const cudaError_t e =
        go(dq, smem, dim3((unsigned)(heads_kv * args.s.group), tq, (unsigned)sequences),
           kAttnThreads);
    if (e != cudaSuccess) return e;
    return go(dkv, smem, dim3((unsigned)heads_kv, tk, (unsigned)sequences), kDkvThreads);
  };
  if (args.s.dim <= 64)
    return bf16 ? both(lin_attn_dq_kernel<64, true>, lin_attn_dkv_kernel<64, true>, BwdCfg<64>::SMEM)
                : both(lin_attn_dq_kernel<64, false>, lin_attn_dkv_kernel<64, false>,
                       BwdCfg<64>::SMEM);
  return bf16
             ? both(lin_attn_dq_kernel<128, true>, lin_attn_dkv_kernel<128, true>, BwdCfg<128>::SMEM)
             : both(lin_attn_dq_kernel<128, false>, lin_attn_dkv_kernel<128, false>,
                    BwdCfg<128>::SMEM);
}

}  // namespace lin
