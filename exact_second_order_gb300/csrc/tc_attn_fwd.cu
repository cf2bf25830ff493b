// Attention with key ranges on sm_103a tensor cores: bf16, head dim 64 or 128.
//   S = Q K^T,  s = score(S) (scale, cap, bias; log2 units),
//   P~ = exp2(s - m) with a running row maximum m,  l = sum P~,
//   O = (sum P~ V) / l,  L = (m + log2 l) ln 2.
//
// Warp 0 TMA, warp 1 TMEM allocation and MMA issue, then NW = 2 elementwise
// warpgroups.  The block's work is a run of units; unit u goes to warpgroup
// u mod 2 and one of three score buffers in TMEM, where P~ (bf16) replaces the
// scores as the A operand of P~ V.  Each warpgroup has its own O~ accumulator
// and raises its m only when a unit's maximum exceeds it by more than 8 (log2
// units), so O~ is rarely rescaled.
//   MT = 1: 128 group rows a block, the warpgroups take alternate key tiles and
//     merge their (m, l, O~) at the end.  Where rows are few (tokens over a
//     cache) the keys are also cut into runs of blocks joined by a second launch.
//   MT = 2: 256 group rows, warpgroup w holds rows 128 w .. and both take every
//     key tile, so a tile from L2 feeds twice the products (see two_blocks).
//   NW = 1 (d = 64, MT = 1): one warpgroup, tiles of 64 keys, half of an SM's
//     TMEM and shared memory, so that two blocks fill and drain beside each
//     other (see small_blocks).
//   TOKEN (MT = 1, up to 32 group rows): Q lies four times in the tile, once for
//     each warp of a warpgroup, and each warp takes a quarter of the columns (its
//     P~ is 0 in the others), so no warp works on a whole tile alone; the warps'
//     parts are merged like those of the warpgroups.
// Key tiles outside the hull of the block's ranges are not visited; tiles
// inside every row's range run without a mask.  V rows outside the hull are
// zeroed in shared memory before they meet P~ = 0, so a cache may hold
// anything behind its last key.
// TMEM: O~ of each warpgroup (DH columns), then three score buffers.
// P~ is rounded to bf16, the MMA's other operand V being bf16 (a product of two
// halves of P~ would double its MMAs); l sums it unrounded.  O is off by 2.3e-3 in
// norm for that and its own rounding (alone 1.7e-3).
// Measured (B1 H8 N16384, no mask): 516 us at d = 64, 1066 TFLOP/s, where the
// hand-offs between MMAs and elementwise warps bound it (with MT = 2, 590 us, a
// copy without arithmetic took 515, one with a quarter of the MMAs 480); 737 us
// at d = 128, 1492 TFLOP/s, bound by the MMAs.  Tokens over a cache: 82% of the copy
// rate (32 requests of up to 8192 keys, 8 heads of 128, 122 us).
#include "tc_attn.cuh"

namespace flashbob {
namespace {
using namespace tc;
using namespace attn;

constexpr int BM = kTcRows;
constexpr int NBUF = 3;
constexpr uint32_t HALF_BLOCK = BM * 64 * 2;
constexpr float kRescale = 8.f;

template <int DH, int MT, int NW, bool TOKEN>
struct Cfg {
  static constexpr int kThreads = 64 + 128 * NW;
  static constexpr int kHalves = DH / 64;
  static constexpr int kBN = DH == 64 && NW == 2 ? 128 : 64;
  static constexpr uint32_t kHalfTile = kBN * 64 * 2;
  // K and V arrive and leave together: the MMA warp's waits count where the MMAs
  // bound the kernel (with rings of their own 890 us for 741 at B1 H8 N16384
  // d128).  For tokens, which the loads bound, they do not: a K tile is free after
  // its scores, a V tile three units later (an SM then reads a cache at more than
  // 45 GB/s: 130 -> 122 us for the 32 requests below).
  static constexpr bool kJoint = !TOKEN;
  static constexpr int kPairs = (MT == 2 || NW == 1 ? 5 : 6) - (DH == 64 ? 0 : 1);
  static constexpr int kK = kJoint ? kPairs : 5;
  static constexpr int kV = kJoint ? kPairs : DH == 64 && NW == 2 ? 7 : 6;
  static constexpr int k_tile(int s) { return kJoint ? 2 * s : s; }  // in the one array of tiles
  static constexpr int v_tile(int s) { return kJoint ? 2 * s + 1 : kK + s; }
  static constexpr int kColumns = 256 * NW;
  static_assert(NW * DH + NBUF * kBN <= kColumns, "TMEM columns");
  static_assert(NBUF <= kK && NBUF <= kV, "the first scores need their tiles at once");
  static_assert(!kJoint || kK == kV, "one ring");
};

constexpr int kStageLd = 64 + 4;  // epilogue: 64 columns of every row at a time

template <int DH, int MT, int NW, bool TOKEN>
struct SmemF {
  using C = Cfg<DH, MT, NW, TOKEN>;
  static constexpr int NK = C::kK, NV = C::kV, NH = C::kHalves;
  alignas(1024) uint8_t q[MT][NH][HALF_BLOCK];
  alignas(1024) uint8_t kv[NK + NV][NH][C::kHalfTile];
  float part_m[2][BM];
  float part_l[2][BM];
  int hull[4 * NW][4];  // of each elementwise warp's rows
  uint64_t bar_q;
  uint64_t k_full[NK], k_empty[NK];
  uint64_t v_full[NV], v_empty[NV];
  uint64_t sc_full[NBUF];
  uint64_t op_ready[NBUF];
  uint64_t pv_done[2];  // of even and odd units
  uint64_t out_full;
  uint32_t tmem_base;
  int abort_flag;
};

// Largest visible score of 16 NQ columns from jbase on (log2 units, relative to
// nothing).  Without a bias the score grows with the raw product, so the
// maximum is taken over those.
template <bool MASKED, int NQ, bool CAP, bool BIAS>
__device__ __forceinline__ float largest(const Score<CAP, BIAS>& sc, const uint32_t (&s)[NQ][16],
                                         int jbase, int lo, int hi, float dist) {
  float mr = -INFINITY;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int j = jbase + 16 * q + e;
      float2 x = f2(s[q][e], s[q][e + 1]);
      if (BIAS) x = sc.from(x, dist + (16 * q + e), 0.f, sc.slope2);
      if (!MASKED || (j >= lo && j < hi)) mr = fmaxf(mr, x.x);
      if (!MASKED || (j + 1 >= lo && j + 1 < hi)) mr = fmaxf(mr, x.y);
    }
  return mr;
}

// P~ of those columns as bf16 pairs, added to the row sum (before rounding).
template <bool MASKED, int NQ, bool CAP, bool BIAS>
__device__ __forceinline__ void weights(const Score<CAP, BIAS>& sc, const uint32_t (&s)[NQ][16],
                                        int jbase, int lo, int hi, float dist, float m, float& l,
                                        uint32_t (&pk)[NQ][8]) {
  float2 acc = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 t = sc.from(f2(s[q][e], s[q][e + 1]), dist + (16 * q + e), m, sc.slope2);
      float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
      if (MASKED) {
        const int j = jbase + 16 * q + e;
        if (j < lo || j >= hi) p.x = 0.f;
        if (j + 1 < lo || j + 1 >= hi) p.y = 0.f;
      }
      acc = fadd2(acc, p);
      pk[q][e >> 1] = pack_bf16x2(p.x, p.y);
    }
  l += acc.x + acc.y;
}

template <int DH, int MT, int NW, bool TOKEN, bool CAP, bool BIAS>
__global__ void __launch_bounds__((Cfg<DH, MT, NW, TOKEN>::kThreads), (NW == 1 ? 2 : 1))
    tc_attn_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                   const __grid_constant__ CUtensorMap mV, const __grid_constant__ AttnArgs a,
                   int blocks, int splits) {
  extern __shared__ uint8_t smem_raw[];
  using C = Cfg<DH, MT, NW, TOKEN>;
  constexpr int NK = C::kK, NV = C::kV, NH = C::kHalves, BN = C::kBN;
  constexpr uint32_t HT = C::kHalfTile;
  constexpr uint32_t kScore = NW * DH;
  SmemF<DH, MT, NW, TOKEN>& sm = *reinterpret_cast<SmemF<DH, MT, NW, TOKEN>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.B * a.Hkv, G = a.H / a.Hkv, rows = G * a.Nq;
  const int g = blockIdx.x % heads, rest = blockIdx.x / heads;
  const int split = rest % splits;
  const int row0 = row_block(rest / splits, blocks, G, a.Nq, MT * BM) * (MT * BM);
  volatile int* abort_flag = &sm.abort_flag;
  unsigned int* err = a.err;

  if (splits > 1) release_next();
  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_q, 1);
    for (int s = 0; s < NK; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < NV; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], 1);
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&sm.sc_full[b], 1);
      mbar_init(&sm.op_ready[b], 4);
    }
    mbar_init(&sm.pv_done[0], 1);
    mbar_init(&sm.pv_done[1], 1);
    mbar_init(&sm.out_full, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    // Q is under way while the ranges are read.
    mbar_expect_tx(&sm.bar_q, MT * NH * HALF_BLOCK);
    for (int w = 0; w < MT; ++w)
      for (int h = 0; h < NH; ++h) {
        if (!TOKEN) tma_load_3d(sm.q[w][h], &mQ, &sm.bar_q, 64 * h, row0 + BM * w, g);
        else  // boxes of 32 rows, the same four times
          for (int q = 0; q < 4; ++q)
            tma_load_3d(sm.q[w][h] + q * (HALF_BLOCK / 4), &mQ, &sm.bar_q, 64 * h, row0, g);
      }
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, C::kColumns);
  // Elementwise threads: TMEM lane r of row block w.
  const int wg = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
  GroupRow gr{empty_view(), 0.f};
  const int row = row0 + (TOKEN ? lane : r) + (MT == 2 ? BM * wg : 0);
  if (warp >= 2) {
    gr = group_row(a, g / a.Hkv, g % a.Hkv, row, rows);
    warp_hull(gr.v, row < rows, lane, sm.hull[4 * wg + quad]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const Hull hull = join_hulls(sm.hull, 4 * NW);
  // Key tiles of the hull, and this split's run of them.
  const int t_lo = hull.lo < hull.hi ? hull.lo / BN : 0;
  const int t_n = hull.lo < hull.hi ? (hull.hi + BN - 1) / BN - t_lo : 0;
  const int tb = t_lo + static_cast<int>(static_cast<long long>(t_n) * split / splits);
  const int T = t_lo + static_cast<int>(static_cast<long long>(t_n) * (split + 1) / splits) - tb;
  const int U = MT * T;  // units

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&mK);
      tma_prefetch_desc(&mV);
      int nk = 0, nv = 0;
      for (int t = 0; t < T; ++t) {
        const int sk = t % NK, sv = t % NV;
        uint64_t* v_bar = C::kJoint ? &sm.k_full[sk] : &sm.v_full[sv];
        if (!C::kJoint && t >= NK &&
            !wait_one(&sm.k_empty[sk], ((t / NK) - 1) & 1, abort_flag, err))
          break;
        if (C::kJoint && t >= NV &&
            !wait_one(&sm.v_empty[sv], ((t / NV) - 1) & 1, abort_flag, err))
          break;
        mbar_expect_tx(&sm.k_full[sk], (C::kJoint ? 2 : 1) * NH * HT);
        for (int h = 0; h < NH; ++h)
          tma_load_3d(sm.kv[C::k_tile(sk)][h], &mK, &sm.k_full[sk], 64 * h, (tb + t) * BN, g);
        nk = t + 1;
        if (!C::kJoint) {
          if (t >= NV && !wait_one(&sm.v_empty[sv], ((t / NV) - 1) & 1, abort_flag, err)) break;
          mbar_expect_tx(v_bar, NH * HT);
        }
        for (int h = 0; h < NH; ++h)
          tma_load_3d(sm.kv[C::v_tile(sv)][h], &mV, v_bar, 64 * h, (tb + t) * BN, g);
        if (!C::kJoint) nv = t + 1;
      }
      drain_wait(&sm.bar_q, 0);
      for (int t = nk > NK ? nk - NK : 0; t < nk; ++t) drain_wait(&sm.k_full[t % NK], (t / NK) & 1);
      for (int t = nv > NV ? nv - NV : 0; t < nv; ++t) drain_wait(&sm.v_full[t % NV], (t / NV) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = idesc_bf16(BM, BN, false);
    constexpr uint32_t idO = idesc_bf16(BM, DH, true);
    const uint64_t dQ = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t dK0 = smem_desc_sw128(smem_u32(sm.kv[C::k_tile(0)][0]), 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(smem_u32(sm.kv[C::v_tile(0)][0]), HT, 1024);
    constexpr uint64_t kStep = (C::k_tile(1) * sizeof(sm.kv[0])) >> 4;  // V's is the same
    auto tile = [](int u) { return MT == 2 ? u >> 1 : u; };
    auto issue_scores = [&](int u) {
      const uint64_t so = (tile(u) % NK) * kStep;
      const uint64_t qo = MT == 2 ? (u & 1) * (uint64_t)((NH * HALF_BLOCK) >> 4) : 0;
      const uint32_t sc = tbase + kScore + BN * (u % NBUF);
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint32_t h = kk >> 2, o = 32 * (kk & 3);
        mma_ss(sc, dQ + qo + ((h * HALF_BLOCK + o) >> 4), dK0 + so + ((h * HT + o) >> 4), idS,
               kk > 0);
      }
      mma_commit(&sm.sc_full[u % NBUF]);
      if (!C::kJoint) mma_commit(&sm.k_empty[tile(u) % NK]);
    };
    auto issue_pv = [&](int u) {
      const int s = tile(u) % NV;
      const uint32_t sc = tbase + kScore + BN * (u % NBUF);
      const uint64_t dv = dV0 + s * kStep;
      const uint32_t acc_col = tbase + DH * (u % NW);
#pragma unroll
      for (int c = 0; c < BN / 16; ++c)
        mma_ts(acc_col, sc + 8 * c, dv + ((16 * 128 * c) >> 4), idO, (u >= NW || c > 0));
      mma_commit(&sm.pv_done[u & 1]);
      if (MT == 1 || (u & 1)) mma_commit(&sm.v_empty[s]);
    };
    if (elect_one()) {
      bool ok = wait_one(&sm.bar_q, 0, abort_flag, err);
      tc_fence_after();
      for (int u = 0; ok && u < NBUF && u < U; ++u) {
        ok = wait_one(&sm.k_full[tile(u) % NK], (tile(u) / NK) & 1, abort_flag, err);
        tc_fence_after();
        if (ok) issue_scores(u);
      }
      for (int u = 0; ok && u < U; ++u) {
        ok = (C::kJoint || wait_one(&sm.v_full[u % NV], (u / NV) & 1, abort_flag, err)) &&
             wait_one(&sm.op_ready[u % NBUF], (u / NBUF) & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        issue_pv(u);
        if (u + NBUF < U) {
          const int tn = tile(u + NBUF);
          ok = wait_one(&sm.k_full[tn % NK], (tn / NK) & 1, abort_flag, err);
          if (!ok) break;
          tc_fence_after();
          issue_scores(u + NBUF);
        }
      }
      mma_commit(&sm.out_full);
    }
    __syncwarp();
  } else {
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t acc_own = tbase + lane_off + DH * wg;
    const int lo = gr.v.lo, hi = gr.v.hi;
    const Hull own = MT == 2 ? join_hulls(sm.hull + 4 * wg, 4) : hull;
    const Score<CAP, BIAS> score(a, gr.slope2);
    const bool any_row = TOKEN || row0 + (MT == 2 ? BM * wg : 0) + quad * 32 < rows;
    // V rows that no row of the block sees meet P~ = 0: make them 0 too.
    auto clear_hidden = [&](int u, int col0) {
      if (col0 >= hull.lo && col0 + BN <= hull.hi) return true;
      const int t = MT == 2 ? u >> 1 : u;
      if (!C::kJoint && !wait_warp(&sm.v_full[t % NV], (t / NV) & 1, abort_flag, err))
        return false;
      if (r < BN && (col0 + r < hull.lo || col0 + r >= hull.hi))
        zero_row<NH, HT>(sm.kv[C::v_tile(t % NV)], r);
      fence_proxy_async_smem();
      return true;
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;  // units of this warpgroup
    for (int u = wg; u < U; u += NW, ++n) {
      const int col0 = (tb + (MT == 2 ? u >> 1 : u)) * BN;
      ok = ok && wait_warp(&sm.sc_full[u % NBUF], (u / NBUF) & 1, abort_flag, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sc = tbase + lane_off + kScore + BN * (u % NBUF);
      const bool masked = col0 < own.in_lo || col0 + BN > own.in_hi;
      const float dist = BIAS ? static_cast<float>(col0 - gr.v.pos) : 0.f;
      if (!any_row) {
        ok = clear_hidden(u, col0);
        if (!ok) break;
        warp_arrive(&sm.op_ready[u % NBUF]);
        continue;
      }
      // Two 64-column groups at d = 64: the second is read twice, so that one
      // group is held in registers at a time, and P~ of columns 16 c .. goes
      // to columns 8 c .., onto scores already used.
      // TOKEN: the columns of this warp alone.
      constexpr int kGroup = TOKEN ? BN / 4 : 64, NQ = kGroup / 16;
      const int c_own = TOKEN ? kGroup * quad : 0, c_end = TOKEN ? c_own + kGroup : BN;
      float mr = -INFINITY;
      uint32_t s[NQ][16];
      auto load = [&](int c) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) tmem_ld16(sc + c + 16 * q, s[q]);
        tmem_wait_ld();
      };
      auto max_of = [&](int c) {
        if (BIAS) score.tanh_of(s, masked);
        mr = fmaxf(mr, masked ? largest<true>(score, s, col0 + c, lo, hi, dist + c)
                              : largest<false>(score, s, col0 + c, lo, hi, dist + c));
      };
      if (!TOKEN && BN == 128) {
        load(64);
        max_of(64);
      }
      load(c_own);
      max_of(c_own);
      float mt = mr;
      if (!BIAS) {
        mt = mr * score.c1;
        if (CAP && mr != -INFINITY) mt = score.c2 * score.tanh_one(mr);
      }
      const bool raise = mt > m + kRescale;
      const float factor = raise ? (m == -INFINITY ? 0.f : ex2_approx(m - mt)) : 1.f;
      if (raise) {
        l *= factor;
        m = mt;
      }
      if (__any_sync(0xffffffffu, raise && factor < 1.f) && n > 0) {
        // The products of this warpgroup's last unit.  S(u) was issued behind
        // those of unit u - 3, so of the barrier's phases only the last may be
        // open, and its parity tells.
        const int last = u - NW;
        ok = wait_warp(&sm.pv_done[last & 1], (last >> 1) & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < DH / 16; ++c) {
          uint32_t v[16];
          tmem_ld16(acc_own + 16 * c, v);
          tmem_wait_ld();
          uint32_t w0[8], w1[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            w0[k] = __float_as_uint(u2f(v[k]) * factor);
            w1[k] = __float_as_uint(u2f(v[8 + k]) * factor);
          }
          tmem_st8(acc_own + 16 * c, w0);
          tmem_st8(acc_own + 16 * c + 8, w1);
        }
      }
#pragma unroll
      for (int c = c_own; c < c_end; c += kGroup) {
        if (c > c_own) load(c);
        if (!BIAS || c > c_own) score.tanh_of(s, masked);
        uint32_t pk[NQ][8];
        if (masked) weights<true>(score, s, col0 + c, lo, hi, dist + c, m, l, pk);
        else weights<false>(score, s, col0 + c, lo, hi, dist + c, m, l, pk);
#pragma unroll
        for (int q = 0; q < NQ; ++q) tmem_st8(sc + c / 2 + 8 * q, pk[q]);
      }
      if (TOKEN) {  // P~ of the columns of the others
        const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
        for (int c = 0; c < BN / 16; ++c)
          if (c / NQ != quad) tmem_st8(sc + 8 * c, none);
      }
      ok = clear_hidden(u, col0);
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&sm.op_ready[u % NBUF]);
    }

    ok = wait_warp(&sm.out_full, 0, abort_flag, err) && ok;
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    tc_fence_after();
    // MT = 1: merge the warpgroups' (m, l, O~): m* = max, s_w = exp2(m_w - m*),
    // O~ = s_0 O~_0 + s_1 O~_1, l = s_0 l_0 + s_1 l_1.  An accumulator whose
    // warpgroup had no unit was never written.
    float mm = m, lsum = l, s0 = 1.f, s1 = 0.f;
    if (TOKEN) {
      // The same for the row's parts in all warps; each warp scales its own.
      sm.part_m[wg][r] = m;
      sm.part_l[wg][r] = l;
      named_bar_sync(1, 128 * NW);
      for (int w = 0; w < 4 * NW; ++w) mm = fmaxf(mm, sm.part_m[w / 4][32 * (w % 4) + lane]);
      lsum = 0.f;
      for (int w = 0; w < 4 * NW; ++w) {
        const float mw = sm.part_m[w / 4][32 * (w % 4) + lane];
        if (mw != -INFINITY) lsum += ex2_approx(mw - mm) * sm.part_l[w / 4][32 * (w % 4) + lane];
      }
      s0 = m == -INFINITY ? 0.f : ex2_approx(m - mm);
    } else if (MT == 1 && NW == 2) {
      sm.part_m[wg][r] = m;
      sm.part_l[wg][r] = l;
      named_bar_sync(1, 128 * NW);
      const float m0 = sm.part_m[0][r], m1 = sm.part_m[1][r];
      mm = fmaxf(m0, m1);
      s0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - mm);
      s1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
      lsum = s0 * sm.part_l[0][r] + s1 * sm.part_l[1][r];
    }
    const bool any0 = T > (TOKEN ? wg : 0), any1 = !TOKEN && MT == 1 && NW == 2 && T > 1;
    const float inv = splits > 1 ? 1.f : lsum > 0.f ? 1.f / lsum : 0.f;
    s0 = any0 ? s0 * inv : 0.f;
    s1 = any1 ? s1 * inv : 0.f;
    const size_t all = static_cast<size_t>(a.B) * a.H * a.Nq;
    const size_t base = static_cast<size_t>(g) * rows;  // first row of the group
    const Partials part = partials(a.workspace, all, DH, splits);
    if (ok && row < rows && (MT == 2 || wg == 0) && (!TOKEN || quad == 0)) {
      if (splits > 1) part.ml[split * all + base + row] = make_float2(mm, lsum);
      else a.L[base + row] = (mm + __log2f(lsum)) * kLn2;
    }
    // Every MMA is done, so the ring is idle: 64 columns of O at a time go
    // through it and leave with coalesced stores.
    float* st = reinterpret_cast<float*>(&sm.kv[0][0][0]);
    static_assert((TOKEN ? NW : MT) * BM * kStageLd * 4 <= sizeof(sm.kv),
                  "epilogue staging fits in the ring");
    const int tid = threadIdx.x - 64;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h > 0) named_bar_sync(1, 128 * NW);
      // With one accumulator for two warpgroups each forms half the columns.
      constexpr bool kShare = !TOKEN && MT == 1 && NW == 2;
      constexpr int kCols = kShare ? 32 : 64;
      const int c0 = kShare ? 32 * wg : 0;
      const int sr = MT == 2 || TOKEN ? BM * wg + r : r;
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        const uint32_t col = 64 * h + c0 + c;
        uint32_t v0[16], v1[16];
        if (!kShare) {
          tmem_ld16(acc_own + col, v0);
        } else {
          tmem_ld16(tbase + lane_off + col, v0);
          tmem_ld16(tbase + lane_off + DH + col, v1);
        }
        tmem_wait_ld();
        float4* s4 = reinterpret_cast<float4*>(st + sr * kStageLd + c0 + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[q] = any0 ? s0 * u2f(v0[4 * k + q]) : 0.f;
            if (kShare && any1) o[q] = fmaf(s1, u2f(v1[4 * k + q]), o[q]);
          }
          s4[k] = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      named_bar_sync(1, 128 * NW);
      const int live = min(MT * BM, rows - row0);
      if (ok) {
        for (int f = tid; f < live * 16; f += 128 * NW) {
          const int rr = f >> 4, c4 = f & 15;
          float4 v = *reinterpret_cast<const float4*>(st + rr * kStageLd + 4 * c4);
          if (TOKEN) {
#pragma unroll
            for (int w = 1; w < 4 * NW; ++w) {
              const float4 x =
                  *reinterpret_cast<const float4*>(st + (32 * w + rr) * kStageLd + 4 * c4);
              v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
          }
          const size_t at = (base + row0 + rr) * DH + 64 * h + 4 * c4;
          if (splits > 1) {
            *reinterpret_cast<float4*>(part.o + split * all * DH + at) = v;
          } else {
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + at) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, C::kColumns);
  }
}

template <int DH, int MT, int NW, bool TOKEN, bool CAP, bool BIAS>
cudaError_t launch(const AttnArgs& a, int splits) {
  const int heads = a.B * a.Hkv, rows = a.H / a.Hkv * a.Nq;
  using C = Cfg<DH, MT, NW, TOKEN>;
  CUtensorMap mq, mk, mv;
  cudaError_t e = tc_map_bf16(&mq, a.Q, heads, rows, TOKEN ? BM / 4 : BM, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mk, a.K, heads, a.Nk, C::kBN, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mv, a.V, heads, a.Nk, C::kBN, DH);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(SmemF<DH, MT, NW, TOKEN>) + 1024;
  static_assert(smem <= (NW == 1 ? 115712 : 232448), "shared memory");
  const auto kernel = tc_attn_kernel<DH, MT, NW, TOKEN, CAP, BIAS>;
  e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int blocks = (rows + MT * BM - 1) / (MT * BM);
  const long long grid = static_cast<long long>(blocks) * splits * heads;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  kernel<<<static_cast<unsigned>(grid), C::kThreads, smem, a.stream>>>(mq, mk, mv, a, blocks, splits);
  return cudaGetLastError();
}

template <int DH, int MT, int NW, bool TOKEN = false>
cudaError_t launch(const AttnArgs& a, int splits) {
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  return cap ? (bias ? launch<DH, MT, NW, TOKEN, true, true>(a, splits)
                     : launch<DH, MT, NW, TOKEN, true, false>(a, splits))
             : (bias ? launch<DH, MT, NW, TOKEN, false, true>(a, splits)
                     : launch<DH, MT, NW, TOKEN, false, false>(a, splits));
}

}  // namespace

bool tc_attn_supported(const AttnArgs& a) { return a.bf16 && (a.d == 64 || a.d == 128); }

namespace {

// 256 rows a block at d = 128 where such blocks fill the GPU twice (B1 H8
// N16384: 747 us, with 128 rows 791); 128 rows below (B2 H16 Hkv4 N2047: 79 us,
// with 256 rows, 1.7 waves, 101) and at d = 64 always (524 us, with 256 rows
// 581: the smaller tiles leave the key stream far from L2's rate).
bool two_blocks(const AttnArgs& a) {
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  return a.d == 128 && rows > BM &&
         static_cast<long long>(a.B) * a.Hkv * ((rows + 255) / 256) >= 2 * kSMs;
}

// Two small blocks an SM at d = 64 where a block's fixed cost counts: few keys
// (B8 H12 N256 causal 20 -> 16 us, B4 H12 N1024 in 5 documents 32 -> 26; equal at
// N1024 without a mask and at N2048 with a causal one, and 52 for 46 without),
// and the tokens of many requests (B64 H8, 2048 keys: 73 -> 65 us).  At d = 128
// only two stages fit (32 requests of 4096 keys: 124 for 108 us).
bool small_blocks(const AttnArgs& a) {
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  return a.Nk <= 1024 ||
         (rows <= BM && static_cast<long long>(a.B) * a.Hkv > kSMs);
}

}  // namespace

// How many runs the keys are cut into: as many as fill the SMs once, with
// kSplitKeys keys at least in each.  (More runs than SMs only add to the join:
// 8 groups of 65536 keys 28 us, with twice the runs 40 us.  With 256 keys a run
// the calls between 512 and 8192 keys gain up to 2 us of 20 on the GPU, but the
// short ones wait for the host, and the join is another launch.)
constexpr int kSplitKeys = 512;
int tc_attn_splits(const AttnArgs& a) {
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  const long long blocks = static_cast<long long>(a.B) * a.Hkv * ((rows + BM - 1) / BM);
  const long long want = kSMs / blocks, most = a.Nk / kSplitKeys;
  const long long s = want < most ? want : most;
  return two_blocks(a) || s < 1 ? 1 : static_cast<int>(s);
}

cudaError_t tc_attn(const AttnArgs& a) {
  const int splits = tc_attn_splits(a);
  cudaError_t e;
  // Up to 32 group rows: the TOKEN kernels (32 requests of up to 8192 keys, capped,
  // H32 Hkv8 d128: 137 -> 130 us; one of 1000 keys, H12 d64: 17.5 -> 13.5 us).
  const bool token = static_cast<long long>(a.H / a.Hkv) * a.Nq <= BM / 4;
  if (a.d == 64 && small_blocks(a))
    e = token ? launch<64, 1, 1, true>(a, splits) : launch<64, 1, 1>(a, splits);
  else if (a.d == 64)
    e = token ? launch<64, 1, 2, true>(a, splits) : launch<64, 1, 2>(a, splits);
  else if (token) e = launch<128, 1, 2, true>(a, splits);
  else e = two_blocks(a) ? launch<128, 2, 2>(a, splits) : launch<128, 1, 2>(a, splits);
  return e == cudaSuccess && splits > 1 ? attn_join(a, splits) : e;
}

}  // namespace flashbob
