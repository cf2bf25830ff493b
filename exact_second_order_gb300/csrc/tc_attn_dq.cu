// dQ of attention with key ranges on sm_103a tensor cores: bf16, head dim 64
// or 128.  128 group rows (Q, dO) stay on chip, the key tiles of their hull
// stream past:
//   S = Q K^T, dP = dO V^T;  P = exp2(score(S) - L log2 e),
//   dS = P (dP - D) (1 - tanh^2),  dQ += dS K;  dQ = tau dQ at the end.
//
// Warp 0 TMA, warp 1 TMEM allocation and MMA issue, then four elementwise
// warpgroups that take 32 columns of every tile each (two of 64 columns left the
// schedulers idle 60% of the time, waiting on latencies).
// SMALL (d = 64, few keys): tiles of 64 keys, two warpgroups, half of an SM's
// TMEM and shared memory, so that two blocks fill and drain beside each other.
// S has two buffers, and dS (bf16) of a tile lies on the scores it came from,
// so S(t + 1) is issued right behind dQ(t - 1); dP has one, handed back as soon
// as it is in registers.  So the score products of tile t + 1 run while the
// warpgroups work on tile t.  Hand-offs are few, because a wait costs a hundred
// cycles or more even when the phase has completed.  Per 128 x 128 tile the
// tensor pipe needs (tcgen05 issue costs) 868 cycles at d = 64 and 1536 at
// d = 128.
// K and V have rings of their own: a V tile is free after dP, a K tile only
// after dQ.
// The launch starts when every block of dK and dV runs, so its blocks fill the SMs
// that their last wave leaves.  It reads nothing that the call's other launches
// write, D is formed here from O and dO (a row's 256 to 512 bytes, beside the first
// tiles' loads); its last block outlasts dK and dV, so whatever follows on the
// stream finds all done.
// TMEM (BN keys a tile): S [0, BN) and [BN, 2 BN), dP [2 BN, 3 BN), dQ from 3 BN
// on; in the large blocks of d = 64 also Q and dO as A operands ([448,480) and
// [480,512)): read from shared memory, they and the key tiles and the TMA writes
// need as many cycles of its 128 bytes as the MMAs take.
// dS is rounded to bf16, K, the MMA's other operand, being bf16: the dQ of normal
// inputs is off by 1.7e-3 in norm for it, as much again for its own rounding, and
// 0.7e-3 for D, which is formed from the O that the call gets, rounded to bf16 (2.4
// to 2.7e-3 in all; more where a row sees few keys and dP - D cancels).  Two bf16
// parts of dS would add half of the MMAs.
// Measured (B1 H8 N16384, no mask): 649 us at d = 64, 1270 TFLOP/s of its 6 N^2 d,
// bound by the chain of waits and arithmetic of a tile (when it took 640, without
// arithmetic 436, with a quarter of the MMAs 650); 893 us at d = 128, 1847 TFLOP/s,
// bound by the MMAs.
#include "tc_attn.cuh"

namespace flashbob {
namespace {
using namespace tc;
using namespace attn;

constexpr int BM = kTcRows;
constexpr int CW = 32, NC = CW / 32;    // columns of a warpgroup, in chunks of 32
constexpr uint32_t HALF = BM * 64 * 2;  // 128 rows x 64 columns

template <int DH, bool SMALL>
struct Cfg {
  static constexpr int BN = SMALL ? 64 : 128, NWG = BN / CW;
  static constexpr int kThreads = 64 + 128 * NWG;
  static constexpr uint32_t kTileHalf = BN * 64 * 2;  // 64 columns of a key tile
  static constexpr uint32_t kP = 2 * BN, kAcc = 3 * BN, kQA = 448, kGA = 480;
  static constexpr int kColumns = SMALL ? 256 : 512;
  static constexpr bool kTmemA = DH == 64 && !SMALL;  // Q and dO as operands in TMEM
  static __device__ __forceinline__ constexpr uint32_t s_col(int t) { return BN * (t & 1); }
  // K step c (16 keys) of tile t's dS operand, on the scores of the warpgroup
  // that wrote it.
  static __device__ __forceinline__ constexpr uint32_t op_col(int t, int c) {
    return s_col(t) + CW * (c / (CW / 16)) + 8 * (c % (CW / 16));
  }
  static_assert(kAcc + DH <= (kTmemA ? kQA : kColumns), "TMEM columns");
};

template <int DH, bool SMALL>
struct SmemQ {
  static constexpr int NH = DH / 64;
  static constexpr int NK = SMALL ? 4 : DH == 64 ? 6 : 3, NV = SMALL ? 4 : DH == 64 ? 5 : 2;
  static constexpr uint32_t kTileHalf = Cfg<DH, SMALL>::kTileHalf;
  alignas(1024) uint8_t q[NH][HALF];
  alignas(1024) uint8_t go[NH][HALF];  // dO
  alignas(1024) uint8_t k[NK][NH][kTileHalf];
  alignas(1024) uint8_t v[NV][NH][kTileHalf];
  int hull[4][4];
  float dd[BM];               // D
  uint64_t bar_q, a_ready;    // Q and dO in shared memory / in TMEM (8 warps)
  uint64_t k_full[NK], k_empty[NK];
  uint64_t v_full[NV], v_empty[NV];
  uint64_t s_full[2];         // S of a tile is complete
  uint64_t p_full, p_free;    // dP of a tile is complete / read
  uint64_t op_ready[2];       // dS written
  uint64_t out_full;
  uint32_t tmem_base;
  int abort_flag;
};

// dS of 32 columns as bf16 pairs from the raw products (capped: their tanh) s
// and dP x.  One pass
// over both, so that the exponentials (MUFU) of some columns run beside the
// multiplications of others.
template <bool CAP, bool BIAS, bool MASKED>
__device__ __forceinline__ void grads(const Score<CAP, BIAS>& sc, const uint32_t (&s)[2][16],
                                      const uint32_t (&x)[2][16], int jbase, int lo, int hi,
                                      float dist, float l2, float dd, uint32_t (&o)[2][8]) {
  const float2 nd = make_float2(-dd, -dd);
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 z = f2(s[q][e], s[q][e + 1]);
      const float2 t = sc.from(z, dist + (16 * q + e), l2, sc.slope2);
      const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
      float2 ds = fmul2(p, sc.damp(fadd2(f2(x[q][e], x[q][e + 1]), nd), z));
      if (MASKED) {  // S and dP of a hidden key may be NaN
        const int j = jbase + 16 * q + e;
        if (j < lo || j >= hi) ds.x = 0.f;
        if (j + 1 < lo || j + 1 >= hi) ds.y = 0.f;
      }
      o[q][e >> 1] = pack_bf16x2(ds.x, ds.y);
    }
}

// The same in two steps: P (1 - tanh^2) of 32 columns in place of the raw
// scores, then dS.
template <bool CAP, bool BIAS, bool MASKED>
__device__ __forceinline__ void weights(const Score<CAP, BIAS>& sc, uint32_t (&s)[2][16], int jbase,
                                        int lo, int hi, float dist, float l2) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 z = f2(s[q][e], s[q][e + 1]);
      const float2 t = sc.from(z, dist + (16 * q + e), l2, sc.slope2);
      float2 p = sc.damp(make_float2(ex2_approx(t.x), ex2_approx(t.y)), z);
      if (MASKED) {
        const int j = jbase + 16 * q + e;
        if (j < lo || j >= hi) p.x = 0.f;
        if (j + 1 < lo || j + 1 >= hi) p.y = 0.f;
      }
      s[q][e] = __float_as_uint(p.x);
      s[q][e + 1] = __float_as_uint(p.y);
    }
}
template <bool MASKED>
__device__ __forceinline__ void finish(const uint32_t (&s)[2][16], const uint32_t (&x)[2][16],
                                       int jbase, int lo, int hi, float dd, uint32_t (&o)[2][8]) {
  const float2 nd = make_float2(-dd, -dd);
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float2 ds = fmul2(f2(s[q][e], s[q][e + 1]), fadd2(f2(x[q][e], x[q][e + 1]), nd));
      if (MASKED) {
        const int j = jbase + 16 * q + e;
        if (j < lo || j >= hi) ds.x = 0.f;
        if (j + 1 < lo || j + 1 >= hi) ds.y = 0.f;
      }
      o[q][e >> 1] = pack_bf16x2(ds.x, ds.y);
    }
}

template <int DH, bool SMALL, bool CAP, bool BIAS>
__global__ void __launch_bounds__((Cfg<DH, SMALL>::kThreads), (SMALL ? 2 : 1))
    tc_dq_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mdO,
                 const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                 const __grid_constant__ AttnArgs a, int blocks) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = SmemQ<DH, SMALL>;
  using C = Cfg<DH, SMALL>;
  constexpr int BN = C::BN, NWG = C::NWG;
  constexpr uint32_t TILE = C::kTileHalf;
  constexpr int NH = Smem::NH, NK = Smem::NK, NV = Smem::NV;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.B * a.Hkv, G = a.H / a.Hkv, rows = G * a.Nq;
  const int g = blockIdx.x % heads;
  const int row0 = row_block(blockIdx.x / heads, blocks, G, a.Nq, BM) * BM;
  volatile int* abort_flag = &sm.abort_flag;
  unsigned int* err = a.err;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_q, 1);
    mbar_init(&sm.a_ready, 8);
    for (int s = 0; s < NK; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < NV; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], 1);
    mbar_init(&sm.p_full, 1);
    mbar_init(&sm.p_free, 4 * NWG);
    for (int b = 0; b < 2; ++b) mbar_init(&sm.s_full[b], 1), mbar_init(&sm.op_ready[b], 4 * NWG);
    mbar_init(&sm.out_full, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    // Q and dO are under way while the ranges and the row state are read.
    mbar_expect_tx(&sm.bar_q, 2 * NH * HALF);
    for (int h = 0; h < NH; ++h) {
      tma_load_3d(sm.q[h], &mQ, &sm.bar_q, 64 * h, row0, g);
      tma_load_3d(sm.go[h], &mdO, &sm.bar_q, 64 * h, row0, g);
    }
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, C::kColumns);
  const int wg = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane, row = row0 + r;
  GroupRow gr{empty_view(), 0.f};
  float l2 = INFINITY, dd = 0.f;
  if (warp >= 2) {
    gr = group_row(a, g / a.Hkv, g % a.Hkv, row, rows);
    if (wg == 0) warp_hull(gr.v, row < rows, lane, sm.hull[quad]);
    // D of 16 NWG rows at a time, eight lanes a row.
    constexpr int kPer = BM / (16 * NWG);
    const size_t base = static_cast<size_t>(g) * rows + row0;
    const auto* o = static_cast<const __nv_bfloat16*>(a.O) + base * DH;
    const auto* go = static_cast<const __nv_bfloat16*>(a.dO) + base * DH;
    const int first = (threadIdx.x - 64) >> 3;
    float dots[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int q = first + 16 * NWG * u;
      dots[u] = 0.f;
      if (row0 + q < rows)
        dots[u] = dot_part<__nv_bfloat16, DH>(o + static_cast<size_t>(q) * DH,
                                              go + static_cast<size_t>(q) * DH, DH, lane & 7);
    }
    if (gr.v.hi > 0) l2 = a.L[base + r] * kLog2e;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const float dot = sum8(dots[u]);
      if ((lane & 7) == 0) sm.dd[first + 16 * NWG * u] = dot;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  if (warp >= 2 && gr.v.hi > 0) dd = sm.dd[r];  // else the row may hold anything
  const Hull hull = join_hulls(sm.hull, 4);
  const int tb = hull.lo < hull.hi ? hull.lo / BN : 0;
  const int T = hull.lo < hull.hi ? (hull.hi + BN - 1) / BN - tb : 0;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&mK);
      tma_prefetch_desc(&mV);
      int nk = 0, nv = 0;
      for (int t = 0; t < T; ++t) {
        const int sk = t % NK, sv = t % NV;
        if (t >= NK && !wait_one(&sm.k_empty[sk], ((t / NK) - 1) & 1, abort_flag, err)) break;
        mbar_expect_tx(&sm.k_full[sk], NH * TILE);
        for (int h = 0; h < NH; ++h)
          tma_load_3d(sm.k[sk][h], &mK, &sm.k_full[sk], 64 * h, (tb + t) * BN, g);
        nk = t + 1;
        if (t >= NV && !wait_one(&sm.v_empty[sv], ((t / NV) - 1) & 1, abort_flag, err)) break;
        mbar_expect_tx(&sm.v_full[sv], NH * TILE);
        for (int h = 0; h < NH; ++h)
          tma_load_3d(sm.v[sv][h], &mV, &sm.v_full[sv], 64 * h, (tb + t) * BN, g);
        nv = t + 1;
      }
      drain_wait(&sm.bar_q, 0);
      for (int t = nk > NK ? nk - NK : 0; t < nk; ++t) drain_wait(&sm.k_full[t % NK], (t / NK) & 1);
      for (int t = nv > NV ? nv - NV : 0; t < nv; ++t) drain_wait(&sm.v_full[t % NV], (t / NV) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = idesc_bf16(BM, BN, false);
    constexpr uint32_t idO = idesc_bf16(BM, DH, true);
    const uint64_t dQ = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
    const uint64_t dG = smem_desc_sw128(smem_u32(sm.go[0]), 16, 1024);
    const uint64_t dK = smem_desc_sw128(smem_u32(sm.k[0][0]), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(sm.v[0][0]), 16, 1024);
    const uint64_t dKm = smem_desc_sw128(smem_u32(sm.k[0][0]), TILE, 1024);  // MN-major
    constexpr uint64_t kTile = (uint64_t)(NH * TILE) >> 4;
    auto scores = [&](uint32_t col, uint64_t da, uint32_t ta, uint64_t db) {
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint64_t oa = ((kk >> 2) * HALF + 32 * (kk & 3)) >> 4;
        const uint64_t ob = ((kk >> 2) * TILE + 32 * (kk & 3)) >> 4;
        if (C::kTmemA) mma_ts(tbase + col, tbase + ta + 8 * kk, db + ob, idS, kk > 0);
        else mma_ss(tbase + col, da + oa, db + ob, idS, kk > 0);
      }
    };
    if (elect_one()) {
      bool ok = wait_one(C::kTmemA ? &sm.a_ready : &sm.bar_q, 0, abort_flag, err);
      auto issue_s = [&](int t) {
        tc_fence_after();
        scores(C::s_col(t), dQ, C::kQA, dK + (t % NK) * kTile);
        mma_commit(&sm.s_full[t & 1]);
      };
      auto issue_p = [&](int t) {
        tc_fence_after();
        scores(C::kP, dG, C::kGA, dV + (t % NV) * kTile);
        mma_commit(&sm.p_full);
        mma_commit(&sm.v_empty[t % NV]);
      };
      if (ok && T > 0) {
        ok = wait_one(&sm.k_full[0], 0, abort_flag, err) &&
             wait_one(&sm.v_full[0], 0, abort_flag, err);
        if (ok) {
          issue_s(0);
          issue_p(0);
        }
      }
      for (int t = 0; ok && t < T; ++t) {
        if (t + 1 < T) {
          // Tile t - 1's dS, which lies on this buffer, was waited for and its
          // dQ issued: the pipe runs in order.
          const int n = t + 1;
          ok = wait_one(&sm.k_full[n % NK], (n / NK) & 1, abort_flag, err);
          if (!ok) break;
          issue_s(n);
          ok = wait_one(&sm.v_full[n % NV], (n / NV) & 1, abort_flag, err) &&
               wait_one(&sm.p_free, t & 1, abort_flag, err);
          if (!ok) break;
          issue_p(n);
        }
        ok = wait_one(&sm.op_ready[t & 1], (t >> 1) & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dk = dKm + (t % NK) * kTile;
#pragma unroll
        for (int c = 0; c < BN / 16; ++c)
          mma_ts(tbase + C::kAcc, tbase + C::op_col(t, c), dk + ((16 * 128 * c) >> 4), idO,
                 t > 0 || c > 0);
        mma_commit(&sm.k_empty[t % NK]);
      }
      mma_commit(&sm.out_full);
    }
    __syncwarp();
  } else {
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int lo = gr.v.lo, hi = gr.v.hi;
    const Score<CAP, BIAS> score(a, gr.slope2);
    bool ok = true;
    if (C::kTmemA && wg < 2) {
      ok = wait_warp(&sm.bar_q, 0, abort_flag, err);
      row_to_tmem(wg ? sm.go[0] : sm.q[0], r, tbase + lane_off + (wg ? C::kGA : C::kQA));
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&sm.a_ready);
    }
    uint32_t s[NC][2][16], x[2][16], pk[2][8];
    auto col_of = [&](int t, int c) { return (tb + t) * BN + CW * wg + 32 * c; };
    auto masked_at = [&](int t) {
      return col_of(t, 0) < hull.in_lo || col_of(t, NC) > hull.in_hi;
    };
    auto dist_at = [&](int t, int c) {
      return BIAS ? static_cast<float>(col_of(t, c) - gr.v.pos) : 0.f;
    };
    auto load = [&](uint32_t col, int c, uint32_t (&d)[2][16]) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        tmem_ld16(tbase + lane_off + col + CW * wg + 32 * c + 16 * q, d[q]);
    };
    auto write = [&](int t, int c) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        tmem_st8(tbase + lane_off + C::op_col(t, (CW / 16) * wg + 2 * c + q), pk[q]);
    };
    auto written = [&](int t) {
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&sm.op_ready[t & 1]);
    };
    if (wg < NWG / 2) {
      // S and dP of a tile together.
      for (int t = 0; t < T; ++t) {
        ok = wait_both_warp(&sm.s_full[t & 1], (t >> 1) & 1, &sm.p_full, t & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; ++c) load(C::s_col(t), c, s[c]);
        const bool masked = masked_at(t);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          load(C::kP, c, x);
          tmem_wait_ld();
          if (c == NC - 1) {
            tc_fence_before();
            warp_arrive(&sm.p_free);
          }
          score.tanh_of(s[c], masked);
          if (masked)
            grads<CAP, BIAS, true>(score, s[c], x, col_of(t, c), lo, hi, dist_at(t, c), l2, dd, pk);
          else
            grads<CAP, BIAS, false>(score, s[c], x, col_of(t, c), lo, hi, dist_at(t, c), l2, dd,
                                    pk);
          write(t, c);
        }
        const int tile0 = (tb + t) * BN;
        if (tile0 < hull.lo || tile0 + BN > hull.hi) {
          // K rows that no row of the block sees meet dS = 0: make them 0 too.
          if (wg == 0 && r < BN && (tile0 + r < hull.lo || tile0 + r >= hull.hi))
            zero_row<NH, TILE>(sm.k[t % NK], r);
          fence_proxy_async_smem();
        }
        written(t);
      }
    } else {
      // Half a tile ahead: the weights of tile t + 1 are formed behind dS of
      // tile t.  So on every scheduler half of the warps use the MUFU pipe
      // while the others load, multiply and store.
      auto ahead = [&](int t) {
        ok = wait_warp(&sm.s_full[t & 1], (t >> 1) & 1, abort_flag, err);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; ++c) load(C::s_col(t), c, s[c]);
        tmem_wait_ld();
        const bool masked = masked_at(t);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          score.tanh_of(s[c], masked);
          if (masked)
            weights<CAP, BIAS, true>(score, s[c], col_of(t, c), lo, hi, dist_at(t, c), l2);
          else
            weights<CAP, BIAS, false>(score, s[c], col_of(t, c), lo, hi, dist_at(t, c), l2);
        }
      };
      if (T > 0) ahead(0);
      for (int t = 0; ok && t < T; ++t) {
        ok = wait_warp(&sm.p_full, t & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        const bool masked = masked_at(t);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          load(C::kP, c, x);
          tmem_wait_ld();
          if (c == NC - 1) {
            tc_fence_before();
            warp_arrive(&sm.p_free);
          }
          if (masked) finish<true>(s[c], x, col_of(t, c), lo, hi, dd, pk);
          else finish<false>(s[c], x, col_of(t, c), lo, hi, dd, pk);
          write(t, c);
        }
        written(t);
        if (t + 1 < T) ahead(t + 1);
      }
    }
    ok = wait_warp(&sm.out_full, 0, abort_flag, err) && ok;
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    tc_fence_after();
    static_assert(BM * (DH * 2 + 16) <= sizeof(sm.k), "epilogue staging fits in the ring");
    store_block<DH, NWG>(tbase + lane_off + C::kAcc, a.tau, T == 0, &sm.k[0][0][0], wg, r,
                         threadIdx.x - 64, min(BM, rows - row0), ok,
                         static_cast<__nv_bfloat16*>(a.dQ) +
                             (static_cast<size_t>(g) * rows + row0) * DH);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, C::kColumns);
  }
  if (blockIdx.x + 1 == gridDim.x) wait_ahead();
}

template <int DH, bool SMALL, bool CAP, bool BIAS>
cudaError_t launch(const AttnArgs& a) {
  const int heads = a.B * a.Hkv, rows = a.H / a.Hkv * a.Nq;
  using C = Cfg<DH, SMALL>;
  CUtensorMap mq, mo, mk, mv;
  cudaError_t e = tc_map_bf16(&mq, a.Q, heads, rows, BM, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mo, a.dO, heads, rows, BM, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mk, a.K, heads, a.Nk, C::BN, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mv, a.V, heads, a.Nk, C::BN, DH);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(SmemQ<DH, SMALL>) + 1024;
  static_assert(smem <= (SMALL ? 115712 : 232448), "shared memory");
  const auto kernel = tc_dq_kernel<DH, SMALL, CAP, BIAS>;
  e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int blocks = (rows + BM - 1) / BM;
  const long long grid = static_cast<long long>(blocks) * heads;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_after(true, kernel, dim3(static_cast<unsigned>(grid)), C::kThreads, smem, 1,
                      a.stream, mq, mo, mk, mv, a, blocks);
}

template <int DH, bool SMALL>
cudaError_t launch(const AttnArgs& a) {
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  return cap ? (bias ? launch<DH, SMALL, true, true>(a) : launch<DH, SMALL, true, false>(a))
             : (bias ? launch<DH, SMALL, false, true>(a) : launch<DH, SMALL, false, false>(a));
}

}  // namespace

// Small blocks up to 2048 keys (the gradient of B4 H12 d64: N1024 causal 61 -> 54
// us, without a mask 75 -> 73; B2 H12 N2048 causal 75 -> 71, without 112 either
// way).
cudaError_t tc_attn_dq(const AttnArgs& a) {
  if (a.d == 128) return launch<128, false>(a);
  return a.Nk <= 2048 ? launch<64, true>(a) : launch<64, false>(a);
}

}  // namespace flashbob
