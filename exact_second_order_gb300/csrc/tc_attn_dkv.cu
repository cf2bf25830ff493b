// dK and dV of attention with key ranges on sm_103a tensor cores: bf16, head
// dim 64 or 128.  128 keys (K, V) stay on chip; the tiles of 128 group rows
// that see any of them stream past, all heads that share the keys in one run,
// so that the sums over rows and heads stay on chip:
//   S^T = K Q^T, dP^T = V dO^T;  P = exp2(score(S) - L log2 e),
//   dS = P (dP - D) (1 - tanh^2),  dV += P^T dO,  dK += dS^T Q (times tau).
//
// 576 threads: warp 0 finds the tiles (the bounds of 32 at a time against the
// block's keys) and loads them with their row state; warp 1 allocates TMEM
// and issues the MMAs; then come four elementwise warpgroups that take 32 rows
// of every tile each, one key per thread.  How many tiles there
// are is known only to warp 0: each ring slot says which tile it holds, and a
// last slot says that there are no more.
// The launch starts beside the row state's, loads K and V, and waits for the row
// state before warp 0 reads any of it.
// When the key blocks are few, a cluster of S blocks shares one: rank q takes
// every S-th of its tiles, and the partial sums meet in distributed shared
// memory, in the order of the ranks, before the one write.
// TMEM at d = 64: S^T, dP^T (128 columns each), operands P^T and dS^T (64
// each), dK, dV (64 each): the scores are handed back when they are in
// registers, and those of tile n + 1 run beside the arithmetic of tile n.
// At d = 64 the row scalars ride in the score products: one more K step of an
// A operand of ones against the rows' -L / tau and -D leaves S^T - L / tau (for
// capped scores S^T) and dP^T - D in TMEM.  Read from shared memory instead,
// 32 values of each for every warp and tile, they cost 350 of 1150 us (8
// heads, 16384 rows); at d = 128, where the operands' own traffic bounds the
// kernel, nothing, so there they are read.
// At d = 128 dK and dV take 256 columns: one buffer of each, P^T on S^T and
// dS^T on dP^T; the pipe runs dV(n), S(n + 1), dK(n), dP(n + 1), so that
// P(n + 1) is formed beside dK(n) and dP(n + 1), and dS beside dV and S.
// P^T and dS^T are rounded to bf16, as operands beside the bf16 dO and Q (tc_attn_dq.cu
// has the errors).
// Measured (B1 H8 N16384, no mask): 840 us at d = 64, 1309 TFLOP/s of its 8 N^2 d,
// and 1460 us at d = 128, 1506 TFLOP/s; waits and arithmetic of a tile bound both.
#include <stddef.h>

#include <type_traits>

#include "tc_attn.cuh"

namespace flashbob {
namespace {
using namespace tc;
using namespace attn;

constexpr int BM = kTcRows, BQ = 128;
constexpr int NWG = 4, CW = BQ / NWG, NC = CW / 32;  // warpgroups; rows of each, in chunks of 32
constexpr int NTHREADS = 64 + 128 * NWG;
constexpr uint32_t HALF = BM * 64 * 2;  // 128 rows x 64 columns

template <int DH>
struct Cols {
  static constexpr bool kOwn = DH == 64;  // the operands have columns of their own
  static constexpr uint32_t S = 0, dP = 128, dK = kOwn ? 384 : 256, dV = dK + DH;
  // Operand K step kk (16 rows): in its own area, or on the scores of the
  // warpgroup that wrote it.
  static __device__ __forceinline__ constexpr uint32_t p(int kk) {
    return kOwn ? 256 + 8 * kk : S + CW * (kk / (CW / 16)) + 8 * (kk % (CW / 16));
  }
  static __device__ __forceinline__ constexpr uint32_t ds(int kk) {
    return kOwn ? 320 + 8 * kk : dP + CW * (kk / (CW / 16)) + 8 * (kk % (CW / 16));
  }
  static_assert(dV + DH <= 512, "TMEM columns");
};

struct Slot {
  int tile;          // -1: no more
  int in_lo, in_hi;  // intersection of the rows' ranges (in_lo INT_MAX: a row sees nothing)
  int line, pos;     // line: row i is at position pos + i, and all have one slope
  float slope2;
};

// Cluster split: floats of a staged row dK | dV (padded by 4 against conflicts).
template <int DH>
constexpr int kPartLd = 2 * DH + 4;

template <int DH>
struct SmemK {
  static constexpr int NH = DH / 64;
  static constexpr bool kFold = DH == 64;  // row scalars in the score products
  static constexpr int NST = DH == 64 ? 4 : 2;
  alignas(1024) uint8_t k[NH][HALF];
  alignas(1024) uint8_t v[NH][HALF];
  alignas(1024) uint8_t q[NST][NH][HALF];
  alignas(1024) uint8_t go[NST][NH][HALF];  // dO
  alignas(1024) uint8_t ex[kFold ? NST : 1][kFold ? BQ * kExRow : 16];
  alignas(128) uint8_t ones[kFold ? 2 : 1][kFold ? BM * kExRow : 16];  // of L and of D
  alignas(16) float l2[NST][BQ];
  alignas(16) float dd[NST][BQ];
  alignas(16) int4 info[NST][BQ];
  Slot slot[NST];
  uint64_t bar_kv;
  uint64_t q_full[NST], q_empty[NST];  // Q, the row state and the slot
  uint64_t o_full[NST], o_empty[NST];  // dO
  uint64_t s_full, s_free;  // S^T of a tile is complete / d = 64: read
  uint64_t p_full, p_free;  // the same for dP^T
  uint64_t w_ready;         // d = 128: P^T written
  uint64_t ds_ready;        // dS^T (d = 64: and P^T) written
  uint64_t op_free;         // d = 64: both read by dV and dK
  uint64_t out_full;
  uint32_t tmem_base;
  int abort_flag;
};

// t minus the distance bias of rows i and i + 1.  LINE: row i is `dist` - i keys
// away and the rows have the score's slope; else each row's position and slope
// are read (one 16-byte shared load an element for every warp).
template <bool LINE, bool CAP>
__device__ __forceinline__ float2 less_bias(float2 t, const Score<CAP, true>& score,
                                            const int4* info, int key, float dist, int i) {
  if (LINE) {
    t.x = fmaf(-score.slope2, fabsf(dist - i), t.x);
    t.y = fmaf(-score.slope2, fabsf(dist - (i + 1)), t.y);
  } else {
    const int4 a = info[i], b = info[i + 1];
    t.x = fmaf(-__int_as_float(a.w), fabsf(static_cast<float>(key - a.z)), t.x);
    t.y = fmaf(-__int_as_float(b.w), fabsf(static_cast<float>(key - b.z)), t.y);
  }
  return t;
}
template <bool LINE, bool CAP>
__device__ __forceinline__ float2 less_bias(float2 t, const Score<CAP, false>&, const int4*, int,
                                            float, int) {
  return t;
}

// 32 rows of one key: P as bf16 pairs, and P (1 - tanh^2) in place of the
// raw scores.
template <bool MASKED, bool LINE, bool CAP, bool BIAS>
__device__ __forceinline__ void weights(const Score<CAP, BIAS>& score, uint32_t (&s)[2][16],
                                        const float* l2s, const int4* info, int key, float dist,
                                        uint32_t seen, uint32_t (&pk)[2][8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 l2 = *reinterpret_cast<const float4*>(l2s + 16 * q + e);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const int i = 16 * q + e + k;
        const float2 x = f2(s[q][e + k], s[q][e + k + 1]);
        const float2 nl = k == 0 ? make_float2(-l2.x, -l2.y) : make_float2(-l2.z, -l2.w);
        const float c = CAP ? score.c2 : score.c1;
        const float2 t =
            less_bias<LINE>(ffma2(x, make_float2(c, c), nl), score, info, key, dist, i);
        float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        if (MASKED) {
          if (!(seen >> i & 1)) p.x = 0.f;
          if (!(seen >> (i + 1) & 1)) p.y = 0.f;
        }
        pk[q][(e + k) >> 1] = pack_bf16x2(p.x, p.y);
        p = score.damp(p, x);
        s[q][e + k] = __float_as_uint(p.x);
        s[q][e + k + 1] = __float_as_uint(p.y);
      }
    }
}

// P and dS of 32 rows of one key in one pass, so that the exponentials (MUFU)
// of some rows run beside the multiplications of others.  s holds S^T - L / tau
// (capped: the tanh), x holds dP^T - D.
template <bool MASKED, bool LINE, bool CAP, bool BIAS>
__device__ __forceinline__ void both(const Score<CAP, BIAS>& score, const uint32_t (&s)[2][16],
                                     const uint32_t (&x)[2][16], const float* l2s,
                                     const int4* info, int key, float dist, uint32_t seen,
                                     uint32_t (&pk)[2][8], uint32_t (&o)[2][8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float4 l2 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (CAP) l2 = *reinterpret_cast<const float4*>(l2s + 16 * q + e);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const int i = 16 * q + e + k;
        const float2 z = f2(s[q][e + k], s[q][e + k + 1]);
        float2 t;
        if (CAP) {
          const float2 nl = k == 0 ? make_float2(-l2.x, -l2.y) : make_float2(-l2.z, -l2.w);
          t = ffma2(z, make_float2(score.c2, score.c2), nl);
        } else {
          t = fmul2(z, make_float2(score.c1, score.c1));
        }
        t = less_bias<LINE>(t, score, info, key, dist, i);
        float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        float2 ds = fmul2(p, score.damp(f2(x[q][e + k], x[q][e + k + 1]), z));
        if (MASKED) {  // S and dP of a row that sees nothing may be NaN
          if (!(seen >> i & 1)) p.x = ds.x = 0.f;
          if (!(seen >> (i + 1) & 1)) p.y = ds.y = 0.f;
        }
        pk[q][(e + k) >> 1] = pack_bf16x2(p.x, p.y);
        o[q][(e + k) >> 1] = pack_bf16x2(ds.x, ds.y);
      }
    }
}

// dS = P (dP - D) of 32 rows of one key as bf16 pairs.
template <bool MASKED>
__device__ __forceinline__ void grads(const uint32_t (&p)[2][16], const uint32_t (&x)[2][16],
                                      const float* dds, uint32_t seen, uint32_t (&o)[2][8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 dd = *reinterpret_cast<const float4*>(dds + 16 * q + e);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const int i = 16 * q + e + k;
        const float2 nd = k == 0 ? make_float2(-dd.x, -dd.y) : make_float2(-dd.z, -dd.w);
        float2 ds = fmul2(f2(p[q][e + k], p[q][e + k + 1]),
                          fadd2(f2(x[q][e + k], x[q][e + k + 1]), nd));
        if (MASKED) {  // dP of a row that sees nothing may be NaN
          if (!(seen >> i & 1)) ds.x = 0.f;
          if (!(seen >> (i + 1) & 1)) ds.y = 0.f;
        }
        o[q][(e + k) >> 1] = pack_bf16x2(ds.x, ds.y);
      }
    }
}

// f with the two conditions as constants (BIAS false: the second is false).
template <bool BIAS, typename F>
__device__ __forceinline__ void choose(bool masked, bool line, F&& f) {
  if (BIAS && line) {
    if (masked) f(std::true_type(), std::true_type());
    else f(std::false_type(), std::true_type());
  } else {
    if (masked) f(std::true_type(), std::false_type());
    else f(std::false_type(), std::false_type());
  }
}

template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(NTHREADS, 1)
    tc_dkv_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mdO,
                  const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                  const __grid_constant__ AttnArgs a, int S) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = SmemK<DH>;
  using C = Cols<DH>;
  constexpr int NH = Smem::NH, NST = Smem::NST;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.B * a.Hkv, rows = a.H / a.Hkv * a.Nq;
  const int rank = blockIdx.x % S, g = blockIdx.x / S % heads;
  const int j0 = static_cast<int>(blockIdx.x / S / heads) * BM;
  volatile int* abort_flag = &sm.abort_flag;
  unsigned int* err = a.err;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_kv, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.o_full[s], 1);
      mbar_init(&sm.o_empty[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, 1);
    mbar_init(&sm.op_free, 1);
    mbar_init(&sm.s_free, 4 * NWG);
    mbar_init(&sm.p_free, 4 * NWG);
    mbar_init(&sm.w_ready, 4 * NWG);
    mbar_init(&sm.ds_ready, 4 * NWG);
    mbar_init(&sm.out_full, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    // K and V are under way while the row state is waited for.
    mbar_expect_tx(&sm.bar_kv, 2 * NH * HALF);
    for (int h = 0; h < NH; ++h) {
      tma_load_3d(sm.k[h], &mK, &sm.bar_kv, 64 * h, j0, g);
      tma_load_3d(sm.v[h], &mV, &sm.bar_kv, 64 * h, j0, g);
    }
    release_next();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
  if (Smem::kFold && threadIdx.x >= 64 && threadIdx.x < 64 + 2 * BM) {
    // Ones in columns 0 - 2 (L) and 3 - 5 (D) of 16, one row a thread.
    const int k = (threadIdx.x - 64) / BM, r = (threadIdx.x - 64) % BM;
    const uint32_t one = 0x3F80u;  // bf16 1.0
    uint8_t* row = sm.ones[k] + (r >> 3) * 256 + (r & 7) * 16;
    *reinterpret_cast<uint4*>(row) = k == 0 ? make_uint4(one | (one << 16), one, 0u, 0u)
                                            : make_uint4(0u, one << 16, one | (one << 16), 0u);
    *reinterpret_cast<uint4*>(row + 128) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;

  if (warp == 0) {
    const GradRows st = grad_rows(a.workspace, heads, rows);
    const size_t base = static_cast<size_t>(g) * st.pitch;
    const int4 *bounds = st.bounds + base / kBoundRows, *lines = st.lines + base / kBoundRows;
    const int tiles = st.pitch / BQ;
    if (lane == 0) {
      tma_prefetch_desc(&mQ);
      tma_prefetch_desc(&mdO);
    }
    wait_ahead();                // the row state is written and visible,
    fence_proxy_async_global();  // to the bulk copies as well
    int nq = 0, no = 0;  // Q and dO loads issued
    int hit = 0;         // tiles found
    bool ok = true;
    for (int t0 = 0; ok && t0 < tiles; t0 += 32) {
      int4 b = make_int4(INT_MAX, 0, 0, INT_MAX), line = make_int4(0, 0, 0, 0);
      if (t0 + lane < tiles) {
        const int4 x = __ldcg(bounds + 2 * (t0 + lane)), y = __ldcg(bounds + 2 * (t0 + lane) + 1);
        b = make_int4(min(x.x, y.x), max(x.y, y.y), max(x.z, y.z), min(x.w, y.w));
        if (BIAS) {
          line = __ldcg(lines + 2 * (t0 + lane));
          const int4 z = __ldcg(lines + 2 * (t0 + lane) + 1);
          if (z.x != 2 && (z.x != 1 || z.z != line.z ||
                           static_cast<unsigned>(z.y) !=
                               static_cast<unsigned>(line.y) + static_cast<unsigned>(kBoundRows)))
            line.x = 0;
        }
      }
      unsigned hits = __ballot_sync(0xffffffffu, b.x < j0 + BM && b.y > j0);
      for (; ok && hits; hits &= hits - 1) {
        if (hit++ % S != rank) continue;
        const int k = __ffs(hits) - 1, tile = t0 + k, s = nq % NST;
        const int in_lo = __shfl_sync(0xffffffffu, b.z, k);
        const int in_hi = __shfl_sync(0xffffffffu, b.w, k);
        const int kind = BIAS ? __shfl_sync(0xffffffffu, line.x, k) : 0;
        const int pos = BIAS ? __shfl_sync(0xffffffffu, line.y, k) : 0;
        const int slope = BIAS ? __shfl_sync(0xffffffffu, line.z, k) : 0;
        if (nq >= NST) ok = wait_warp(&sm.q_empty[s], ((nq / NST) - 1) & 1, abort_flag, err);
        if (!ok) break;
        if (lane == 0) {
          sm.slot[s] = Slot{tile, in_lo, in_hi, kind, pos, __int_as_float(slope)};
          constexpr bool kL2 = !Smem::kFold || CAP;  // L is read by the warpgroups
          mbar_expect_tx(&sm.q_full[s], NH * HALF + BQ * 16 + (kL2 ? BQ * 4 : 0) +
                                            (Smem::kFold ? BQ * kExRow : BQ * 4));
          for (int h = 0; h < NH; ++h)
            tma_load_3d(sm.q[s][h], &mQ, &sm.q_full[s], 64 * h, tile * BQ, g);
          const size_t at = base + static_cast<size_t>(tile) * BQ;
          if (kL2) bulk_load(sm.l2[s], st.l2 + at, BQ * 4, &sm.q_full[s]);
          if (Smem::kFold) bulk_load(sm.ex[s], st.ex + at * kExRow, BQ * kExRow, &sm.q_full[s]);
          else bulk_load(sm.dd[s], st.dd + at, BQ * 4, &sm.q_full[s]);
          bulk_load(sm.info[s], st.info + at, BQ * 16, &sm.q_full[s]);
        }
        ++nq;
        if (no >= NST) ok = wait_warp(&sm.o_empty[s], ((no / NST) - 1) & 1, abort_flag, err);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(&sm.o_full[s], NH * HALF);
          for (int h = 0; h < NH; ++h)
            tma_load_3d(sm.go[s][h], &mdO, &sm.o_full[s], 64 * h, tile * BQ, g);
        }
        ++no;
      }
    }
    if (lane == 0) {
      // No copy may still be in flight when the block exits; then the slot
      // that ends the run (waited for before, so no phase is reused).
      drain_wait(&sm.bar_kv, 0);
      for (int n = nq > NST ? nq - NST : 0; n < nq; ++n)
        drain_wait(&sm.q_full[n % NST], (n / NST) & 1);
      for (int n = no > NST ? no - NST : 0; n < no; ++n)
        drain_wait(&sm.o_full[n % NST], (n / NST) & 1);
      const int s = nq % NST;
      if (ok && (nq < NST || wait_one(&sm.q_empty[s], ((nq / NST) - 1) & 1, abort_flag, err))) {
        sm.slot[s].tile = -1;
        mbar_arrive(&sm.q_full[s]);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idS = idesc_bf16(BM, BQ, false);
    constexpr uint32_t idO = idesc_bf16(BM, DH, true);
    const uint64_t dK = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(sm.v[0]), 16, 1024);
    const uint64_t dQ = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t dG = smem_desc_sw128(smem_u32(sm.go[0][0]), 16, 1024);
    const uint64_t dQm = smem_desc_sw128(smem_u32(sm.q[0][0]), HALF, 1024);  // MN-major
    const uint64_t dGm = smem_desc_sw128(smem_u32(sm.go[0][0]), HALF, 1024);
    constexpr uint64_t kTile = (uint64_t)(NH * HALF) >> 4;
    const uint64_t dOnes = smem_desc_noswz(smem_u32(sm.ones[0]), 128, 256);
    const uint64_t dEx = smem_desc_noswz(smem_u32(sm.ex[0]), 128, 256);
    constexpr uint64_t kEx = (BQ * kExRow) >> 4;
    auto scores = [&](uint32_t col, uint64_t da, uint64_t db) {
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint64_t o = ((kk >> 2) * HALF + 32 * (kk & 3)) >> 4;
        mma_ss(tbase + col, da + o, db + o, idS, kk > 0);
      }
    };
    if (elect_one()) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = wait_one(bar, parity, abort_flag, err);
        tc_fence_after();
        return got;
      };
      auto issue_s = [&](int n) {
        scores(C::S, dK, dQ + (n % NST) * kTile);
        if (Smem::kFold && !CAP) mma_ss(tbase + C::S, dOnes, dEx + (n % NST) * kEx, idS, 1);
        mma_commit(&sm.s_full);
      };
      auto issue_p = [&](int n) {
        scores(C::dP, dV, dG + (n % NST) * kTile);
        if (Smem::kFold) mma_ss(tbase + C::dP, dOnes + kEx, dEx + (n % NST) * kEx, idS, 1);
        mma_commit(&sm.p_full);
      };
      auto issue_dv = [&](int n) {
        const uint64_t b = dGm + (n % NST) * kTile;
#pragma unroll
        for (int c = 0; c < BQ / 16; ++c)
          mma_ts(tbase + C::dV, tbase + C::p(c), b + ((16 * 128 * c) >> 4), idO,
                 n > 0 || c > 0);
        mma_commit(&sm.o_empty[n % NST]);
      };
      auto issue_dk = [&](int n) {
        const uint64_t b = dQm + (n % NST) * kTile;
#pragma unroll
        for (int c = 0; c < BQ / 16; ++c)
          mma_ts(tbase + C::dK, tbase + C::ds(c), b + ((16 * 128 * c) >> 4), idO,
                 n > 0 || c > 0);
        mma_commit(&sm.op_free);
        mma_commit(&sm.q_empty[n % NST]);
      };
      bool ok = wait(&sm.bar_kv, 0) && wait(&sm.q_full[0], 0);
      bool more = ok && sm.slot[0].tile >= 0;
      if (more) {
        issue_s(0);
        ok = wait(&sm.o_full[0], 0);
        if (ok) issue_p(0);
      }
      for (int n = 0; ok && more; ++n) {
        const int s1 = (n + 1) % NST;
        const uint32_t f1 = ((n + 1) / NST) & 1;
        if (C::kOwn) {
          ok = wait(&sm.q_full[s1], f1);
          if (!ok) break;
          more = sm.slot[s1].tile >= 0;
          if (more) {
            ok = wait(&sm.s_free, n & 1);
            if (!ok) break;
            issue_s(n + 1);
            ok = wait(&sm.o_full[s1], f1) && wait(&sm.p_free, n & 1);
            if (!ok) break;
            issue_p(n + 1);
          }
          ok = wait(&sm.ds_ready, n & 1);
          if (!ok) break;
          issue_dv(n);
          issue_dk(n);
        } else {
          ok = wait(&sm.w_ready, n & 1);
          if (!ok) break;
          issue_dv(n);
          ok = wait(&sm.q_full[s1], f1);
          if (!ok) break;
          more = sm.slot[s1].tile >= 0;
          if (more) issue_s(n + 1);  // after dV(n) has read P on S's columns
          ok = wait(&sm.ds_ready, n & 1);
          if (!ok) break;
          issue_dk(n);
          if (more) {
            ok = wait(&sm.o_full[s1], f1);
            if (ok) issue_p(n + 1);
          }
        }
      }
      mma_commit(&sm.out_full);
    }
    __syncwarp();
  } else {
    const int wg = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int key = j0 + r, c0 = CW * wg;
    const int key_end = min(j0 + BM, a.Nk);
    Score<CAP, BIAS> score(a, 0.f);
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      const int st = n % NST;
      ok = wait_warp(&sm.q_full[st], (n / NST) & 1, abort_flag, err);
      if (!ok) break;
      const Slot slot = sm.slot[st];
      if (slot.tile < 0) break;
      // Rows behind the last (zeros) run masked: their P is not 0, a bias may even
      // make it infinite.
      const bool masked = slot.in_lo > j0 || slot.in_hi < key_end || rows - slot.tile * BQ < BQ;
      const bool line = BIAS && slot.line == 1;
      const float dist = static_cast<float>(key - slot.pos) - c0;
      score.slope2 = slot.slope2;
      ok = wait_warp(&sm.s_full, n & 1, abort_flag, err);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[NC][2][16], x[2][16], pk[2][8], gk[2][8];
      auto load = [&](uint32_t col, int c, uint32_t (&d)[2][16]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld16(tbase + lane_off + col + c0 + 32 * c + 16 * q, d[q]);
      };
      const float *l2 = &sm.l2[st][c0], *dd = &sm.dd[st][c0];
      const int4* info = &sm.info[st][c0];
#pragma unroll
      for (int c = 0; c < NC; ++c) load(C::S, c, s[c]);
      tmem_wait_ld();
      if (C::kOwn) {
        tc_fence_before();
        warp_arrive(&sm.s_free);
      }
      uint32_t seen[NC];  // masked tiles: which rows see this key
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        seen[c] = ~0u;
        if (masked) {
          seen[c] = 0;
          for (int i = 0; i < 32; ++i) {
            const int2 in = *reinterpret_cast<const int2*>(&info[32 * c + i]);
            if (key >= in.x && key < in.y) seen[c] |= 1u << i;
          }
        }
      }
      if (!C::kOwn) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          score.tanh_of(s[c], masked);
          auto form = [&](auto m, auto l) {
            weights<decltype(m)::value, decltype(l)::value>(
                score, s[c], l2 + 32 * c, info + 32 * c, key, dist - 32 * c, seen[c], pk);
          };
          choose<BIAS>(masked, line, form);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            tmem_st8(tbase + lane_off + C::p((CW / 16) * wg + 2 * c + q), pk[q]);
        }
        if (slot.in_lo != INT_MAX) {
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.w_ready);
        }
      }
      ok = wait_warp(&sm.p_full, n & 1, abort_flag, err);
      if (!ok) break;
      tc_fence_after();
      if (slot.in_lo == INT_MAX) {
        // Rows that see nothing meet P = dS = 0: make Q and dO 0 there, now
        // that both score products have read them; dV(n) and dK(n) wait for
        // the arrivals of all warpgroups below, so they find every zero.
        if (wg < 2 && sm.info[st][r].y == 0)
          zero_row<NH, HALF>(wg == 0 ? sm.q[st] : sm.go[st], r);
        fence_proxy_async_smem();
        if (!C::kOwn) {
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.w_ready);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        load(C::dP, c, x);
        tmem_wait_ld();
        if (C::kOwn && c == NC - 1) {
          tc_fence_before();
          warp_arrive(&sm.p_free);
        }
        if (C::kOwn) {
          score.tanh_of(s[c], masked);
          auto form = [&](auto m, auto l) {
            both<decltype(m)::value, decltype(l)::value>(score, s[c], x, l2 + 32 * c,
                                                         info + 32 * c, key, dist - 32 * c,
                                                         seen[c], pk, gk);
          };
          choose<BIAS>(masked, line, form);
          if (c == 0 && n > 0) {
            ok = wait_warp(&sm.op_free, (n - 1) & 1, abort_flag, err);
            tc_fence_after();
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
            tmem_st8(tbase + lane_off + C::p((CW / 16) * wg + 2 * c + q), pk[q]);
        } else {
          if (masked) grads<true>(s[c], x, dd + 32 * c, seen[c], gk);
          else grads<false>(s[c], x, dd + 32 * c, seen[c], gk);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          tmem_st8(tbase + lane_off + C::ds((CW / 16) * wg + 2 * c + q), gk[q]);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&sm.ds_ready);
    }
    ok = wait_warp(&sm.out_full, 0, abort_flag, err) && ok;
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    tc_fence_after();
    if (S == 1) {
      constexpr uint32_t kStage = BM * (DH * 2 + 16);
      static_assert(kStage <= sizeof(sm.q) && kStage <= sizeof(sm.go), "staging fits in the ring");
      const size_t at = (static_cast<size_t>(g) * a.Nk + j0) * DH;
      store_block<DH, NWG>(tbase + lane_off + C::dK, a.tau, n == 0, &sm.q[0][0][0], wg, r,
                           threadIdx.x - 64, key_end - j0, ok,
                           static_cast<__nv_bfloat16*>(a.dK) + at);
      store_block<DH, NWG>(tbase + lane_off + C::dV, 1.f, n == 0, &sm.go[0][0][0], wg, r,
                           threadIdx.x - 64, key_end - j0, ok,
                           static_cast<__nv_bfloat16*>(a.dV) + at);
    } else {
      // This block's partial rows dK | dV, fp32, over the idle tiles.
      float* row = reinterpret_cast<float*>(&sm.k[0][0]) + r * kPartLd<DH>;
#pragma unroll
      for (int c = 0; c < 2 * DH / NWG; c += 16) {
        const int col = 2 * DH / NWG * wg + c;
        uint32_t v[16];
        tmem_ld16(tbase + lane_off + C::dK + col, v);
        tmem_wait_ld();
        const float scale = col < DH ? a.tau : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<float4*>(row + col)[k] =
              n == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(scale * u2f(v[4 * k]), scale * u2f(v[4 * k + 1]),
                                   scale * u2f(v[4 * k + 2]), scale * u2f(v[4 * k + 3]));
      }
    }
  }

  if (S > 1) {
    // Rank q sums key rows [128 q / S, 128 (q + 1) / S) over the cluster.  All
    // threads pass both barriers; the second keeps every block's rows alive
    // until all reads are done.
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
      const int rb = BM * rank / S, re = min(BM * (rank + 1) / S, a.Nk - j0);
      const uint32_t part = smem_u32(&sm.k[0][0]);
      constexpr int kRow4 = DH / 2;  // float4 of a row dK | dV
      for (int e = threadIdx.x - 64; e < (re - rb) * kRow4; e += 128 * NWG) {
        const int rr = rb + e / kRow4, c4 = e % kRow4;
        const uint32_t off = static_cast<uint32_t>((rr * kPartLd<DH> + 4 * c4) * 4);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < S; ++p) {
          const float4 v = ld_shared_cluster_f4(mapa_shared(part + off, p));
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(4 * c4 < DH ? a.dK : a.dV);
        const size_t at = (static_cast<size_t>(g) * a.Nk + j0 + rr) * DH + 4 * c4 % DH;
        if (!*abort_flag)
          *reinterpret_cast<uint2*>(out + at) =
              make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      }
    }
    __syncwarp();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// How many blocks share a key block: the power of two with the least of an
// estimate in row tiles (1.65 us at d = 128, 0.93 at d = 64).  A block costs `own`
// tiles to fill and drain, in a cluster `shared` (its launch and the exchange, 19
// us); the longest block has all the tiles, the average one half of them under a
// mask.  Clusters of 8 fit 16 times.  B2 H16 Hkv4 N2047 d128 causal, 128 key blocks
// of up to 64 tiles: alone 109 us, in twos 86, in fours 109; B1 H8 N2048, 128 of up
// to 16 (the whole gradient): 44, 54, 77; B1 H4 Hkv1 N4096, 32 of up to 128: in fours
// 77, in eights 97.
int cluster_size(const AttnArgs& a) {
  const double blocks = static_cast<double>((a.Nk + BM - 1) / BM) * a.B * a.Hkv;
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  const double tiles = static_cast<double>((rows + BQ - 1) / BQ);
  const double mean = a.causal || a.ranges ? tiles / 2 : tiles;
  const double own = a.d == 128 ? 5 : 9, shared = a.d == 128 ? 12 : 20;
  int best = 1;
  double least = 0;
  for (int S = 1; S <= 8 && tiles >= S; S *= 2) {
    const double fixed = S == 1 ? own : shared, waves = blocks * S / (S == 8 ? 128 : kSMs);
    const double longest = fixed + tiles / S, all = waves * (fixed + mean / S);
    if (S == 8 && waves > 1) break;
    const double cost = waves > 1 && all > longest ? all : longest;
    if (S == 1 || cost < least) best = S, least = cost;
  }
  return best;
}

template <int DH, bool CAP, bool BIAS>
cudaError_t launch(const AttnArgs& a) {
  const int heads = a.B * a.Hkv, rows = a.H / a.Hkv * a.Nq;
  CUtensorMap mq, mo, mk, mv;
  cudaError_t e = tc_map_bf16(&mq, a.Q, heads, rows, BQ, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mo, a.dO, heads, rows, BQ, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mk, a.K, heads, a.Nk, BM, DH);
  if (e == cudaSuccess) e = tc_map_bf16(&mv, a.V, heads, a.Nk, BM, DH);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(SmemK<DH>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  const auto kernel = tc_dkv_kernel<DH, CAP, BIAS>;
  e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // The staged rows lie over K, V, Q and dO, which follow one another.
  static_assert(BM * kPartLd<DH> * 4 <= offsetof(SmemK<DH>, ex), "partial rows fit in the tiles");
  const int S = cluster_size(a);
  const long long grid = static_cast<long long>((a.Nk + BM - 1) / BM) * heads * S;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_after(true, kernel, dim3(static_cast<unsigned>(grid)), NTHREADS, smem, S, a.stream,
                      mq, mo, mk, mv, a, S);
}

template <int DH>
cudaError_t launch(const AttnArgs& a) {
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  return cap ? (bias ? launch<DH, true, true>(a) : launch<DH, true, false>(a))
             : (bias ? launch<DH, false, true>(a) : launch<DH, false, false>(a));
}

}  // namespace

// At d = 64 without a cap L / tau is an operand: far outside tau's usual range it
// would overflow (a bias can make L large) or lose its low parts to underflow, and
// the gradient runs on CUDA cores, whose row state is the same.
bool tc_attn_grad_supported(const AttnArgs& a) {
  return tc_attn_supported(a) &&
         (a.d != 64 || a.cap > 0.f || (a.tau >= 0x1p-60f && a.tau <= 0x1p60f));
}

cudaError_t tc_attn_dkv(const AttnArgs& a) { return a.d == 64 ? launch<64>(a) : launch<128>(a); }

}  // namespace flashbob
