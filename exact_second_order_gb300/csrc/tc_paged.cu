// Attention of many query rows over a paged cache on sm_103a tensor cores: bf16
// queries, head dim 64 or 128, pages in e4m3 or bf16.
//   S = Q K^T,  y = score(S) + log2 s_V (scale, cap, bias; log2 units),
//   P~ = exp2(y - m) with a running row reference m >= max y - 8,
//   l = sum exp2(score(S) - m),  O = (sum P~ V) / l,  L = (m + log2 l) ln 2,
// where K and V are a page's codes: s_K goes into the score of its 16-column chunks
// and s_V into the exponent of their weights, so the MMAs' operands are codes (exact in
// fp16) and weights of at most 2^8 (11 significant bits), with sums in 32 bits that hold
// however far the pages' scales are apart (paged.cuh).  Q is scaled row by row, by a power
// of two, into fp16's reach.  A bf16 cache runs in bf16, its weights too, the MMA's other
// operand V being bf16 (a product of two halves of P~ would double its MMAs); l sums them
// unrounded, and O is off by 2.2e-3 in norm for that and its own rounding (alone 1.7e-3,
// which is what 8-bit caches are off by).
//
// As in the dense kernel, two elementwise warpgroups work on score tiles in TMEM, P~
// takes the scores' place as the A operand of P~ V, and one thread issues the MMAs.
// One warp looks up the pages, 32 chunks of 16 keys at a time, one a lane, and each lane
// asks for the boxes of its own chunks; a page outside the pool is a slab past the end,
// which TMA fills with zeros.  e4m3 has no MMA with a 16-bit partner, so its boxes land
// in a ring of codes, and converter warps turn them into fp16 in the operands' swizzled
// layout, keys so many tiles ahead of values as the MMA warp asks for them (in_order).  They
// load nothing from global memory themselves: the proxy fence behind their stores waits
// for every load of the thread that is under way (with the next tiles' codes in registers
// the kernel took 854 us, with more of them 1037, with the ring 452 in the end).
//   MT = 2: 256 group rows a block, warpgroup w holds rows 128 w .., so that a
//     converted tile feeds twice the products.
//   MT = 1: 128 rows, the warpgroups take alternate key tiles and merge their (m, l,
//     O~) at the end; few blocks are also cut along the keys and joined by a second
//     launch.
// Measured (H32 Hkv8 d128, 2048 rows behind 14336 keys): 456 us, 1130 TFLOP/s, in 1.7 waves
// (the longest SM has 480 key tiles where even shares are 408); dense bf16 keys 427, a bf16
// cache 372.  Four such prompts, padded, 1328 us, a bf16 cache 1103, dense keys 1109.  At
// d = 128 the MMAs of 64-key tiles cost 641 cycles for 512 of products and shared memory
// gives them 100 of its 128 bytes a cycle: the converters' 32 KB a tile take most of the
// rest, and 51% of the tensor pipe's cycles are busy (16-bit caches 64%).  Tiles of 128 keys
// would cost less, but with two score buffers only a warpgroup waits for its MMAs (749 us
// before the ring).  At d = 64 the same rows take 339 us, a bf16 cache 294, dense keys 290:
// no pipe is full (tensor 35%, exponentials 35%, issue 57%), the hand-offs between MMAs and
// elementwise warps bound it as in the dense kernel.
#include "paged.cuh"
#include "tc_attn.cuh"

namespace flashbob {
namespace {
using namespace tc;
using namespace attn;
using namespace paged;

constexpr int BM = kTcRows;
constexpr uint32_t HALF_BLOCK = BM * 64 * 2;
constexpr float kRescale = 8.f;
constexpr float kLargeScore = 0x1p20f;  // from here on y and m are off by 1/16

template <int DH, int MT, bool CODES>
struct Cfg {
  static constexpr int NH = DH / 64;
  static constexpr int BN = DH == 64 ? 128 : 64;  // keys of a tile
  static constexpr int kChunks = BN / 16;         // 16 keys lie on one page
  static constexpr uint32_t HT = BN * 64 * 2;     // bytes of 64 columns of a tile
  // Score buffers (O~ takes the rest of TMEM).  With MT = 1 a fourth asks for keys so early
  // that the ring has none under way: 82 us for 99 at B2 H16 Hkv4 N1000 of 5000 keys d128.
  static constexpr int NBUF = DH == 64 || MT == 1 ? 3 : 4;
  // Tiles of keys and of values as operands, and of codes on their way there.  Where they
  // arrive and leave together (kJoint) the MMA warp waits and commits less; converters,
  // which work in order, want slots of their own for keys that are asked for earlier.
  static constexpr bool kJoint = !CODES;
  static constexpr int NK = kJoint ? (MT == 2 ? 5 : 6) - (DH == 64 ? 0 : 1) : DH == 64 ? 4 : 3;
  static constexpr int NV = kJoint ? NK : DH == 64 || MT == 1 ? 3 : 2;
  static constexpr int k_tile(int s) { return kJoint ? 2 * s : s; }  // in the one array of tiles
  static constexpr int v_tile(int s) { return kJoint ? 2 * s + 1 : NK + s; }
  static constexpr int NI = CODES ? 8 : 0;
  // Keys come so many tiles ahead of values, as the MMA warp asks for them.
  static constexpr int kLead = kJoint ? 0 : (NBUF + MT - 1) / MT;
  // The scales of tile t are written when the codes that lay in its slot have been taken,
  // those of tile t - NI / 2 - kLead at least; so the scores of the tile NK before that are
  // done, which were issued behind the products of a unit NBUF earlier: its readers are
  // through.
  static constexpr int NS = 16;
  static_assert(NS >= NI / 2 + kLead + NK + NBUF, "scales");
  // Elementwise warps 0 - 7, converters (codes), loads, MMA.  With two converters the
  // elementwise threads have 168 registers, with four 128: MT = 2 1416 us for 1445 at four
  // prompts of 2048 behind 14336; MT = 1, with twice the tiles a product, 128 for 122 above.
  static constexpr int kConv = !CODES ? 0 : MT == 2 ? 2 : 4;
  // Of four, two turn keys and two values, neither waiting for the other's slots (500 rows of
  // 32 heads behind 4620 keys, d128: 75 us in turn, 67 in teams).
  static constexpr bool kTeams = kConv == 4;
  static constexpr int kTeam = kTeams ? 2 : kConv;  // converters of an item
  static constexpr int kLoad = 8 + kConv, kMma = kLoad + 1, kThreads = 32 * (kMma + 1);
  static_assert(2 * DH + NBUF * BN <= 512, "TMEM columns");
  // In the order of in_order the slot that a tile takes is free without any later one: keys
  // of tile t need the scores of t - NK, values the products of t - NV, which need no keys
  // beyond those of t - NV + kLead.
  static_assert(NK >= 2 && NV >= 2 && (!kJoint || NBUF <= MT * NK), "rings");
};

template <int DH, int MT, bool CODES>
struct Smem {
  using C = Cfg<DH, MT, CODES>;
  alignas(1024) uint8_t q[MT][C::NH][HALF_BLOCK];
  alignas(1024) uint8_t kv[C::NK + C::NV][C::NH][C::HT];
  alignas(1024) uint8_t item[C::NI > 0 ? C::NI : 1][C::NI > 0 ? C::BN * DH : 16];  // codes
  // Of each chunk of a tile: s_K, log2 s_V, 1 / s_V or 0 (kLeastLog), and whether any chunk of
  // the tile has 0 there.
  float4 scale[C::NS][C::kChunks];
  float part_m[2][BM], part_l[2][BM];
  int hull[8][4];  // of each elementwise warp's rows
  uint64_t k_full[C::NK], k_empty[C::NK], v_full[C::NV], v_empty[C::NV];
  uint64_t i_full[C::NI + 1], i_empty[C::NI + 1];
  uint64_t sc_full[C::NBUF], op_ready[C::NBUF];
  uint64_t pv_done[2];  // of even and odd units
  uint64_t out_full;
  uint64_t q_full, q_ready;
  uint32_t tmem_base;
  int abort_flag;
};

__host__ __device__ constexpr uint32_t idesc(bool codes, int N, bool b_mn_major) {
  return idesc_bf16(BM, N, b_mn_major) & (codes ? ~((1u << 7) | (1u << 10)) : ~0u);  // fp16: 0
}

template <bool CODES>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if (!CODES) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Scores of 64 columns from jbase on, 16 of a page each.  CAP: `s` holds products times
// tau / cap (scale), and for `weights`, and with a bias for `largest`, their tanh.
template <bool CODES, bool CAP, bool BIAS>
struct PagedScore {
  Score<CAP, BIAS> sc;
  float c1;  // not capped: log2 units a product; capped: tau / cap
  float c2;

  // `blind`: of a row that sees nothing.  Its tiles need not run masked, so its products, 0
  // or NaN here, must take no part in a warp's vote on the form of tanh.
  __device__ __forceinline__ PagedScore(const AttnArgs& a, float slope, float grow, bool blind)
      : sc(a, slope) {
    c1 = CAP && blind ? 0.f : sc.c1 * grow;
    c2 = sc.c2;
    sc.c1 = 1.f;  // its tanh is of products that are scaled already
    sc.a1 = kTanh[0], sc.a2 = kTanh[1], sc.a3 = kTanh[2];
    sc.most_raw = kTanhTo;
  }
  __device__ __forceinline__ void scale(uint32_t (&s)[4][16], const float4* chunk) const {
    if (!CAP) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = CODES ? c1 * chunk[q].x : c1;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 x = fmul2(f2(s[q][e], s[q][e + 1]), make_float2(f, f));
        s[q][e] = __float_as_uint(x.x);
        s[q][e + 1] = __float_as_uint(x.y);
      }
    }
  }
  __device__ __forceinline__ float factor(const float4& chunk) const {
    return CAP ? c2 : CODES ? c1 * chunk.x : c1;
  }
  __device__ __forceinline__ float2 at(float2 x, float f, float off, float dist) const {
    float2 y = ffma2(x, make_float2(f, f), make_float2(off, off));
    if (BIAS) {
      y.x = fmaf(-sc.slope2, fabsf(dist), y.x);
      y.y = fmaf(-sc.slope2, fabsf(dist + 1.f), y.y);
    }
    return y;
  }
  // The largest y.  Without a bias it grows with the raw product.
  template <bool MASKED>
  __device__ __forceinline__ float largest(const uint32_t (&s)[4][16], const float4* chunk,
                                           int jbase, int lo, int hi, float dist) const {
    float most = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float mr = -INFINITY;
      const float lv = CODES ? chunk[q].y : 0.f, f = factor(chunk[q]);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int j = jbase + 16 * q + e;
        float2 x = f2(s[q][e], s[q][e + 1]);
        if (BIAS) x = at(x, f, lv, dist + (16 * q + e));
        if (!MASKED || (j >= lo && j < hi)) mr = fmaxf(mr, x.x);
        if (!MASKED || (j + 1 >= lo && j + 1 < hi)) mr = fmaxf(mr, x.y);
      }
      if (!BIAS && mr != -INFINITY) mr = fmaf(f, CAP ? sc.tanh_one(mr) : mr, lv);
      most = fmaxf(most, mr);
    }
    return most;
  }
  // P~ to the TMEM columns from `out` on.
  template <bool MASKED>
  __device__ __forceinline__ void weights(const uint32_t (&s)[4][16], const float4* chunk,
                                          int jbase, int lo, int hi, float dist, float m, float& l,
                                          uint32_t out) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float2 acc = make_float2(0.f, 0.f);
      uint32_t pk[8];
      const float f = factor(chunk[q]), off = CODES ? chunk[q].y - m : -m;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 y = at(f2(s[q][e], s[q][e + 1]), f, off, dist + (16 * q + e));
        float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        if (MASKED) {
          const int j = jbase + 16 * q + e;
          if (j < lo || j >= hi) p.x = 0.f;
          if (j + 1 < lo || j + 1 >= hi) p.y = 0.f;
        }
        acc = fadd2(acc, p);
        pk[e >> 1] = pack<CODES>(p.x, p.y);
      }
      tmem_st8(out + 8 * q, pk);
      l = CODES ? fmaf(chunk[q].z, acc.x + acc.y, l) : l + (acc.x + acc.y);
    }
  }
  // The same for a tile that has chunks of the least scales, whose part of l is summed apart
  // (kLeastLog), or for scores so large that their rounding would be seen in y - m where the
  // two are one fma: here y is rounded as it was for m, so that no weight is above 2^8.  A
  // chunk of 16 columns at a time, from TMEM, and a call: inlined it took the hot path's
  // registers (capped prompts at d = 64 355 -> 387 us).
  static __device__ __noinline__ float careful(const PagedScore me, uint32_t tmem,
                                               const float4* chunk, int chunks, int jbase, int lo,
                                               int hi, float dist, float m, float l) {
#pragma unroll 1
    for (int q = 0; q < chunks; ++q) {
      uint32_t s[1][16], pk[8];
      tmem_ld16(tmem + 16 * q, s[0]);
      tmem_wait_ld();
      const float4 c = chunk[q];
      if (CAP) {
        const float f = me.c1 * c.x;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[0][e] = __float_as_uint(f * u2f(s[0][e]));
        me.sc.tanh_of(s, true);
      }
      const float f = me.factor(c);
      const bool least = c.z == 0.f;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 y = me.at(f2(s[0][e], s[0][e + 1]), f, c.y, dist + (16 * q + e));
        const int j = jbase + 16 * q + e;
        const float x[2] = {y.x - m, y.y - m};
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool seen = j + k >= lo && j + k < hi;
          p[k] = seen ? ex2_approx(x[k]) : 0.f;
          sum += !least ? p[k] : seen ? ex2_approx(x[k] - c.y) : 0.f;
        }
        pk[e >> 1] = pack<true>(p[0], p[1]);
      }
      tmem_st8(tmem + 8 * q, pk);
      l = least ? l + sum : fmaf(c.z, sum, l);
    }
    return l;
  }
};

// Tiles in the order in which they are loaded, converted and asked for: the keys of the
// first kLead, then values of tile t and keys of tile t + kLead (kLead = 0: keys and
// values of each tile).
template <int LEAD, typename F>
__device__ __forceinline__ void in_order(int T, const F& item) {
  bool ok = true;
  int i = 0;
  for (int x = 0; ok && x < T + LEAD; ++x) {
    if (LEAD == 0) ok = item(i++, x, false);
    if (ok && x >= LEAD) ok = item(i++, x - LEAD, true);
    if (LEAD > 0 && ok && x < T) ok = item(i++, x, false);
  }
}

// The converters' threads: run i of a thread is 16-byte run `col` of row row0 +
// kStep i of an item.  Eight lanes read 16-byte runs of codes, and store runs of fp16, on
// different banks: with rows of 128 bytes (two halves of fp16) four runs of one half of
// rows r and r ^ 5, else four of two rows.
template <int DH, int NT>
struct Feed {
  static constexpr int kPerRow = DH / 16, kStep = NT / kPerRow;
  int col, row0;
  __device__ __forceinline__ explicit Feed(int tid) {
    col = tid & 3;
    row0 = tid >> 2;
    if (DH == 128) {
      col |= (tid >> 1) & 4;
      row0 = ((tid >> 2 & 1) * 5) ^ ((tid >> 4 & 1) * 2) ^ ((tid >> 5 & 1) * 4) ^ (tid >> 6 << 3);
    }
  }
};

template <int DH, int MT, bool CODES, bool CAP, bool BIAS>
__global__ void __launch_bounds__((Cfg<DH, MT, CODES>::kThreads), 1)
    tc_paged_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                    const __grid_constant__ CUtensorMap mV,
                    const __grid_constant__ PagedAttnArgs a, int blocks, int splits) {
  extern __shared__ uint8_t smem_raw[];
  using C = Cfg<DH, MT, CODES>;
  constexpr int NK = C::NK, NV = C::NV, NH = C::NH, NBUF = C::NBUF, BN = C::BN;
  constexpr int kChunks = C::kChunks;
  constexpr uint32_t HT = C::HT;
  constexpr uint32_t kScore = 2 * DH;
  Smem<DH, MT, CODES>& sm = *reinterpret_cast<Smem<DH, MT, CODES>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.B * a.Hkv, G = a.H / a.Hkv, rows = G * a.Nq;
  const int g = blockIdx.x % heads, rest = blockIdx.x / heads;
  const int b = g / a.Hkv, hkv = g % a.Hkv;
  const int split = rest % splits;
  const int row0 = row_block(rest / splits, blocks, G, a.Nq, MT * BM) * (MT * BM);
  volatile int* abort_flag = &sm.abort_flag;
  unsigned int* err = a.err;

  if (splits > 1) release_next();
  if (threadIdx.x == 0) {
    constexpr int kFull = CODES ? C::kTeam : 1;
    for (int s = 0; s < NK; ++s) mbar_init(&sm.k_full[s], kFull), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < NV; ++s) mbar_init(&sm.v_full[s], kFull), mbar_init(&sm.v_empty[s], 1);
    for (int s = 0; s < C::NI; ++s) mbar_init(&sm.i_full[s], 1), mbar_init(&sm.i_empty[s], C::kTeam);
    for (int s = 0; s < NBUF; ++s) mbar_init(&sm.sc_full[s], 1), mbar_init(&sm.op_ready[s], 4);
    mbar_init(&sm.pv_done[0], 1);
    mbar_init(&sm.pv_done[1], 1);
    mbar_init(&sm.out_full, 1);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_ready, 8);
    sm.abort_flag = 0;
    fence_barrier_init();
    // Q is under way while the ranges are read.
    mbar_expect_tx(&sm.q_full, MT * NH * HALF_BLOCK);
    for (int w = 0; w < MT; ++w)
      for (int h = 0; h < NH; ++h)
        tma_load_3d(sm.q[w][h], &mQ, &sm.q_full, 64 * h, row0 + BM * w, g);
  }
  if (warp == C::kMma) tmem_alloc(&sm.tmem_base, 512);
  const int wg = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
  GroupRow gr{empty_view(), 0.f};
  const int row = row0 + r + (MT == 2 ? BM * wg : 0);
  if (warp < 8) {
    gr = group_row(a, b, hkv, row, rows);
    // Rows that see nothing (padding of a batch) do not make every tile a masked one.
    warp_hull(gr.v, row < rows && gr.v.hi > 0, lane, sm.hull[warp]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const Hull hull = join_hulls(sm.hull, 8);
  // Key tiles of the hull, and this split's run of them.
  const int t_lo = hull.lo < hull.hi ? hull.lo / BN : 0;
  const int t_n = hull.lo < hull.hi ? (hull.hi + BN - 1) / BN - t_lo : 0;
  const int tb = t_lo + static_cast<int>(static_cast<long long>(t_n) * split / splits);
  const int T = t_lo + static_cast<int>(static_cast<long long>(t_n) * (split + 1) / splits) - tb;
  const int U = MT * T;  // units

  if (warp == C::kMma) {
    constexpr uint32_t idS = idesc(CODES, BN, false), idO = idesc(CODES, DH, true);
    const uint64_t dQ = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t dK0 = smem_desc_sw128(smem_u32(sm.kv[C::k_tile(0)][0]), 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(smem_u32(sm.kv[C::v_tile(0)][0]), HT, 1024);
    constexpr uint64_t kStep = (C::k_tile(1) * NH * HT) >> 4;  // V's is the same
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
      if (!C::kJoint && (MT == 1 || (u & 1))) mma_commit(&sm.k_empty[tile(u) % NK]);
    };
    auto issue_pv = [&](int u) {
      const int s = tile(u) % NV;
      const uint32_t sc = tbase + kScore + BN * (u % NBUF);
      const uint64_t dv = dV0 + s * kStep;
      const uint32_t acc_col = tbase + DH * (u & 1);
#pragma unroll
      for (int c = 0; c < BN / 16; ++c)
        mma_ts(acc_col, sc + 8 * c, dv + ((16 * 128 * c) >> 4), idO, (u >= 2 || c > 0));
      mma_commit(&sm.pv_done[u & 1]);
      if (MT == 1 || (u & 1)) mma_commit(&sm.v_empty[s]);
    };
    if (elect_one()) {
      bool ok = wait_one(CODES ? &sm.q_ready : &sm.q_full, 0, abort_flag, err);
      tc_fence_after();
      auto scores = [&](int u) {
        const int t = tile(u);  // MT = 2: the second unit of a tile finds it there
        if (MT == 1 || !(u & 1)) {
          ok = wait_one(&sm.k_full[t % NK], (t / NK) & 1, abort_flag, err);
          tc_fence_after();
        }
        if (ok) issue_scores(u);
      };
      for (int u = 0; ok && u < NBUF && u < U; ++u) scores(u);
      for (int u = 0; ok && u < U; ++u) {
        const int t = tile(u);
        ok = (C::kJoint || (MT == 2 && (u & 1)) ||
              wait_one(&sm.v_full[t % NV], (t / NV) & 1, abort_flag, err)) &&
             wait_one(&sm.op_ready[u % NBUF], (u / NBUF) & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        issue_pv(u);
        if (u + NBUF < U) scores(u + NBUF);
      }
      mma_commit(&sm.out_full);
    }
    __syncwarp();
  } else if (warp == C::kLoad) {
    // One lane for each of the next 32 chunks of 16 keys, and of the 32 behind: the page
    // and head that holds it (one past the last where there is nothing to read, which
    // the copies fill with zeros) and its scales.
    struct Meta {
      int slab;
      float4 scale;  // as in Smem
    };
    const int chunks = T * kChunks, chunk0 = tb * kChunks;
    const int box = min(a.page.T, BN);  // keys of one copy
    auto meta_of = [&](int n) {
      Meta m{a.page.P * a.Hkv, make_float4(1.f, 0.f, 1.f, 0.f)};
      const int j = (chunk0 + n) * 16 & ~(box - 1);
      if (n < chunks && j < hull.hi && j + box > hull.lo) {
        const int page = page_at(a.page, b, j);
        if (page_ok(a.page, page)) {
          m.slab = page * a.Hkv + hkv;
          if (CODES) {
            const float vs = a.page.v_scale[m.slab];
            const float lv = __log2f(vs);
            m.scale = make_float4(a.page.k_scale[m.slab], lv, lv < kLeastLog ? 0.f : 1.f / vs, 0.f);
          }
        }
      }
      return m;
    };
    constexpr int kAhead = 32 / kChunks;  // tiles that 32 chunks are
    static_assert(C::kLead <= kAhead, "values are at most one batch behind the keys");
    Meta prv, cur = meta_of(lane), nxt = meta_of(32 + lane);
    prv = cur;
    // This lane's chunk: of the tiles `turn` of kAhead, at byte `to` of a tile, and
    // whether it asks for a box there (the lane of the box's first chunk does).
    const int turn = lane / kChunks, chunk = lane % kChunks;
    const bool asks = (16 * chunk & (box - 1)) == 0;
    const uint32_t to = 16 * chunk * (CODES ? DH : 128);
    const int page_y = (tb * BN + 16 * chunk) & (a.page.T - 1), turn_y = BN & (a.page.T - 1);
    int nk = 0, ni = 0;  // tiles and items that are under way
    in_order<C::kLead>(T, [&](int i, int t, bool values) {
      const int s = t % NK, it = i % (C::NI + !CODES);
      if (!values && t > 0 && t % kAhead == 0) {
        prv = cur;
        cur = nxt;
        nxt = meta_of((t / kAhead + 1) * 32 + lane);
      }
      // A joint slot is waited for with the keys, and its barrier counts both.
      bool ok = true;
      if (CODES)
        ok = i < C::NI ||
             wait_warp(&sm.i_empty[it], ((i / (C::NI + !CODES)) - 1) & 1, abort_flag, err);
      else if (!values)
        ok = t < NV || wait_warp(&sm.v_empty[s], ((t / NV) - 1) & 1, abort_flag, err);
      if (!ok) return false;
      uint64_t* bar = CODES ? &sm.i_full[it] : &sm.k_full[s];
      const bool mine = turn == t % kAhead;
      // Values may be of the batch before: the keys are nk - 1 tiles on.
      const int slab = values && t / kAhead != (nk - 1) / kAhead ? prv.slab : cur.slab;
      if (CODES && !values) {
        const bool least = __any_sync(0xffffffffu, mine && cur.scale.z == 0.f);
        if (mine)
          sm.scale[t % C::NS][chunk] =
              make_float4(cur.scale.x, cur.scale.y, cur.scale.z, least ? 1.f : 0.f);
        __syncwarp();
      }
      if (lane == 0 && (CODES || !values)) mbar_expect_tx(bar, CODES ? BN * DH : 2 * NH * HT);
      if (mine && asks) {
        uint8_t* dst = (CODES ? sm.item[it] : sm.kv[values ? C::v_tile(s) : C::k_tile(s)][0]) + to;
        const CUtensorMap* map = values ? &mV : &mK;
        const int y = (page_y + t * turn_y) & (a.page.T - 1);
        tma_load_3d(dst, map, bar, 0, y, slab);
        if (!CODES && NH == 2) tma_load_3d(dst + HT, map, bar, 64, y, slab);
      }
      ni = i + 1;
      if (!values) nk = t + 1;
      return true;
    });
    if (lane == 0) {  // what is under way has to land before the block ends
      drain_wait(&sm.q_full, 0);
      if (CODES) {
        for (int i = ni > C::NI ? ni - C::NI : 0; i < ni; ++i)
          drain_wait(&sm.i_full[i % (C::NI + !CODES)], (i / (C::NI + !CODES)) & 1);
      } else {
        for (int t = nk > NK ? nk - NK : 0; t < nk; ++t) drain_wait(&sm.k_full[t % NK], (t / NK) & 1);
      }
    }
    __syncwarp();
  } else if (CODES && warp >= 8) {
    const bool of_values = warp >= 8 + C::kTeam;  // of two teams
    const int tid = threadIdx.x - 256 - (of_values ? 32 * C::kTeam : 0);
    using F = Feed<DH, CODES ? 32 * C::kTeam : 128>;
    const F f(tid);
    constexpr int kRuns = BN / F::kStep, kStep = F::kStep;
    static_assert(kStep % 8 == 0, "a thread's runs have one place in the swizzles");
    const uint32_t c = (16 * f.col % 64) / 8, line = (16 * f.col / 64) * HT + f.row0 * 128;
    const uint32_t at0 = line + ((c ^ (f.row0 & 7)) << 4);
    const uint32_t at1 = line + (((c + 1) ^ (f.row0 & 7)) << 4);
    const uint32_t from =
        f.row0 * DH + ((f.col ^ (DH == 128 ? f.row0 & 7 : (f.row0 >> 1) & 3)) << 4);
    in_order<C::kLead>(T, [&](int i, int t, bool values) {
      if (C::kTeams && values != of_values) return true;
      const int N = values ? NV : NK, s = t % N, it = i % (C::NI + !CODES);
      const bool ok = wait_warp(&sm.i_full[it], (i / (C::NI + !CODES)) & 1, abort_flag, err) &&
                      (t < N || wait_warp(values ? &sm.v_empty[s] : &sm.k_empty[s],
                                          ((t / N) - 1) & 1, abort_flag, err));
      if (!ok) return false;
      const uint32_t src = smem_u32(sm.item[it]) + from;
      const uint32_t dst = smem_u32(sm.kv[values ? C::v_tile(s) : C::k_tile(s)][0]);
      uint32_t w[kRuns][4];
#pragma unroll
      for (int u = 0; u < kRuns; ++u)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                     : "r"(src + u * kStep * DH)
                     : "memory");
      // What no row of the block sees may be anything: zeros, which weights of 0 meet.
      const int j0 = (tb + t) * BN;
      if (j0 < hull.lo || j0 + BN > hull.hi) {
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
          const int j = j0 + f.row0 + kStep * u;
          if (j < hull.lo || j >= hull.hi) w[u][0] = w[u][1] = w[u][2] = w[u][3] = 0u;
        }
      }
#pragma unroll
      for (int u = 0; u < kRuns; ++u) {
        uint32_t h[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[2 * q] = codes_to_half2(static_cast<uint16_t>(w[u][q]));
          h[2 * q + 1] = codes_to_half2(static_cast<uint16_t>(w[u][q] >> 16));
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + at0 + u * kStep * 128),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + at1 + u * kStep * 128),
                     "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                     : "memory");
      }
      fence_proxy_async_smem();
      warp_arrive(values ? &sm.v_full[s] : &sm.k_full[s]);
      if (lane == 0) mbar_arrive(&sm.i_empty[it]);
      return true;
    });
  } else {
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t acc_own = tbase + lane_off + DH * wg;
    const int lo = gr.v.lo, hi = gr.v.hi;
    const Hull own = MT == 2 ? join_hulls(sm.hull + 4 * wg, 4) : hull;
    bool ok = wait_warp(&sm.q_full, 0, abort_flag, err);
    float grow = 1.f;
    if (CODES) {
      // Q to fp16 in place, this thread's row (MT = 1: of two threads each writes half of
      // the runs, when both have seen the row).
      uint8_t* q = sm.q[MT == 2 ? wg : 0][0] + r * 128;
      constexpr int kRuns = DH / 8;
      auto run = [&](int k) {
        return reinterpret_cast<uint4*>(q + (k / 8) * HALF_BLOCK + (((k % 8) ^ (r & 7)) << 4));
      };
      float most = 0.f;
#pragma unroll 4
      for (int k = 0; k < kRuns; ++k) {
        const uint4 v = *run(k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = fmaxf(most, fmaxf(finite_abs(u2f(w[e] << 16)), finite_abs(u2f(w[e] & 0xFFFF0000u))));
      }
      const float shrink = row_shrink(most);
      grow = 1.f / shrink;
      if (MT == 1) named_bar_sync(1, 256);
#pragma unroll 4
      for (int k = MT == 1 ? wg * kRuns / 2 : 0; k < (MT == 1 ? (wg + 1) * kRuns / 2 : kRuns); ++k) {
        const uint4 v = *run(k);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack<true>(u2f(w[e] << 16) * shrink, u2f(w[e] & 0xFFFF0000u) * shrink);
        *run(k) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      warp_arrive(&sm.q_ready);
    }
    // A row that sees nothing, whatever its Q is: all its weights are 0 (or NaN), and O is
    // not taken from them.
    const bool blind = hi <= 0;
    const PagedScore<CODES, CAP, BIAS> score(a, gr.slope2, grow, blind);
    const bool any_row = row0 + (MT == 2 ? BM * wg : 0) + quad * 32 < rows;
    // Values that no row of the block sees meet P~ = 0: make them 0 too (codes are
    // already).
    auto clear_hidden = [&](int t, int col0) {
      if (CODES || (col0 >= hull.lo && col0 + BN <= hull.hi)) return true;
      if (!wait_warp(&sm.k_full[t % NK], (t / NK) & 1, abort_flag, err)) return false;
      if (r < BN && (col0 + r < hull.lo || col0 + r >= hull.hi))
        zero_row<NH, HT>(sm.kv[C::v_tile(t % NV)], r);
      fence_proxy_async_smem();
      return true;
    };
    float m = -INFINITY, l = 0.f;
    int n = 0;  // units of this warpgroup
    for (int u = wg; u < U; u += 2, ++n) {
      const int t = MT == 2 ? u >> 1 : u, col0 = (tb + t) * BN;
      ok = ok && wait_warp(&sm.sc_full[u % NBUF], (u / NBUF) & 1, abort_flag, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sc = tbase + lane_off + kScore + BN * (u % NBUF);
      const bool masked = col0 < own.in_lo || col0 + BN > own.in_hi;
      const float dist = BIAS ? static_cast<float>(col0 - gr.v.pos) : 0.f;
      const float4* chunk = sm.scale[t % C::NS];
      if (!any_row) {
        ok = clear_hidden(t, col0);
        if (!ok) break;
        warp_arrive(&sm.op_ready[u % NBUF]);
        continue;
      }
      // Groups of 64 columns; of two the second is read twice, so that one is held in
      // registers at a time.  P~ of columns 16 c .. goes to columns 8 c .., onto scores
      // already used.
      uint32_t s[4][16];
      auto load = [&](int c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld16(sc + c + 16 * q, s[q]);
        tmem_wait_ld();
        score.scale(s, chunk + c / 16);
        if (CAP && BIAS) score.sc.tanh_of(s, masked);
      };
      auto max_of = [&](int c) {
        return masked ? score.template largest<true>(s, chunk + c / 16, col0 + c, lo, hi, dist + c)
                      : score.template largest<false>(s, chunk + c / 16, col0 + c, lo, hi, dist + c);
      };
      float mt = -INFINITY;
      if (BN == 128) {
        load(64);
        mt = max_of(64);
      }
      load(0);
      mt = fmaxf(mt, max_of(0));
      const bool raise = !blind && mt > m + kRescale;
      const PartFactor<CODES> pf(m == -INFINITY ? -INFINITY : m - mt);
      const float fac = raise ? pf.all() : 1.f;
      if (raise) {
        l = pf.of(l);
        m = mt;
      }
      // Tiles for careful().  Large references vote with the raised ones: a vote of their own
      // is a wait between maximum and weights (2% at d = 128).
      bool special = CODES && chunk[0].w != 0.f;
      const bool large = CODES && m != -INFINITY && fabsf(m) > kLargeScore;
      const bool any_raise = __any_sync(0xffffffffu, (raise && fac < 1.f) || large);
      if (CODES && any_raise) special = special || __any_sync(0xffffffffu, large);
      if (any_raise && n > 0) {
        // The products of this warpgroup's last unit.  S(u) was issued behind those of
        // unit u - NBUF, so of the barrier's phases only the last may be open.
        const int last = u - 2;
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
            w0[k] = __float_as_uint(u2f(v[k]) * fac);
            w1[k] = __float_as_uint(u2f(v[8 + k]) * fac);
          }
          tmem_st8(acc_own + 16 * c, w0);
          tmem_st8(acc_own + 16 * c + 8, w1);
        }
      }
      const float base = blind ? INFINITY : m == -INFINITY ? 0.f : m;  // nothing seen so far: 0
      if (CODES && __builtin_expect(special, 0)) {
        l = PagedScore<CODES, CAP, BIAS>::careful(score, sc, chunk, kChunks, col0, lo, hi, dist,
                                                  base, l);
      } else {
#pragma unroll
        for (int c = 0; c < BN; c += 64) {
          if (c > 0) load(c);
          if (!BIAS) score.sc.tanh_of(s, masked);
          const float4* sca = chunk + c / 16;
          if (masked)
            score.template weights<true>(s, sca, col0 + c, lo, hi, dist + c, base, l, sc + c / 2);
          else
            score.template weights<false>(s, sca, col0 + c, lo, hi, dist + c, base, l, sc + c / 2);
        }
      }
      ok = clear_hidden(t, col0);
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
    if (MT == 1) {
      sm.part_m[wg][r] = m;
      sm.part_l[wg][r] = l;
      named_bar_sync(1, 256);
      const float m0 = sm.part_m[0][r], m1 = sm.part_m[1][r];
      mm = fmaxf(m0, m1);
      const PartFactor<CODES> f0(m0 == -INFINITY ? -INFINITY : m0 - mm);
      const PartFactor<CODES> f1(m1 == -INFINITY ? -INFINITY : m1 - mm);
      s0 = f0.all(), s1 = f1.all();
      lsum = f0.of(sm.part_l[0][r]) + f1.of(sm.part_l[1][r]);
    }
    if (blind) lsum = 0.f;
    const bool any0 = T > 0 && !blind, any1 = MT == 1 && T > 1 && !blind;
    const float inv = splits > 1 ? 1.f : lsum > 0.f ? 1.f / lsum : 0.f;
    s0 = any0 ? s0 * inv : 0.f;
    s1 = any1 ? s1 * inv : 0.f;
    const size_t all = static_cast<size_t>(a.B) * a.H * a.Nq;
    const size_t base = static_cast<size_t>(g) * rows;  // first row of the group
    const Partials part = partials(a.workspace, all, DH, splits);
    if (ok && row < rows && (MT == 2 || wg == 0)) {
      if (splits > 1) part.ml[split * all + base + row] = make_float2(mm, lsum);
      else a.L[base + row] = (mm + __log2f(lsum)) * kLn2;
    }
    // Every MMA is done, so the ring is idle: 64 columns of O at a time go through it
    // and leave with coalesced stores.
    constexpr int kStageLd = 64 + 4;
    float* st = reinterpret_cast<float*>(&sm.kv[0][0][0]);
    static_assert(MT * BM * kStageLd * 4 <= sizeof(sm.kv), "epilogue staging fits in the ring");
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h > 0) named_bar_sync(1, 256);
      // With two accumulators for the same rows each warpgroup forms half the columns.
      constexpr int kCols = MT == 1 ? 32 : 64;
      const int c0 = MT == 1 ? 32 * wg : 0, sr = MT == 2 ? BM * wg + r : r;
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        const uint32_t col = 64 * h + c0 + c;
        uint32_t v0[16], v1[16];
        if (MT == 2) {
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
            if (MT == 1 && any1) o[q] = fmaf(s1, u2f(v1[4 * k + q]), o[q]);
          }
          s4[k] = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      named_bar_sync(1, 256);
      const int live = min(MT * BM, rows - row0);
      if (ok) {
        for (int f = threadIdx.x; f < live * 16; f += 256) {
          const int rr = f >> 4, c4 = f & 15;
          const float4 v = *reinterpret_cast<const float4*>(st + rr * kStageLd + 4 * c4);
          const size_t at = (base + row0 + rr) * DH + 64 * h + 4 * c4;
          if (splits > 1)
            *reinterpret_cast<float4*>(part.o + split * all * DH + at) = v;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + at) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int DH, int MT, bool CODES, bool CAP, bool BIAS>
cudaError_t launch(const PagedAttnArgs& a, int splits) {
  constexpr size_t smem = sizeof(Smem<DH, MT, CODES>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  const auto kernel = tc_paged_kernel<DH, MT, CODES, CAP, BIAS>;
  CUtensorMap mq, mk, mv;
  const int rows = a.H / a.Hkv * a.Nq, blocks = (rows + MT * BM - 1) / (MT * BM);
  const int slabs = a.page.P * a.Hkv, box = a.page.T < Cfg<DH, MT, CODES>::BN
                                               ? a.page.T : Cfg<DH, MT, CODES>::BN;
  cudaError_t e = tc_map_bf16(&mq, a.Q, a.B * a.Hkv, rows, BM, DH);
  if (e == cudaSuccess) e = tc_map(&mk, a.K, slabs, a.page.T, box, DH, CODES);
  if (e == cudaSuccess) e = tc_map(&mv, a.V, slabs, a.page.T, box, DH, CODES);
  if (e == cudaSuccess)
    e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(blocks) * splits * a.B * a.Hkv;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  kernel<<<static_cast<unsigned>(grid), Cfg<DH, MT, CODES>::kThreads, smem, a.stream>>>(
      mq, mk, mv, a, blocks, splits);
  return cudaGetLastError();
}

template <int DH, int MT, bool CODES>
cudaError_t launch(const PagedAttnArgs& a, int splits) {
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  return cap ? (bias ? launch<DH, MT, CODES, true, true>(a, splits)
                     : launch<DH, MT, CODES, true, false>(a, splits))
             : (bias ? launch<DH, MT, CODES, false, true>(a, splits)
                     : launch<DH, MT, CODES, false, false>(a, splits));
}

// 256 rows a block at d = 128 where such blocks have three quarters of the SMs or more (1024
// rows of 32 heads behind 4096 keys, e4m3: 89 us for 126 with 128 rows; half as many rows 90
// for 75).  At d = 64 only with codes, whose conversion is shared, and from one and a half
// waves on (2048 rows of 32 heads behind 14336 keys: 341 for 433; 16-bit 292 for 298; four
// windows of 1024 keys, 192 such blocks, 69 for 61, 16-bit 65 for 52).
bool two_blocks(const PagedAttnArgs& a) {
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  const long long blocks = static_cast<long long>(a.B) * a.Hkv * ((rows + 255) / 256);
  return rows > BM && (a.d == 128 ? 4 * blocks >= 3 * kSMs
                                  : a.page.e4m3 && 2 * blocks >= 3 * kSMs);
}

}  // namespace

bool tc_paged_supported(const PagedAttnArgs& a) { return a.bf16 && (a.d == 64 || a.d == 128); }

// Runs that the keys are cut into where blocks leave SMs idle, 256 keys at least in each
// (100 rows of 8 heads behind 3900 keys: 21.6 us, with 512 23.7, with 1024 29.9).
int tc_paged_splits(const PagedAttnArgs& a) {
  if (two_blocks(a)) return 1;
  const long long rows = static_cast<long long>(a.H / a.Hkv) * a.Nq;
  const long long blocks = static_cast<long long>(a.B) * a.Hkv * ((rows + BM - 1) / BM);
  const long long want = kSMs / blocks, most = a.Nk / 256;
  const long long s = want < most ? want : most;
  return s < 1 ? 1 : static_cast<int>(s);
}

cudaError_t tc_paged(const PagedAttnArgs& a) {
  const int splits = tc_paged_splits(a);
  cudaError_t e;
  const bool two = two_blocks(a);
  if (a.d == 64)
    e = two              ? launch<64, 2, true>(a, 1)
        : a.page.e4m3    ? launch<64, 1, true>(a, splits)
                         : launch<64, 1, false>(a, splits);
  else if (a.page.e4m3)
    e = two ? launch<128, 2, true>(a, 1) : launch<128, 1, true>(a, splits);
  else
    e = two ? launch<128, 2, false>(a, 1) : launch<128, 1, false>(a, splits);
  return e == cudaSuccess && splits > 1 ? attn_join(a, splits) : e;
}

}  // namespace flashbob
