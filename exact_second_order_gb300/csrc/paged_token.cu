// Attention of a few query rows over a paged cache: bf16 queries, head dim 64 or
// 128, pages in e4m3 or bf16, up to 32 group rows (single tokens, drafted ones).
//   S^T = K Q^T,  x = score(S) (scale, cap, bias; log2 units),
//   y = x + log2 s_V,  p = exp2(y - R) with a running reference R >= max y - 8,
//   l = sum exp2(x - R),  O^T = (sum V^T p) / l,  L = (R + log2 l) ln 2,
// where K and V are a page's codes: the scale of the keys goes into the scores, that
// of the values into the exponent of the weights, so that a product's operands are
// codes (exact in fp16) and weights of at most 2^8 (16 bits each, 11 significant), with
// sums in 32 bits that hold however far the pages' scales are apart (paged.cuh).  Q is
// scaled row by row, by a power of two, into fp16's reach.  With a bf16 cache weights are
// bf16, as in the dense call: both operands of a product have one type, fp16 would not
// hold what V may be, and two halves of a weight would double the products with V; l sums
// them unrounded.
//
// The keys' bytes bound it (2 d bytes a key and head for e4m3), not the products: a
// warp holds all rows and streams pages alone, 16 tokens at a time, through a ring of
// its own in shared memory (TMA boxes that one lane asks for, no block-wide barrier
// between the first and the end).  With tokens along M and rows along N = 8 a product
// (mma.sync m16n8k16) wastes nothing on rows that are not there: tcgen05 would want 64
// rows or more, and its operands in shared memory in 16 bits, twice the bytes that
// arrive.  Along the contracted side any order will do, so a lane takes whole 16-byte
// runs of a key's code (four steps of 4 elements) and of a value's (its own head columns
// of four tokens, paired by byte permutes); which token of a tile is which row of a
// product (token_of) is chosen so that in the boxes' swizzle both reads are without bank
// conflicts.  The weights go from accumulator to operand by two 8 x 8 transposes.
// Measured: 32 requests of up to 8192 keys (H32 Hkv8 d128, e4m3) 54 to 55 us and 5 for the
// join, 329 MB, 5.9 to 6.1 TB/s (5.5 with the join, 81% of the copy rate); 64 of 8192 keys,
// after a flush, 185 us with the join, 5.8 TB/s; a bf16 cache 94 us, 655 MB, 7.0 TB/s of
// which a part lay in the L2.  Drafted tokens (16 requests of 4, up to 4096 keys, H16
// Hkv4) 28 us capped, 24 not: 128 blocks on 152 SMs, the longest with 2048 keys.
// The warps' parts meet in shared memory.  A group's keys are cut into runs: where the
// groups are few, as many as fill the SMs once, in clusters whose parts meet in
// distributed shared memory (and across clusters in a second launch); where they are
// more, two waves of them, longest requests first, joined by a second launch (clusters
// that wait for one another's SMs cost several us a wave).  Equal shares of all units,
// one a block, with a block's work going on from group to group, took longer: a group's
// beginning is a chain of four memory latencies (ranges, pages, codes, and Q), which
// blocks beside each other hide and a single one does not (32 requests of up to 8192
// keys 87 us for 75, 16 with 4 drafted tokens 46 for 32, after a flush of the L2).
#include "paged.cuh"
#include "tc_attn.cuh"

namespace flashbob {
namespace {
using namespace attn;
using namespace paged;
using tc::ex2_approx;
using tc::smem_u32;

constexpr int NW = 8;
constexpr int kUnit = 16;  // tokens; a page is one unit or several
constexpr float kRaise = 8.f;
constexpr int kMostRows = 32;
constexpr int kMostSorted = 128;  // batch entries; of more than that few blocks are the end

// Runs that a group's keys are cut into, of 512 keys at least.
struct TokenRuns {
  int cluster;   // runs that meet in distributed shared memory
  int partials;  // and so many of those are joined by a second launch
  int sorted;    // blocks of long batch entries first
};

template <int DH, bool CODES, int NT>
struct Tok {
  static constexpr int kRow = DH * (CODES ? 1 : 2);     // bytes of a token's row
  static constexpr int kTile = kUnit * kRow;            // of a unit's keys, or values
  static constexpr int kRun = CODES ? 16 : 8;           // elements in 16 bytes
  static constexpr int kK = DH / 16;                    // steps of the score products
  static constexpr int kMT = DH / 16;                   // row tiles of O^T
  // Two blocks an SM where registers and shared memory allow.
  static constexpr bool kTwo = NT == 1 && kTile <= 2048;
  static constexpr int kRing = kTwo ? 12288 : 24576;    // bytes of a warp's ring
  static constexpr int kStages = kRing / (2 * kTile);
  static constexpr int kPitch = DH + 4;                 // of a row of O in shared memory
  static constexpr bool kQInSmem = NT == 4;
  static constexpr int kQBytes = kQInSmem ? NT * kK * 32 * 8 : 0;
  static constexpr int kSmem = NW * kRing + kQBytes + 1024;
  static_assert(NT * 8 * (kPitch + 4) * 4 <= kRing, "a warp's part fits in its ring");
  static_assert(kStages >= 3 && kStages < 32, "ring");
};

// The token of eight that is row n of a product.  A phase of eight lanes reads keys of
// rows 2 p and 2 p + 1, values of rows 0, 2, 4, 6 or 1, 3, 5, 7: rows of 128 bytes in
// their swizzle (chunk c of row r at c ^ (r mod 8)) want these two to differ in bit 2 and
// those four in bits 1 and 2, rows of 64 bytes (c ^ (r / 2 mod 4)) in bit 0 and in bits 0
// and 2.
template <int ROW>
__device__ __forceinline__ int token_of(int n) {
  const int t = n >> 1;
  const int even = ROW == 64 ? (t & 1) | ((t & 2) << 1) : 2 * t;
  return n & 1 ? even ^ (ROW == 64 ? 3 : 5) : even;
}
// Byte offset of 16-byte chunk c (of the first 128 bytes) of token row r in a tile.
template <int ROW>
__device__ __forceinline__ uint32_t place(int r, int c) {
  return ROW == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

template <bool CODES>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if (CODES)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t w;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(w) : "r"(v));
  return w;
}

template <bool CODES>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if (!CODES) return tc::pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// tanh of x, each value by the form for its size.
__device__ __forceinline__ float tanh_score(float x) {
  if (fabsf(x) <= kTanhTo)
    return Score<true, false>::odd(make_float2(x, x), 1.f, kTanh[0], kTanh[1], kTanh[2]).x;
  return Score<true, false>::tanh_large(x * (2.f * kLog2e));
}

template <int DH, bool CODES, int NT, bool PLAIN>
__global__ void __launch_bounds__(32 * NW, (Tok<DH, CODES, NT>::kTwo ? 2 : 1))
    token_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                 const __grid_constant__ PagedAttnArgs a, const TokenRuns runs) {
  using C = Tok<DH, CODES, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[NW][C::kStages];
  __shared__ int abort_word, entry, keys_of[kMostSorted];
  // The same offset in every block of a cluster: its blocks read each other's.
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile int* abort_flag = &abort_word;
  const PageArgs& pg = a.page;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cluster = runs.cluster, partials = runs.partials, splits = cluster * partials;
  const int nth = blockIdx.x / splits, split = blockIdx.x % splits;
  const int hkv = nth % a.Hkv, rows = a.H / a.Hkv * a.Nq;
  if (partials > 1) release_next();
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&mK);
    tc::tma_prefetch_desc(&mV);
  }
  int b = nth / a.Hkv;
  if (runs.sorted) {
    if (threadIdx.x < a.B) {
      int lo = INT_MAX, hi = 0;
      for (int i = 0; i < a.Nq; ++i) {
        const RowView v = row_view(a.ranges, a.q_pos, static_cast<size_t>(threadIdx.x) * a.Nq, i,
                                   a.Nk, a.causal);
        lo = min(lo, v.lo), hi = max(hi, v.hi);
      }
      keys_of[threadIdx.x] = lo < hi ? hi - lo : 0;
    }
    __syncthreads();
    if (threadIdx.x < a.B) {
      const int mine = keys_of[threadIdx.x];
      int rank = 0;
      for (int i = 0; i < a.B; ++i)
        rank += keys_of[i] > mine || (keys_of[i] == mine && i < static_cast<int>(threadIdx.x));
      if (rank == b) entry = threadIdx.x;
    }
    __syncthreads();
    b = entry;
  }
  const int group = b * a.Hkv + hkv;
  if (threadIdx.x < NW * C::kStages) tc::mbar_init(&full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) abort_word = 0;
  tc::fence_barrier_init();

  // What each row sees (lane r: row r), and their hull; the same in every warp.
  const GroupRow own = group_row(a, b, hkv, lane, rows);
  const int h_lo = warp_min(own.v.lo), h_hi = warp_max(own.v.hi);
  const int in_lo = warp_max(lane < rows ? own.v.lo : 0);
  const int in_hi = warp_min(lane < rows ? own.v.hi : INT_MAX);
  const int u_lo = h_lo < h_hi ? h_lo / kUnit : 0;
  const int u_n = h_lo < h_hi ? (h_hi + kUnit - 1) / kUnit - u_lo : 0;
  const int ub = u_lo + static_cast<int>(static_cast<long long>(u_n) * split / splits);
  const int ue = u_lo + static_cast<int>(static_cast<long long>(u_n) * (split + 1) / splits);
  const int first = ub + warp, count = ue > first ? (ue - first + NW - 1) / NW : 0;

  // Pages and scales of this warp's next 32 units, one a lane, and of the 32 behind.
  struct Meta {
    int slab;  // page and head; one past the last where there is nothing: zeros
    float ks, lv;
  };
  auto meta_of = [&](int n) {
    Meta m{pg.P * a.Hkv, 1.f, 0.f};
    if (n < count) {
      const int page = page_at(pg, b, (first + NW * n) * kUnit);
      if (page_ok(pg, page)) {
        m.slab = page * a.Hkv + hkv;
        if (CODES) {
          m.ks = pg.k_scale[m.slab];
          m.lv = __log2f(pg.v_scale[m.slab]);
        }
      }
    }
    return m;
  };
  Meta cur = meta_of(lane), nxt = meta_of(32 + lane);
  int batch = 0;
  __syncthreads();  // the barriers are there

  uint8_t* const ring = smem + warp * C::kRing;
  auto issue = [&](int n) {
    if (n < count) {
      const int slab = __shfl_sync(0xffffffffu, (n >> 5) == batch ? cur.slab : nxt.slab, n & 31);
      if (lane == 0) {
        const int s = n % C::kStages, y = ((first + NW * n) * kUnit) & (pg.T - 1);
        uint8_t* dst = ring + s * (2 * C::kTile);
        uint64_t* bar = &full[warp][s];
        tc::mbar_expect_tx(bar, 2 * C::kTile);
#pragma unroll
        for (int h = 0; h < C::kRow; h += 128) {
          tc::tma_load_3d(dst + h * kUnit, &mK, bar, h / 2, y, slab);
          tc::tma_load_3d(dst + C::kTile + h * kUnit, &mV, bar, h / 2, y, slab);
        }
      }
    }
  };
#pragma unroll
  for (int n = 0; n < C::kStages - 1; ++n) issue(n);

  // Q as the B operand: columns are rows 8 nt + g; lane t's elements of step (q, s) are
  // those of the key chunks that it reads.
  uint32_t qf[C::kQInSmem ? 1 : NT][C::kK][2];
  uint2* q_smem = reinterpret_cast<uint2*>(smem + NW * C::kRing);
  float c1[NT][2];  // from a product to the score: rows 8 nt + 2 t, + 1
  float slope2[NT][2];
  int pos[NT][2];
  const __nv_bfloat16* Q =
      static_cast<const __nv_bfloat16*>(a.Q) + static_cast<size_t>(group) * rows * DH;
  const float c0 = a.cap > 0.f ? a.tau / a.cap : a.tau * kLog2e, c2 = a.cap * kLog2e;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    uint2 w[C::kK];
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int q = k / (C::kRun / 4), s = k % (C::kRun / 4);
      w[k] = r < rows ? *reinterpret_cast<const uint2*>(Q + static_cast<size_t>(r) * DH +
                                                        (t + 4 * q) * C::kRun + 4 * s)
                      : make_uint2(0u, 0u);
      if (CODES) {
        const uint32_t e[4] = {w[k].x << 16, w[k].x & 0xFFFF0000u, w[k].y << 16,
                               w[k].y & 0xFFFF0000u};
#pragma unroll
        for (int i = 0; i < 4; ++i) most = fmaxf(most, finite_abs(__uint_as_float(e[i])));
      }
    }
    float shrink = 1.f;
    if (CODES) {
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      shrink = row_shrink(most);
#pragma unroll
      for (int k = 0; k < C::kK; ++k) {
        w[k].x = pack<true>(__uint_as_float(w[k].x << 16) * shrink,
                            __uint_as_float(w[k].x & 0xFFFF0000u) * shrink);
        w[k].y = pack<true>(__uint_as_float(w[k].y << 16) * shrink,
                            __uint_as_float(w[k].y & 0xFFFF0000u) * shrink);
      }
    }
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      if (C::kQInSmem) {
        if (warp == 0) q_smem[(nt * C::kK + k) * 32 + lane] = w[k];
      } else {
        qf[C::kQInSmem ? 0 : nt][k][0] = w[k].x;
        qf[C::kQInSmem ? 0 : nt][k][1] = w[k].y;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 8 * nt + 2 * t + j;
      c1[nt][j] = c0 / __shfl_sync(0xffffffffu, shrink, 4 * (2 * t + j));
      if (!PLAIN) {
        slope2[nt][j] = __shfl_sync(0xffffffffu, own.slope2, row);
        pos[nt][j] = __shfl_sync(0xffffffffu, own.v.pos, row);
      }
    }
  }
  if (C::kQInSmem) __syncthreads();

  float R[NT][2], l[NT][2], O[NT][C::kMT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    R[nt][0] = R[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < C::kMT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[nt][i][e] = 0.f;
  }

  // This lane's runs in a tile: keys of row g (and 8 further) in two halves of 64 bytes,
  // values of rows 2 t and 2 t + 1 (and 8 further).
  constexpr int kTok = C::kRow == 64 ? 64 : 128;  // bytes from token to token
  const int tok = token_of<C::kRow>(g), tok0 = token_of<C::kRow>(2 * t);
  const int tok1 = token_of<C::kRow>(2 * t + 1);
  const uint32_t k_at[2] = {place<C::kRow>(tok, t), place<C::kRow>(tok, t + 4)};
  const uint32_t v_at[2] = {
      C::kTile + (C::kRow == 64 ? place<64>(tok0, g >> 1) + 8 * (g & 1) : place<C::kRow>(tok0, g)),
      C::kTile + (C::kRow == 64 ? place<64>(tok1, g >> 1) + 8 * (g & 1) : place<C::kRow>(tok1, g))};
  bool ok = true;
  int n = 0;
  for (; n < count; ++n) {
    if ((n >> 5) != batch) {
      cur = nxt;
      nxt = meta_of(n + 32 + lane);
      batch = n >> 5;
    }
    issue(n + C::kStages - 1);
    ok = wait_warp(&full[warp][n % C::kStages], (n / C::kStages) & 1, abort_flag, a.err);
    if (!ok) break;
    const uint32_t kt = smem_u32(ring) + (n % C::kStages) * (2 * C::kTile);
    const int j0 = (first + NW * n) * kUnit;

    float S[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
#pragma unroll
    for (int q = 0; q < DH / (4 * C::kRun); ++q) {
      const uint32_t at = kt + k_at[q & 1] + (q >> 1) * (128 * kUnit);
      const uint4 x = lds16(at), y = lds16(at + 8 * kTok);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int s = 0; s < C::kRun / 4; ++s) {
        uint32_t f[4];
        if (CODES) {
          f[0] = codes_to_half2(static_cast<uint16_t>(xs[s]));
          f[1] = codes_to_half2(static_cast<uint16_t>(ys[s]));
          f[2] = codes_to_half2(static_cast<uint16_t>(xs[s] >> 16));
          f[3] = codes_to_half2(static_cast<uint16_t>(ys[s] >> 16));
        } else {
          f[0] = xs[2 * s % 4], f[1] = ys[2 * s % 4];
          f[2] = xs[(2 * s + 1) % 4], f[3] = ys[(2 * s + 1) % 4];
        }
        const int k = q * (C::kRun / 4) + s;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (C::kQInSmem) {
            const uint2 w = q_smem[(nt * C::kK + k) * 32 + lane];
            mma<CODES>(S[nt], f, w.x, w.y);
          } else {
            mma<CODES>(S[nt], f, qf[C::kQInSmem ? 0 : nt][k][0], qf[C::kQInSmem ? 0 : nt][k][1]);
          }
        }
      }
    }

    // Scores: element e of S[nt] is the token of row g + 8 (e / 2), row 8 nt + 2 t + e % 2.
    float ks = 1.f, lv = 0.f;
    if (CODES) {
      ks = __shfl_sync(0xffffffffu, cur.ks, n & 31);
      lv = __shfl_sync(0xffffffffu, cur.lv, n & 31);
    }
    const float inv_vs = CODES ? ex2_approx(-lv) : 1.f;
    const int j_of = j0 + tok;
    const bool masked = j0 < in_lo || j0 + kUnit > in_hi;
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j_of + 8 * (e >> 1);
        if (PLAIN) {
          S[nt][e] = fmaf(S[nt][e], c1[nt][e & 1] * ks, lv);
          continue;
        }
        float x = S[nt][e] * (c1[nt][e & 1] * ks);
        if (a.cap > 0.f) x = c2 * tanh_score(x);
        if (a.slopes)
          x = fmaf(-slope2[nt][e & 1], fabsf(static_cast<float>(j - pos[nt][e & 1])), x);
        S[nt][e] = x + lv;
      }
    if (masked) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int lo = __shfl_sync(0xffffffffu, own.v.lo, 8 * nt + 2 * t + e);
          const int hi = __shfl_sync(0xffffffffu, own.v.hi, 8 * nt + 2 * t + e);
          if (j_of < lo || j_of >= hi) S[nt][e] = -INFINITY;
          if (j_of + 8 < lo || j_of + 8 >= hi) S[nt][e + 2] = -INFINITY;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        raise = raise || fmaxf(S[nt][e], S[nt][e + 2]) > R[nt][e] + kRaise;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(S[nt][e], S[nt][e + 2]);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          m = fmaxf(R[nt][e], m);
          const PartFactor<CODES> pf(R[nt][e] == -INFINITY ? -INFINITY : R[nt][e] - m);
          const float f = pf.all();
          R[nt][e] = m;
          l[nt][e] = pf.of(l[nt][e]);
#pragma unroll
          for (int i = 0; i < C::kMT; ++i) {
            O[nt][i][e] *= f;
            O[nt][i][e + 2] *= f;
          }
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float base = R[nt][e & 1] == -INFINITY ? 0.f : R[nt][e & 1];  // nothing seen yet
        // Codes: as a square, whose root lasts where p is below 2^-126 (paged.cuh).  A
        // branch for pages with small scales took as long or longer.
        p[e] = ex2_approx(CODES ? 0.5f * (S[nt][e] - base) : S[nt][e] - base);
        l[nt][e & 1] = fmaf(CODES ? p[e] * inv_vs : 1.f, p[e], l[nt][e & 1]);
        if (CODES) p[e] *= p[e];
      }
      pb[nt][0] = transpose8(pack<CODES>(p[0], p[1]));
      pb[nt][1] = transpose8(pack<CODES>(p[2], p[3]));
    }

    // Values of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (v[0 .. 3]), this lane's columns: what
    // lies outside the hull may be anything and is made 0.
    constexpr int kWords = DH / 8 * (CODES ? 1 : 2) / 4;  // 32-bit words of a lane's columns
    uint32_t v[4][kWords];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = kt + v_at[i & 1] + (i >> 1) * (8 * kTok);
      if (kWords == 2) {
        const uint2 x = lds8(at);
        v[i][0] = x.x, v[i][1] = x.y;
      } else {
#pragma unroll
        for (int q = 0; q < kWords / 4; ++q) {
          const uint4 x = lds16(at + q * (128 * kUnit));
          v[i][4 * q] = x.x, v[i][4 * q + 1] = x.y, v[i][4 * q + 2] = x.z, v[i][4 * q + 3] = x.w;
        }
      }
    }
    if (j0 < h_lo || j0 + kUnit > h_hi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + (i & 1 ? tok1 : tok0) + 8 * (i >> 1);
        if (j < h_lo || j >= h_hi)
#pragma unroll
          for (int q = 0; q < kWords; ++q) v[i][q] = 0u;
      }
    }
    // Row tile i: rows g and g + 8 are the lane's columns 2 i and 2 i + 1 (column()).
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      uint32_t f[CODES ? 2 : 1][4];
      if (CODES) {
        const uint32_t x = __byte_perm(v[0][q], v[1][q], 0x5140);
        const uint32_t y = __byte_perm(v[0][q], v[1][q], 0x7362);
        const uint32_t z = __byte_perm(v[2][q], v[3][q], 0x5140);
        const uint32_t w = __byte_perm(v[2][q], v[3][q], 0x7362);
        f[0][0] = codes_to_half2(static_cast<uint16_t>(x));
        f[0][1] = codes_to_half2(static_cast<uint16_t>(x >> 16));
        f[0][2] = codes_to_half2(static_cast<uint16_t>(z));
        f[0][3] = codes_to_half2(static_cast<uint16_t>(z >> 16));
        f[CODES ? 1 : 0][0] = codes_to_half2(static_cast<uint16_t>(y));
        f[CODES ? 1 : 0][1] = codes_to_half2(static_cast<uint16_t>(y >> 16));
        f[CODES ? 1 : 0][2] = codes_to_half2(static_cast<uint16_t>(w));
        f[CODES ? 1 : 0][3] = codes_to_half2(static_cast<uint16_t>(w >> 16));
      } else {
        f[0][0] = __byte_perm(v[0][q], v[1][q], 0x5410);
        f[0][1] = __byte_perm(v[0][q], v[1][q], 0x7632);
        f[0][2] = __byte_perm(v[2][q], v[3][q], 0x5410);
        f[0][3] = __byte_perm(v[2][q], v[3][q], 0x7632);
      }
#pragma unroll
      for (int i = 0; i < (CODES ? 2 : 1); ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma<CODES>(O[nt][(CODES ? 2 : 1) * q + i], f[i], pb[nt][0], pb[nt][1]);
    }
    __syncwarp();  // the next copies overwrite this unit
  }
  if (!ok && lane == 0)  // what is under way has to land before the block ends
    for (int k = n; k < min(n + C::kStages, count); ++k)
      tc::drain_wait(&full[warp][k % C::kStages], (k / C::kStages) & 1);
  __syncwarp();

  // The warps' parts: O row by row, then R and l of each row.
  float* part = reinterpret_cast<float*>(smem + warp * C::kRing);
  constexpr int kRowsPadded = 8 * NT, kRL = kRowsPadded * C::kPitch;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[nt][e];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      const int row = 8 * nt + 2 * t + e;
      if (g == 0) {
        part[kRL + row] = R[nt][e];
        part[kRL + kRowsPadded + row] = s;
      }
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) {
        const int column = CODES ? DH / 8 * g + 2 * i : 64 * (i / 4) + 8 * g + 2 * (i % 4);
        *reinterpret_cast<float2*>(part + row * C::kPitch + column) =
            make_float2(O[nt][i][e], O[nt][i][e + 2]);
      }
    }
  __syncthreads();
  // Four columns of a row a thread: the warps' parts with their maximum as reference.
  constexpr int kQuads = DH / 4, kMine = (kRowsPadded * kQuads + 32 * NW - 1) / (32 * NW);
  float4 o[kMine];
  float m[kMine], sum[kMine];
  const float* w0 = reinterpret_cast<const float*>(smem);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int x = threadIdx.x + 32 * NW * i, row = x / kQuads, c = 4 * (x % kQuads);
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[i] = -INFINITY;
    sum[i] = 0.f;
    if (row >= rows) continue;
    constexpr int kStep = C::kRing / 4;
#pragma unroll
    for (int w = 0; w < NW; ++w) m[i] = fmaxf(m[i], w0[w * kStep + kRL + row]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* p = w0 + w * kStep;
      const float r = p[kRL + row];
      const PartFactor<CODES> pf(r == -INFINITY ? -INFINITY : r - m[i]);
      const float f = pf.all();
      const float4 v = *reinterpret_cast<const float4*>(p + row * C::kPitch + c);
      sum[i] = fmaf(pf.root, p[kRL + kRowsPadded + row] * (CODES ? pf.root : 1.f), sum[i]);
      o[i].x = fmaf(f, v.x, o[i].x), o[i].y = fmaf(f, v.y, o[i].y);
      o[i].z = fmaf(f, v.z, o[i].z), o[i].w = fmaf(f, v.w, o[i].w);
    }
  }
  // The same over the blocks of a cluster: block `rank` takes every cluster-th row.
  const int rank = split % cluster;
  if (cluster > 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int x = threadIdx.x + 32 * NW * i, row = x / kQuads, c = 4 * (x % kQuads);
      if (row >= rows) continue;
      float* p = reinterpret_cast<float*>(smem);
      *reinterpret_cast<float4*>(p + row * C::kPitch + c) = o[i];
      if (c == 0) *reinterpret_cast<float4*>(p + kRL + 4 * row) = make_float4(m[i], sum[i], 0.f, 0.f);
    }
    tc::cluster_sync();
    const uint32_t here = smem_u32(smem);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int x = threadIdx.x + 32 * NW * i, row = x / kQuads, c = 4 * (x % kQuads);
      if (row >= rows || row % cluster != rank) continue;
      m[i] = -INFINITY;
      sum[i] = 0.f;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < cluster; ++q)
        m[i] = fmaxf(m[i], tc::ld_shared_cluster_f4(
                               tc::mapa_shared(here + (kRL + 4 * row) * 4, q)).x);
      for (int q = 0; q < cluster; ++q) {
        const float4 ml = tc::ld_shared_cluster_f4(tc::mapa_shared(here + (kRL + 4 * row) * 4, q));
        const float4 v =
            tc::ld_shared_cluster_f4(tc::mapa_shared(here + (row * C::kPitch + c) * 4, q));
        const PartFactor<CODES> pf(ml.x == -INFINITY ? -INFINITY : ml.x - m[i]);
        const float f = pf.all();
        sum[i] = fmaf(pf.root, ml.y * (CODES ? pf.root : 1.f), sum[i]);
        o[i].x = fmaf(f, v.x, o[i].x), o[i].y = fmaf(f, v.y, o[i].y);
        o[i].z = fmaf(f, v.z, o[i].z), o[i].w = fmaf(f, v.w, o[i].w);
      }
    }
    tc::cluster_sync();  // no block leaves while its memory is read
  }
  const size_t all = static_cast<size_t>(a.B) * a.H * a.Nq;
  const size_t base = static_cast<size_t>(group) * rows;
  const Partials out = attn::partials(a.workspace, all, DH, partials);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int x = threadIdx.x + 32 * NW * i, row = x / kQuads, c = 4 * (x % kQuads);
    if (row >= rows || row % cluster != rank) continue;
    if (partials > 1) {
      const size_t at = split / cluster * all + base + row;
      *reinterpret_cast<float4*>(out.o + at * DH + c) = o[i];
      if (c == 0) out.ml[at] = make_float2(m[i], sum[i]);
    } else {
      const float inv = sum[i] > 0.f ? 1.f / sum[i] : 0.f;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + (base + row) * DH + c) =
          make_uint2(tc::pack_bf16x2(o[i].x * inv, o[i].y * inv),
                     tc::pack_bf16x2(o[i].z * inv, o[i].w * inv));
      if (c == 0) a.L[base + row] = (m[i] + __log2f(sum[i])) * kLn2;
    }
  }
}

bool token_supported(const PagedAttnArgs& a) {
  return a.bf16 && (a.d == 64 || a.d == 128) &&
         static_cast<long long>(a.H / a.Hkv) * a.Nq <= kMostRows;
}

// Blocks of an SM at a time (Tok::kTwo).
int token_blocks_per_sm(const PagedAttnArgs& a) {
  return a.H / a.Hkv * a.Nq <= 8 && (a.page.e4m3 || a.d == 64) ? 2 : 1;
}

TokenRuns token_runs(const PagedAttnArgs& a) {
  const long long groups = static_cast<long long>(a.B) * a.Hkv;
  const long long slots = static_cast<long long>(kSMs) * token_blocks_per_sm(a);
  const bool many = 2 * groups > slots;
  long long s = (many ? 2 * slots : slots) / groups;
  const long long most = a.Nk / 512;
  s = s > most ? most : s;
  s = s < 1 ? 1 : s;
  if (many) {
    const bool sorted = a.ranges && a.B > 1 && a.B <= kMostSorted && s * groups > slots;
    return {1, static_cast<int>(s), sorted ? 1 : 0};
  }
  return s <= 8 ? TokenRuns{static_cast<int>(s), 1, 0} : TokenRuns{8, static_cast<int>(s / 8), 0};
}

template <int DH, bool CODES, int NT, bool PLAIN>
cudaError_t launch(const PagedAttnArgs& a, const TokenRuns& runs) {
  using C = Tok<DH, CODES, NT>;
  const auto kernel = token_kernel<DH, CODES, NT, PLAIN>;
  CUtensorMap mk, mv;
  cudaError_t e = tc_map(&mk, a.K, a.page.P * a.Hkv, a.page.T, kUnit, DH, CODES);
  if (e == cudaSuccess) e = tc_map(&mv, a.V, a.page.P * a.Hkv, a.page.T, kUnit, DH, CODES);
  if (e == cudaSuccess) e = tc_set_smem(reinterpret_cast<const void*>(kernel), C::kSmem);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(a.B) * a.Hkv * runs.cluster * runs.partials;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_after(false, kernel, dim3(static_cast<unsigned>(grid)), 32 * NW, C::kSmem,
                      runs.cluster, a.stream, mk, mv, a, runs);
}

template <int DH, bool CODES>
cudaError_t launch(const PagedAttnArgs& a, const TokenRuns& runs) {
  const int rows = a.H / a.Hkv * a.Nq;
  const bool plain = a.cap == 0.f && !a.slopes;
  if (rows <= 8)
    return plain ? launch<DH, CODES, 1, true>(a, runs) : launch<DH, CODES, 1, false>(a, runs);
  if (rows <= 16)
    return plain ? launch<DH, CODES, 2, true>(a, runs) : launch<DH, CODES, 2, false>(a, runs);
  return plain ? launch<DH, CODES, 4, true>(a, runs) : launch<DH, CODES, 4, false>(a, runs);
}

cudaError_t token_attn(const PagedAttnArgs& a) {
  const TokenRuns runs = token_runs(a);
  cudaError_t e;
  if (a.d == 64) e = a.page.e4m3 ? launch<64, true>(a, runs) : launch<64, false>(a, runs);
  else e = a.page.e4m3 ? launch<128, true>(a, runs) : launch<128, false>(a, runs);
  return e == cudaSuccess && runs.partials > 1 ? attn_join(a, runs.partials) : e;
}

int splits_of(const PagedAttnArgs& a) {
  return token_supported(a) ? token_runs(a).partials
         : tc_paged_supported(a) ? tc_paged_splits(a) : simt_splits(a);
}

}  // namespace

size_t paged_workspace(const PagedAttnArgs& a) {
  const int splits = splits_of(a);
  return splits == 1 ? 0 : partial_bytes(static_cast<size_t>(a.B) * a.H * a.Nq, a.d, splits);
}

cudaError_t paged_attn(const PagedAttnArgs& a) {
  // The tensor-core forms multiply sums of codes by tau / cap, the page's scale and Q's at
  // once: fp32's smallest numbers times a cap beyond 2^80 would be seen in the scores.  A
  // workspace is by sizes alone, so no runs of keys then.
  if (a.page.e4m3 && a.cap > 0x1p80f) return simt_paged(a, 1);
  return token_supported(a)      ? token_attn(a)
         : tc_paged_supported(a) ? tc_paged(a)
                                 : simt_paged(a, simt_splits(a));
}

}  // namespace flashbob
