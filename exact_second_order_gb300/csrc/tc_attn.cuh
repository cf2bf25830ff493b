// Shared by the tensor-core kernels of attention with key ranges (bf16,
// d = 64 and 128): block numbering, what the 128 rows of a block see, and the
// score of a raw product in log2 units.
#pragma once

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace flashbob {
namespace attn {

// tanh x = x + x^3 (k0 + k1 x^2 + k2 x^4) for |x| <= kTanhTo, off by 1.9e-7:
// least squares with weights adapted until the largest error is smallest
// (Lawson's method).
__device__ constexpr float kTanh[3] = {-0.33326461911201477f, 0.13185861706733704f,
                                       -0.044229257851839066f};
constexpr float kTanhTo = 0.5f;

// rcp.approx (1 ulp) of a value in [1, inf]: 1 / inf is 0.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte
// aligned, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

// Orders this thread's view of global memory before its bulk copies from it.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Bounded waits that suspend the thread until the phase completes, or for
// kHintNs at a time.  The loops of the shared header read the global timer on
// entry and poll often; here a wake-up is what an MMA round trip waits for, and
// polling warps take issue slots from the working ones (4% of the gradient).
// As everywhere, a wait that gives up (2 s) records error code 1 and raises
// the flag that makes the others of the block give up.
constexpr uint32_t kHintNs = 1000000;
constexpr int kMaxTries = 2000;

__device__ __forceinline__ bool try_hint(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(kHintNs)
      : "memory");
  return ok != 0;
}
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity,
                                              volatile int* abort_flag, unsigned int* err) {
#pragma unroll 1
  for (int i = 0; i < kMaxTries; ++i) {
    if (try_hint(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  atomicExch(err, 1u);
  return false;
}
// One thread.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         unsigned int* err) {
  return try_hint(bar, parity) || wait_slow(bar, parity, abort_flag, err);
}
// A whole warp (all lanes wait; the vote keeps the result uniform).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned int* err) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, abort_flag, err));
}
// On two barriers: the polls are issued together, and only a barrier that is
// not there yet is waited for.
__device__ __forceinline__ bool wait_both_warp(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                               volatile int* abort_flag, unsigned int* err) {
  const bool ra = tc::mbar_try_wait(a, pa), rb = tc::mbar_try_wait(b, pb);
  const bool ok = (ra && rb) || ((ra || wait_slow(a, pa, abort_flag, err)) &&
                                 (rb || wait_slow(b, pb, abort_flag, err)));
  return __all_sync(0xffffffffu, ok);
}

// Row blocks are launched heads fastest and from the last rows of a head to
// the first, so that under a causal mask the long blocks start first and the
// short ones fill the end.  A rank is the r-th block of `blocks` row blocks
// of one group; the blocks of its G heads interleave when they do not
// straddle heads.
__device__ __forceinline__ int row_block(int rank, int blocks, int G, int Nq, int rows_per_block) {
  if (G > 1 && Nq % rows_per_block == 0) {
    const int per = Nq / rows_per_block;
    return (rank % G) * per + per - 1 - rank / G;
  }
  return blocks - 1 - rank;
}

// The view of one group row r (r >= rows: sees nothing) and its slope.
struct GroupRow {
  RowView v;
  float slope2;  // slope log2 e
};

__device__ __forceinline__ GroupRow group_row(const AttnArgs& a, int b, int hkv, int r, int rows) {
  GroupRow g{empty_view(), 0.f};
  if (r < rows) {
    const int h = r / a.Nq, i = r - h * a.Nq;
    g.v = row_view(a.ranges, a.q_pos, static_cast<size_t>(b) * a.Nq, i, a.Nk, a.causal);
    if (a.slopes) g.slope2 = a.slopes[hkv * (a.H / a.Hkv) + h] * kLog2e;
  }
  return g;
}

// Hull [lo, hi) and intersection [in_lo, in_hi) of the ranges of 128 rows
// (in_lo is INT_MAX when a row sees nothing, unless it lies beyond the last).
struct Hull {
  int lo, hi, in_lo, in_hi;
};

__device__ __forceinline__ void warp_hull(const RowView& v, bool live, int lane, int* out4) {
  const int lo = warp_min(v.lo), hi = warp_max(v.hi);
  const int in_lo = warp_max(live ? v.lo : 0), in_hi = warp_min(live ? v.hi : INT_MAX);
  if (lane == 0) {
    out4[0] = lo;
    out4[1] = hi;
    out4[2] = in_lo;
    out4[3] = in_hi;
  }
}

__device__ __forceinline__ Hull join_hulls(const int (*h)[4], int n) {
  Hull r{INT_MAX, 0, 0, INT_MAX};
  for (int i = 0; i < n; ++i) {
    r.lo = min(r.lo, h[i][0]);
    r.hi = max(r.hi, h[i][1]);
    r.in_lo = max(r.in_lo, h[i][2]);
    r.in_hi = min(r.in_hi, h[i][3]);
  }
  return r;
}

// Scores of raw products in log2 units:
//   not capped: raw c1;  capped: c2 t with t = tanh(raw tau / cap), which
//   tanh_of puts in place of the raw products;  biased: minus slope2 |j - pos|.
// tanh x is an odd polynomial for |x| <= 0.5, whose first term is x itself (2^-21
// relative with the roundings), beyond it 1 - 2 / (1 + e^{2 x}), two MUFU operations
// (2^-23 absolute).  The cap multiplies that error: up to a cap of kMufuCap a group
// of products with one beyond 0.5 takes the second form as a whole (at most 2^-17 of a
// score, less than the rounding of its dot product); above, each product takes the
// form of its own x, or a cap of 1e6 would cost 5% of O and one of 1e9 all of it.
// Where all of a warp's arguments are small (mostly: the cap is there for outliers)
// the polynomial runs alone, tau / cap in its coefficients, in 2.5 packed fp32
// instructions an element.  With the exponential of the softmax the second form would
// be three MUFU operations an element, and that pipe bounds the kernel: the forward of
// B1 H8 N16384 d64 took 1370 us with them, against 570 without a cap; 1100 with a
// polynomial to 0.7 (3.5 instructions, one more coefficient); now 921 and 516, and
// 1310 where every group of products has one beyond 0.5 (with a cap above kMufuCap
// 1540).
// (tanh.approx leaves 2^-11, which exp turns into percents of P.)
constexpr float kMufuCap = 64.f;

template <bool CAP, bool BIAS>
struct Score {
  float c1;      // tau log2 e; capped: tau / cap
  float c2;      // cap log2 e
  float slope2;
  float a1, a2, a3;  // capped: k0 c1^3, k1 c1^5, k2 c1^7
  float most_raw;    // the polynomial's range in raw products

  __device__ __forceinline__ Score(const AttnArgs& a, float slope) {
    c1 = CAP ? a.tau / a.cap : a.tau * kLog2e;
    c2 = a.cap * kLog2e;
    slope2 = slope;
    const float q = c1 * c1;
    a1 = kTanh[0] * (q * c1);
    a2 = kTanh[1] * (q * q * c1);
    a3 = kTanh[2] * (q * q * (q * c1));
    // Beyond these c1^7 or raw^2 would leave fp32's range: the products are
    // scaled first.
    most_raw = c1 >= 0x1p-16f && c1 <= 0x1p16f ? kTanhTo / c1 : -1.f;
  }
  static __device__ __forceinline__ float tanh_large(float x2) {  // of x2 / (2 log2 e)
    return fmaf(-2.f, rcp_approx(1.f + tc::ex2_approx(x2)), 1.f);
  }
  // v (k + a v^2 + b v^4 + c v^6)
  static __device__ __forceinline__ float2 odd(float2 v, float k, float a, float b, float c) {
    auto two = [](float x) { return make_float2(x, x); };
    const float2 w = tc::fmul2(v, v);
    float2 p = tc::ffma2(w, two(c), two(b));
    p = tc::ffma2(p, w, two(a));
    p = tc::ffma2(p, w, two(k));
    return tc::fmul2(v, p);
  }
  // Each product by the form of its own argument; `small`: of all that are
  // worked on together none is beyond 0.5.
  __device__ __forceinline__ float2 tanh_each(float2 raw, bool small) const {
    const float2 x = tc::fmul2(raw, make_float2(c1, c1));
    float2 t = odd(x, 1.f, kTanh[0], kTanh[1], kTanh[2]);
    if (small) return t;
    if (!(fabsf(x.x) <= kTanhTo)) t.x = tanh_large(x.x * (2.f * kLog2e));
    if (!(fabsf(x.y) <= kTanhTo)) t.y = tanh_large(x.y * (2.f * kLog2e));
    return t;
  }
  __device__ __forceinline__ float tanh_one(float raw) const {
    if (c2 <= kMufuCap * kLog2e) return tanh_large(raw * (2.f * kLog2e * c1));
    return tanh_each(make_float2(raw, raw), false).x;
  }
  // In `masked` tiles always each by its own: products that nobody sees must not
  // decide which form the others take, or they would reach last bits.
  template <int N>
  __device__ __forceinline__ void tanh_of(uint32_t (&s)[N][16], bool masked) const {
    if (!CAP) return;
    float most = 0.f;
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(tc::u2f(s[q][e])));
    if (__builtin_expect(masked || __any_sync(0xffffffffu, !(most <= most_raw)), 0)) {
      if (!masked && c2 <= kMufuCap * kLog2e) {
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[q][e] = __float_as_uint(tanh_large(tc::u2f(s[q][e]) * (2.f * kLog2e * c1)));
        return;
      }
      // `small` decides over instructions, not over any product's result.
      const bool small = __all_sync(0xffffffffu, most * c1 <= kTanhTo);
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 t = tanh_each(tc::f2(s[q][e], s[q][e + 1]), small);
          s[q][e] = __float_as_uint(t.x);
          s[q][e + 1] = __float_as_uint(t.y);
        }
      return;
    }
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 t = odd(tc::f2(s[q][e], s[q][e + 1]), c1, a1, a2, a3);
        s[q][e] = __float_as_uint(t.x);
        s[q][e + 1] = __float_as_uint(t.y);
      }
  }
  // raw or t, plus the bias at j - pos = dist; minus m.
  __device__ __forceinline__ float2 from(float2 x, float dist, float m, float slope) const {
    const float c = CAP ? c2 : c1;
    float2 s = tc::ffma2(x, make_float2(c, c), make_float2(-m, -m));
    if (BIAS) {
      s.x = fmaf(-slope, fabsf(dist), s.x);
      s.y = fmaf(-slope, fabsf(dist + 1.f), s.y);
    }
    return s;
  }
  // v (1 - t^2) when capped.
  static __device__ __forceinline__ float2 damp(float2 v, float2 t) {
    if (!CAP) return v;
    return tc::fmul2(v, tc::ffma2(t, make_float2(-t.x, -t.y), make_float2(1.f, 1.f)));
  }
};

// 128 x DH accumulator columns of TMEM lane r (NWG warpgroups share the
// columns), times `scale`, as bf16 rows in shared memory (pitch DH + 8:
// 16-byte accesses of 8 consecutive rows fall on all 32 banks), then to
// `rows` consecutive global rows with coalesced 16-byte stores.  `zero`: the
// accumulator was never written.  All elementwise threads, named barrier 1.
template <int DH, int NWG>
__device__ __forceinline__ void store_block(uint32_t acc, float scale, bool zero, uint8_t* stage,
                                            int wg, int r, int tid, int rows, bool ok,
                                            __nv_bfloat16* __restrict__ out) {
  constexpr int kPitch = DH * 2 + 16;
#pragma unroll
  for (int c = 0; c < DH / NWG; c += 16) {
    const int col = DH / NWG * wg + c;
    uint32_t v[16], w[8];
    tc::tmem_ld16(acc + col, v);
    tc::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k] = zero ? 0u : tc::pack_bf16x2(scale * tc::u2f(v[2 * k]), scale * tc::u2f(v[2 * k + 1]));
    uint4* d = reinterpret_cast<uint4*>(stage + r * kPitch + col * 2);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  tc::named_bar_sync(1, 128 * NWG);
  if (ok) {
    constexpr int kChunks = DH / 8;
    for (int f = tid; f < rows * kChunks; f += 128 * NWG)
      reinterpret_cast<uint4*>(out)[f] =
          *reinterpret_cast<const uint4*>(stage + (f / kChunks) * kPitch + (f % kChunks) * 16);
  }
}

// Row r of a 64-column tile in the 128-byte swizzle (16-byte chunk c at chunk
// c ^ (r mod 8)) as the A operand in TMEM: K step kk at columns 8 kk.
__device__ __forceinline__ void row_to_tmem(const uint8_t* tile, int r, uint32_t taddr) {
  const uint8_t* row = tile + r * 128;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + (((2 * kk) ^ (r & 7)) << 4));
    const uint4 b = *reinterpret_cast<const uint4*>(row + (((2 * kk + 1) ^ (r & 7)) << 4));
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    tc::tmem_st8(taddr + 8 * kk, v);
  }
}

// Zeroes row r (128 bytes in each 64-column half) of a tile in shared memory.
template <int NH, uint32_t HALF>
__device__ __forceinline__ void zero_row(uint8_t (*tile)[HALF], int r) {
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    uint4* v = reinterpret_cast<uint4*>(tile[h] + r * 128);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace attn
}  // namespace flashbob
