// Shared by the kernels of the paged cache: where a token lies, and the numbers
// of an 8-bit cache.
//
// e4m3 with one scale for each page and head, a power of two in 2^-60 .. 2^60: the
// least whose 448-fold (e4m3's largest number) is no less than the largest finite
// magnitude.  A power of two costs no precision of a floating-point number (only the
// reach of its smallest ones, at most one of its 15 binades), a value times its scale
// is exact in bf16 and fp32, and codes move to a larger scale without a rounding
// unless they become subnormal.
#pragma once

#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace flashbob {
namespace paged {

constexpr int kLeastExp = -60, kMostExp = 60;

// Row (of d elements) of token j of batch entry b in a pool, or -1: a table entry
// outside 0 .. P - 1 is a page of zeros, so that no table can lead out of the pool.
__device__ __forceinline__ int page_at(const PageArgs& p, int b, int j) {
  return p.table[static_cast<size_t>(b) * p.M + (j >> p.shift)];
}
__device__ __forceinline__ bool page_ok(const PageArgs& p, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(p.P);
}
__device__ __forceinline__ size_t page_row(const PageArgs& p, int page, int Hkv, int hkv, int j) {
  return ((static_cast<size_t>(page) * Hkv + hkv) << p.shift) + (j & (p.T - 1));
}

// The scale for a largest finite magnitude.
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t bits = __float_as_uint(most);  // 1.f x 2^(e - 127); 448 = 1.75 2^8
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(kLeastExp, min(kMostExp, e)) + 127) << 23);
}
// A scale that a page has, whatever the array holds.
__device__ __forceinline__ float held_scale(float s) {
  return fminf(fmaxf(s, 0x1p-60f), 0x1p60f);
}

// The weights of the tensor-core forms are p = exp2(x + log2 s_V - R), with R >= the
// largest x + log2 s_V - 8, and a row's sum is that of exp2(x - R).  So a sum is at least
// the largest scale's inverse, 2^-60; but p of a page with a small scale s_V falls below
// fp32's least 2^-126 where exp2(x - R) is still 2^-126 / s_V, and that may be most of the
// sum (pages of zeros have the least scale, 2^-60).  For few rows p is a square there,
// whose root does not leave fp32's reach.  For many, where every exponential counts,
// p / s_V is added for scales from 2^-20 on (what it loses is 2^-46 of the sum at most:
// nothing that a row of 2^20 keys would notice), and the others get a second exponential.
constexpr float kLeastLog = -20.f;

// Parts of a row meet with factors 2^d (d <= 0).  With codes, whose references hold their
// pages' scales, a part's sum of weights may count although its factor is below 2^-126: the
// factor is a square, too, and its root taken twice.  What a factor below 2^-126 leaves of
// products with V is nothing beside the nearer part's.
template <bool CODES>
struct PartFactor {
  float root;
  __device__ __forceinline__ explicit PartFactor(float d)
      : root(tc::ex2_approx(CODES ? 0.5f * d : d)) {}
  __device__ __forceinline__ float all() const { return CODES ? root * root : root; }
  __device__ __forceinline__ float of(float l) const { return CODES ? l * root * root : l * root; }
};

// |x| for the largest magnitude: NaN and infinity do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float y = fabsf(x);
  return y <= 3.402823466e38f ? y : 0.f;
}

// Two values to codes (x in the low byte) and back; beyond 448 (and infinite): 448.
__device__ __forceinline__ uint32_t to_codes(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ float2 from_codes(uint32_t c) {
  const uint32_t h = codes_to_half2(static_cast<uint16_t>(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^-e for a row whose largest finite magnitude is in [2^e, 2^(e + 1)), 1 for a row of
// zeros: scales it into fp16's reach.
__device__ __forceinline__ float row_shrink(float most) {
  const int e = static_cast<int>(__float_as_uint(most) >> 23);
  return e == 0 ? 1.f : __uint_as_float(static_cast<uint32_t>(max(254 - e, 1)) << 23);
}

}  // namespace paged
}  // namespace flashbob
