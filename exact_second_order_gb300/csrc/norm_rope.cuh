// Shared by the kernels that turn queries and keys by position: the angles as
// fractions of a turn, and a row of a head as pairs in a few lanes.
#pragma once

#include "attn_common.cuh"

namespace flashbob {
namespace rope {
using namespace attn;

// Angles as fractions of a turn in 64-bit fixed point: f / (2 pi) mod 1 is
// scaled by 2^64, and the integer product with the position wraps as the angle
// does.  Its top 32 bits go to sincospif, so the
// angle of any position is exact to about 2^-24 of a half turn, which a
// product in 32 bits would lose from a position of a few hundred on.

// f / (2 pi) turns per position, as a fraction of a turn in 64 bits: the 24-bit
// significand m of f = m 2^e times 2^66 / (2 pi) (64 bits, so to 2^-64), shifted
// to 2^64 units of a turn.  (In fp64, whose rate here is a hundredth of fp32's,
// this took longer than a short call's memory traffic.)
__device__ __forceinline__ unsigned long long turn_step(float f) {
  constexpr unsigned long long kInv2Pi = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(f), ex = (bits >> 23) & 255u;
  const unsigned long long m = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int shift = 152 - static_cast<int>(ex ? ex : 1);  // right, of the 88-bit product
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  unsigned long long t;
  if (shift <= 0) t = shift > -64 ? lo << -shift : 0;
  else if (shift < 64) t = (lo >> shift) | (hi << (64 - shift));
  else t = shift < 128 ? hi >> (shift - 64) : 0;
  return bits >> 31 ? 0 - t : t;
}

// (cos, sin) of every pair of one token.
__device__ __forceinline__ float2 turn(const unsigned long long* steps, int half, int k, int axes,
                                       const int* __restrict__ positions, size_t tokens,
                                       size_t token, long long own) {
  unsigned long long phase = 0;
  for (int a = 0; a < axes; ++a) {
    const long long p = positions ? positions[a * tokens + token] : own;
    phase += static_cast<unsigned long long>(p) * steps[a * half + k];
  }
  float2 cs;
  sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &cs.y, &cs.x);
  return cs;
}

// The eight elements (four pairs) of lane `c` of a row, as pairs
// (v[2 u], v[2 u + 1]).  VEC: d and R are multiples of 8, so that a lane's
// pairs are all rotated or none and its elements are two or one aligned runs;
// otherwise element by element, absent ones 0.
struct Shape {
  int d, half;  // half = R / 2 rotated pairs
  bool interleaved;
};

// First and second element of pair p: rotated pairs first, the rest in order.
__device__ __forceinline__ int2 pair_at(const Shape& s, int p) {
  if (p < s.half && !s.interleaved) return make_int2(p, p + s.half);
  return make_int2(2 * p, 2 * p + 1);  // 2 half = R, so the rest follows on
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ x, const Shape& s, int c,
                                         float (&v)[8]) {
  if (VEC) {
    if (8 * c >= s.d) {
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = 0.f;
    } else if (4 * c < s.half && !s.interleaved) {
      const float4 a = ld4(x + 4 * c), b = ld4(x + s.half + 4 * c);
      v[0] = a.x, v[2] = a.y, v[4] = a.z, v[6] = a.w;
      v[1] = b.x, v[3] = b.y, v[5] = b.z, v[7] = b.w;
    } else {
      const float4 a = ld4(x + 8 * c), b = ld4(x + 8 * c + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int2 at = pair_at(s, 4 * c + u);
      v[2 * u] = at.x < s.d ? to_f(x[at.x]) : 0.f;
      v[2 * u + 1] = at.y < s.d ? to_f(x[at.y]) : 0.f;
    }
  }
}

__device__ __forceinline__ void st4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, float a, float b, float c, float d) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T* __restrict__ x, const Shape& s, int c,
                                          const float (&v)[8]) {
  if (VEC) {
    if (8 * c >= s.d) return;
    if (4 * c < s.half && !s.interleaved) {
      st4(x + 4 * c, v[0], v[2], v[4], v[6]);
      st4(x + s.half + 4 * c, v[1], v[3], v[5], v[7]);
    } else {
      st4(x + 8 * c, v[0], v[1], v[2], v[3]);
      st4(x + 8 * c + 4, v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int2 at = pair_at(s, 4 * c + u);
      if (at.x < s.d) put(x + at.x, v[2 * u]);
      if (at.y < s.d) put(x + at.y, v[2 * u + 1]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Turn the lane's pairs by (cos, sin); SIGN = -1 turns back.  Pairs that do not
// turn have (1, 0).
template <int SIGN>
__device__ __forceinline__ void rotate(float (&v)[8], const float2 (&cs)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float a = v[2 * u], b = v[2 * u + 1], sn = SIGN * cs[u].y;
    v[2 * u] = a * cs[u].x - b * sn;
    v[2 * u + 1] = b * cs[u].x + a * sn;
  }
}

__device__ __forceinline__ void fill_steps(unsigned long long* steps, const NormArgs& a) {
  for (int k = threadIdx.x; k < a.axes * (a.R / 2); k += blockDim.x) steps[k] = turn_step(a.freqs[k]);
  __syncthreads();
}

__device__ __forceinline__ void token_turns(float2 (&cs)[4], const unsigned long long* steps,
                                            const NormArgs& a, int c, size_t tokens,
                                            size_t token, long long own) {
  const int half = a.R / 2;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    cs[u] = 4 * c + u < half
                ? turn(steps, half, 4 * c + u, a.axes, a.positions, tokens, token, own)
                : make_float2(1.f, 0.f);
}

// The lane's eight elements as loaded, unpacked at use: fewer registers for
// rows in flight.
template <typename T, bool VEC>
struct Raw {
  float v[8];
  __device__ __forceinline__ void load(const T* x, const Shape& s, int c) {
    load_row<VEC>(x, s, c, v);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.f;
  }
  __device__ __forceinline__ void get(float (&o)[8], const Shape&, int) const {
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = v[u];
  }
};
template <>
struct Raw<__nv_bfloat16, true> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* x, const Shape& s, int c) {
    if (8 * c >= s.d) return zero();
    const bool apart = 4 * c < s.half && !s.interleaved;
    a = *reinterpret_cast<const uint2*>(x + (apart ? 4 * c : 8 * c));
    b = *reinterpret_cast<const uint2*>(x + (apart ? s.half + 4 * c : 8 * c + 4));
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(float (&o)[8], const Shape& s, int c) const {
    const float4 x = make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
                                 __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u));
    const float4 y = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u),
                                 __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
    if (4 * c < s.half && !s.interleaved) {
      o[0] = x.x, o[2] = x.y, o[4] = x.z, o[6] = x.w;
      o[1] = y.x, o[3] = y.y, o[5] = y.z, o[7] = y.w;
    } else {
      o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
      o[4] = y.x, o[5] = y.y, o[6] = y.z, o[7] = y.w;
    }
  }
};

// Vector accesses: a lane's elements are one aligned run (neighbouring pairs),
// or two when the halves of its pairs are, and all of them turn or none.
inline bool vec_ok(const NormArgs& a) { return a.d % 8 == 0 && (a.interleaved || a.R % 8 == 0); }

}  // namespace rope
}  // namespace flashbob
