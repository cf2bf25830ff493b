// Norm of queries and keys for each head with the rotation by position, from
// the packed projection [B, N, H + 2 Hkv, d] to head-major Q, K, V, and its
// gradient:
//   r = rsqrt(mean(x^2) + eps),  y = x r w,
//   angle_k = sum_a pos_a f_ak,  (z_i, z_j) = the pair (y_i, y_j) turned by it;
//   dy = dz turned back,  dw = sum over rows of dy x r,  g = dy w,
//   dx = r (g - x r mean(g x r)).
//
// Every element is read and written once: memory bounds both directions.  A
// row (one head of one token) is taken by 8 lanes (d <= 64) or 16, four pairs
// each, so that both elements of a pair sit in one lane: the rotation needs
// no exchange and the row sums are three or four shuffles.  Angles are
// computed once for each token and pair and shared by its heads.
//
// Angles as fractions of a turn in 64-bit fixed point: f / (2 pi) mod 1 is
// scaled by 2^64 (from fp64, so to 2^-53), and the integer product with the
// position wraps as the angle does.  Its top 32 bits go to sincospif, so the
// angle of any position is exact to about 2^-24 of a half turn, which a
// product in 32 bits would lose from a position of a few hundred on.
#include <math.h>

#include "attn_common.cuh"

namespace flashbob {
namespace {
using namespace attn;

constexpr int NT = 256;
constexpr int kMaxAxes = 4;
constexpr int kGradBlocks = 4 * kSMs;  // blocks of the gradient: one partial dw each

// 2 pi / f turns ... the frequency as a 64-bit fraction of a turn per position.
__device__ __forceinline__ unsigned long long turn_step(float f) {
  double t = static_cast<double>(f) * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return static_cast<unsigned long long>(t * 18446744073709551616.0);
}

// (cos, sin) of every pair of one token.
__device__ __forceinline__ float2 turn(const unsigned long long* steps, int half, int k, int axes,
                                       const int* __restrict__ positions, size_t tokens,
                                       size_t token, int own) {
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

// Turn the lane's pairs by (cos, sin) of pairs 4 c ..; sign = -1 turns back.
__device__ __forceinline__ void rotate(float (&v)[8], const float2* cs, int c, int half,
                                       float sign) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (4 * c + u < half) {
      const float2 t = cs[4 * c + u];
      const float a = v[2 * u], b = v[2 * u + 1], sn = sign * t.y;
      v[2 * u] = a * t.x - b * sn;
      v[2 * u + 1] = b * t.x + a * sn;
    }
  }
}

// Tables of a block in dynamic shared memory: the steps [axes][half], then
// (cos, sin) of its tokens [TOK][half].
__device__ __forceinline__ void fill_steps(unsigned long long* steps, const NormArgs& a) {
  for (int k = threadIdx.x; k < a.axes * (a.R / 2); k += NT) steps[k] = turn_step(a.freqs[k]);
}

template <int TOK>
__device__ __forceinline__ void fill_turns(float2* cs, const unsigned long long* steps,
                                           const NormArgs& a, size_t token0, size_t tokens) {
  const int half = a.R / 2;
  for (int x = threadIdx.x; x < TOK * half; x += NT) {
    const size_t token = token0 + x / half;
    if (token < tokens)
      cs[x] = turn(steps, half, x % half, a.axes, a.positions, tokens, token,
                   static_cast<int>(token % a.N));
  }
}

// ---------------------------------------------------------------------------
// Forward.  A block takes TOK tokens; its row slots walk the heads and take
// TOK tokens of a head at a time, all loads before any arithmetic.
// ---------------------------------------------------------------------------
template <typename T, int LPR, bool VEC, int TOK>
__global__ void __launch_bounds__(NT) norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ unsigned long long smem[];
  const int half = a.R / 2;
  float2* cs = reinterpret_cast<float2*>(smem + a.axes * half);
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const size_t token0 = static_cast<size_t>(blockIdx.x) * TOK;
  const Shape s{a.d, half, a.interleaved};
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, heads = a.H + 2 * a.Hkv;
  const T* X = static_cast<const T*>(a.QKV);

  fill_steps(smem, a);
  __syncthreads();
  fill_turns<TOK>(cs, smem, a, token0, tokens);
  __syncthreads();
  // A warp's slots run the same number of steps: the shuffles need all lanes.
  for (int h0 = 0; h0 < heads; h0 += NT / LPR) {
    const int h = h0 + slot;
    float v[TOK][8];
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      if (h < heads && token0 + u < tokens) {
        load_row<VEC>(X + ((token0 + u) * heads + h) * a.d, s, c, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
      }
    }
    const bool is_q = h < a.H, is_v = h >= a.H + a.Hkv;
    const float* gain = is_q ? a.wq : a.wk;
    float w[8];
    if (gain && !is_v) load_row<VEC>(gain, s, c, w);
    else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
    }
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(v[u][e], v[u][e], sq);
      sq = row_sum<LPR>(sq);
      if (!is_v) {
        const float r = rsqrtf(sq / a.d + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = v[u][e] * r * w[e];
        rotate(v[u], cs + u * half, c, half, 1.f);
      }
      if (h >= heads || token0 + u >= tokens) continue;
      const int b = static_cast<int>((token0 + u) / a.N), n = static_cast<int>((token0 + u) % a.N);
      if (is_q) {
        store_row<VEC>(static_cast<T*>(a.Q) + ((static_cast<size_t>(b) * a.H + h) * a.N + n) * a.d,
                       s, c, v[u]);
      } else {
        const int hk = is_v ? h - a.H - a.Hkv : h - a.H;
        const long long row = static_cast<long long>(n) + (a.kv_start ? a.kv_start[b] : 0);
        if (row >= 0 && row < a.Nk)  // a row outside the cache is dropped
          store_row<VEC>(static_cast<T*>(is_v ? a.V : a.K) +
                             ((static_cast<size_t>(b) * a.Hkv + hk) * a.Nk + row) * a.d,
                         s, c, v[u]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient.  A fixed number of blocks walks the tokens; each lane keeps dw of
// its eight columns for q and k, the block sums its row slots in order and
// leaves one partial, and a second kernel sums the partials in order: the
// result does not depend on timing.
// ---------------------------------------------------------------------------
template <typename T, typename TG, int LPR, bool VEC, int TOK>
__global__ void __launch_bounds__(NT) norm_grad_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ unsigned long long smem[];
  __shared__ float part[NT * 8];
  const int half = a.R / 2;
  float2* cs = reinterpret_cast<float2*>(smem + a.axes * half);
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const Shape s{a.d, half, a.interleaved};
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, heads = a.H + 2 * a.Hkv;
  const T* X = static_cast<const T*>(a.QKV);
  T* dX = static_cast<T*>(a.dQKV);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;

  fill_steps(smem, a);
  for (size_t token0 = static_cast<size_t>(blockIdx.x) * TOK; token0 < tokens;
       token0 += static_cast<size_t>(gridDim.x) * TOK) {
    __syncthreads();
    fill_turns<TOK>(cs, smem, a, token0, tokens);
    __syncthreads();
    for (int h0 = 0; h0 < heads; h0 += NT / LPR) {
      const int h = h0 + slot;
      const bool is_q = h < a.H, is_v = h >= a.H + a.Hkv;
      const int hk = is_v ? h - a.H - a.Hkv : h - a.H;
      float x[TOK][8], g[TOK][8];
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = g[u][e] = 0.f;
        if (h < heads && token0 + u < tokens) {
          const size_t b = (token0 + u) / a.N, n = (token0 + u) % a.N;
          const TG* dz = static_cast<const TG*>(is_q ? a.Q : is_v ? a.V : a.K) +
                         ((is_q ? b * a.H + h : b * a.Hkv + hk) * a.N + n) * a.d;
          load_row<VEC>(dz, s, c, g[u]);
          if (!is_v) load_row<VEC>(X + ((token0 + u) * heads + h) * a.d, s, c, x[u]);
        }
      }
      const float* gain = is_q ? a.wq : a.wk;
      float w[8];
      if (gain && !is_v) load_row<VEC>(gain, s, c, w);
      else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(x[u][e], x[u][e], sq);
        const float r = rsqrtf(row_sum<LPR>(sq) / a.d + a.eps);
        float dot = 0.f;
        if (!is_v) {
          rotate(g[u], cs + u * half, c, half, -1.f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[u][e] *= r;
            const float y = g[u][e] * x[u][e];
            dw[0][e] += is_q ? y : 0.f;
            dw[1][e] += is_q ? 0.f : y;
            g[u][e] *= w[e];
            dot = fmaf(g[u][e], x[u][e], dot);
          }
        }
        dot = row_sum<LPR>(dot) / a.d;
        if (!is_v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[u][e] = r * (g[u][e] - x[u][e] * dot);
        }
        if (h < heads && token0 + u < tokens)
          store_row<VEC>(dX + ((token0 + u) * heads + h) * a.d, s, c, g[u]);
      }
    }
  }
  if (a.dwq == nullptr) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[(slot * LPR + c) * 8 + e] = dw[k][e];
    __syncthreads();
    for (int x = threadIdx.x; x < LPR * 8; x += NT) {
      float sum = 0.f;
      for (int q = 0; q < NT / LPR; ++q) sum += part[q * LPR * 8 + x];
      // Position x of the lanes' order; the sum kernel puts it in place.
      a.workspace[(static_cast<size_t>(blockIdx.x) * 2 + k) * 128 + x] = sum;
    }
  }
}

// dw[k][element] = the sum of the blocks' partials in their order.  256
// threads: 32 columns by 8 runs of partials, joined in order.
__global__ void __launch_bounds__(NT) norm_dw_kernel(const float* __restrict__ part, int blocks,
                                                     float* __restrict__ dwq,
                                                     float* __restrict__ dwk, int d, int half,
                                                     int interleaved, int vec) {
  __shared__ float s[8][32];
  const int k = blockIdx.y, x = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float sum = 0.f;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * run / 8);
  const int b1 = static_cast<int>(static_cast<long long>(blocks) * (run + 1) / 8);
  for (int b = b0; b < b1; ++b) sum += part[(static_cast<size_t>(b) * 2 + k) * 128 + x];
  s[run][threadIdx.x & 31] = sum;
  __syncthreads();
  if (run) return;
  sum = 0.f;
  for (int q = 0; q < 8; ++q) sum += s[q][threadIdx.x];
  const Shape sh{d, half, interleaved != 0};
  // Element e = x % 8 of lane x / 8: pair 4 (x / 8) + e / 2.
  const int2 at = pair_at(sh, 4 * (x >> 3) + ((x & 7) >> 1));
  const int col = x & 1 ? at.y : at.x;
  if (col < d) (k ? dwk : dwq)[col] = sum;
}

template <typename T, int LPR, bool VEC, int TOK>
cudaError_t forward(const NormArgs& a) {
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const size_t smem = static_cast<size_t>(a.R / 2) * (8 * a.axes + 8 * TOK);
  norm_kernel<T, LPR, VEC, TOK>
      <<<static_cast<unsigned>((tokens + TOK - 1) / TOK), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}

bool vec_ok(const NormArgs& a) { return a.d % 8 == 0 && a.R % 8 == 0; }

template <typename T>
cudaError_t forward(const NormArgs& a) {
  // Four tokens a block once there are enough blocks to fill the GPU twice.
  const bool many = static_cast<size_t>(a.B) * a.N >= 4u * 2u * kSMs;
  if (a.d <= 64) {
    if (vec_ok(a)) return many ? forward<T, 8, true, 4>(a) : forward<T, 8, true, 1>(a);
    return many ? forward<T, 8, false, 4>(a) : forward<T, 8, false, 1>(a);
  }
  if (vec_ok(a)) return many ? forward<T, 16, true, 4>(a) : forward<T, 16, true, 1>(a);
  return many ? forward<T, 16, false, 4>(a) : forward<T, 16, false, 1>(a);
}

constexpr int kGradTok = 2;

unsigned grad_blocks(const NormArgs& a) {
  const size_t n = (static_cast<size_t>(a.B) * a.N + kGradTok - 1) / kGradTok;
  return static_cast<unsigned>(n < kGradBlocks ? n : kGradBlocks);
}

template <typename T, typename TG, int LPR, bool VEC>
cudaError_t backward(const NormArgs& a) {
  const unsigned blocks = grad_blocks(a);
  const size_t smem = static_cast<size_t>(a.R / 2) * (8 * a.axes + 8 * kGradTok);
  norm_grad_kernel<T, TG, LPR, VEC, kGradTok><<<blocks, NT, smem, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.dwq == nullptr) return e;
  norm_dw_kernel<<<dim3(LPR / 4, 2), NT, 0, a.stream>>>(a.workspace, static_cast<int>(blocks),
                                                        a.dwq, a.dwk, a.d, a.R / 2,
                                                        a.interleaved ? 1 : 0, VEC ? 1 : 0);
  return cudaGetLastError();
}

template <typename T, typename TG>
cudaError_t backward(const NormArgs& a) {
  if (a.d <= 64) return vec_ok(a) ? backward<T, TG, 8, true>(a) : backward<T, TG, 8, false>(a);
  return vec_ok(a) ? backward<T, TG, 16, true>(a) : backward<T, TG, 16, false>(a);
}

}  // namespace

size_t norm_grad_workspace(const NormArgs& a) {
  return a.wq ? static_cast<size_t>(grad_blocks(a)) * 2 * 128 * sizeof(float) : 0;
}

cudaError_t qk_norm(const NormArgs& a) {
  return a.bf16 ? forward<__nv_bfloat16>(a) : forward<float>(a);
}

cudaError_t qk_norm_grad(const NormArgs& a) {
  if (a.bf16)
    return a.grad_bf16 ? backward<__nv_bfloat16, __nv_bfloat16>(a)
                       : backward<__nv_bfloat16, float>(a);
  return a.grad_bf16 ? backward<float, __nv_bfloat16>(a) : backward<float, float>(a);
}

}  // namespace flashbob
