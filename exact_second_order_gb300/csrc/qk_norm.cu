// Norm of queries and keys for each head with the rotation by position, from
// the packed projection [B, N, H + 2 Hkv, d] to head-major Q, K, V, and its
// gradient:
//   r = rsqrt(mean(x^2) + eps),  y = x r w,
//   angle_k = sum_a pos_a f_ak,  (z_i, z_j) = the pair (y_i, y_j) turned by it;
//   dy = dz turned back,  dw = sum over rows of dy x r,  g = dy w,
//   dx = r (g - x r mean(g x r)).
//
// Every element is read and written once: memory bounds both directions.  A
// token is taken by 8 lanes (d <= 64) or 16, each with four pairs of every
// head's row, so both elements of a pair sit in one lane, the row sums are three
// or four shuffles, and the token's cosines and sines stay in 8 registers while
// its heads stream past, several rows in flight (a block of 4 tokens with the
// angles in shared memory, computed before the first load, ran at 2.1 TB/s).
// Neighbouring tokens of a block write neighbouring rows of a head.
// Measured (16384 tokens, 32 + 2 * 8 heads of 128, bf16): 76 us forward, 79% of
// the copy rate, 118 us gradient, 72% (x of the value heads is not read), and 5 us
// for the sum of dw.  Bound by both the bytes in flight and the
// issue (63% and 49% of the slots before the gradient loaded ahead): with the
// rows in rings in shared memory 91 and 136 us, with 16 elements a lane 79 and
// 140, with packed fp32 87 and 130 (graph replays, 81 and 124 for this).
#include <math.h>

#include <type_traits>

#include "norm_rope.cuh"

namespace flashbob {
namespace {
using namespace rope;

constexpr int NT = 256;
constexpr int kMaxAxes = 4;
constexpr unsigned kForwardBlocks = 8 * kSMs;
constexpr unsigned kGradBlocks = 2 * kSMs;  // along the tokens; one partial dw a block

// Which of a token's heads a block takes: part blockIdx.y of gridDim.y of the
// query heads, of the key heads and of the value heads.
__device__ __forceinline__ int2 head_part(int heads) {
  return make_int2(heads * static_cast<int>(blockIdx.y) / static_cast<int>(gridDim.y),
                   heads * (static_cast<int>(blockIdx.y) + 1) / static_cast<int>(gridDim.y));
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
constexpr int kRows = 4;  // rows in flight of each lane, with 64 registers and 4 blocks an SM:
                         // 81 us (16384 tokens, 48 heads of 128); 8 rows and 2 blocks 91 us

template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(NT, 4) norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ unsigned long long steps[];
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const Shape s{a.d, a.R / 2, a.interleaved};
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, heads = a.H + 2 * a.Hkv;
  constexpr int kSlots = NT / LPR;
  const float inv_d = 1.f / a.d;
  fill_steps(steps, a);
  // The lanes of a warp stay together (the shuffles need them all); a slot
  // without a token only loads and stores nothing.
  for (size_t first = static_cast<size_t>(blockIdx.x) * kSlots; first < tokens;
       first += static_cast<size_t>(gridDim.x) * kSlots) {
    const size_t token = first + slot;
    const bool live = token < tokens;
    const size_t b = live ? token / a.N : 0, n = live ? token % a.N : 0;
    const T* X = static_cast<const T*>(a.QKV) + (live ? token : 0) * heads * a.d;
    const long long kv = static_cast<long long>(n) + (a.kv_start && live ? a.kv_start[b] : 0);
    const bool kept = kv >= 0 && kv < a.Nk;  // a row outside the cache is dropped
    float2 cs[4];
    bool turned = false;
    auto run = [&](auto kind, int nh, int h0, T* out, size_t pitch, const float* gain, bool keep) {
      constexpr int kKind = decltype(kind)::value;  // 0 query, 1 key, 2 value
      const int2 part = head_part(nh);
      float w[8];
      if (kKind < 2 && gain) load_row<VEC>(gain, s, c, w);
      for (int h = part.x; h < part.y; h += kRows) {
        Raw<T, VEC> x[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (live && h + u < part.y) x[u].load(X + static_cast<size_t>(h0 + h + u) * a.d, s, c);
          else x[u].zero();
        }
        if (kKind < 2 && !turned) {  // behind the first loads
          token_turns(cs, steps, a, c, tokens, live ? token : 0, static_cast<long long>(n));
          turned = true;
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          float v[8];
          x[u].get(v, s, c);
          if (kKind < 2) {
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(v[e], v[e], sq);
            const float r = rsqrtf(fmaf(row_sum<LPR>(sq), inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = gain ? v[e] * r * w[e] : v[e] * r;
            rotate<1>(v, cs);
          }
          if (live && keep && h + u < part.y) store_row<VEC>(out + (h + u) * pitch, s, c, v);
        }
      }
    };
    T* Q = static_cast<T*>(a.Q) + (b * a.H * a.N + n) * a.d;
    const size_t kvrow = (b * a.Hkv * static_cast<size_t>(a.Nk) + (kept ? kv : 0)) * a.d;
    const size_t kvpitch = static_cast<size_t>(a.Nk) * a.d;
    run(std::integral_constant<int, 0>(), a.H, 0, Q, static_cast<size_t>(a.N) * a.d, a.wq, true);
    run(std::integral_constant<int, 1>(), a.Hkv, a.H, static_cast<T*>(a.K) + kvrow, kvpitch, a.wk,
        kept);
    run(std::integral_constant<int, 2>(), a.Hkv, a.H + a.Hkv, static_cast<T*>(a.V) + kvrow, kvpitch,
        nullptr, kept);
  }
}

// ---------------------------------------------------------------------------
// Gradient.  A fixed number of blocks walks the tokens; each lane keeps dw of
// its eight columns for q and k, the block sums its slots in order and leaves
// one partial, and a second kernel sums the partials in order: the result does
// not depend on timing.
// ---------------------------------------------------------------------------
// Rows of x and of dz that each lane works on, with as many of the next ones in
// flight and 2 blocks an SM: 124 us (16384 tokens, 48 heads of 128); 2 rows 129, 4
// rows 136, 4 rows loaded and then worked on 134, 2 rows and 3 blocks 179.
constexpr int kGradRows = 3;

template <typename T, typename TG, int LPR, bool VEC>
__global__ void __launch_bounds__(NT, 2) norm_grad_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ unsigned long long steps[];
  __shared__ float part_dw[NT * 8];
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const Shape s{a.d, a.R / 2, a.interleaved};
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, heads = a.H + 2 * a.Hkv;
  constexpr int kSlots = NT / LPR;
  const float inv_d = 1.f / a.d;
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  if (a.dwq) release_next();
  fill_steps(steps, a);
  for (size_t first = static_cast<size_t>(blockIdx.x) * kSlots; first < tokens;
       first += static_cast<size_t>(gridDim.x) * kSlots) {
    const size_t token = first + slot;
    const bool live = token < tokens;
    const size_t b = live ? token / a.N : 0, n = live ? token % a.N : 0;
    const T* X = static_cast<const T*>(a.QKV) + (live ? token : 0) * heads * a.d;
    T* dX = static_cast<T*>(a.dQKV) + (live ? token : 0) * heads * a.d;
    const size_t pitch = static_cast<size_t>(a.N) * a.d;
    float2 cs[4];
    bool turned = false;
    auto run = [&](auto kind, int nh, int h0, const TG* dz, const float* gain) {
      constexpr int kKind = decltype(kind)::value;
      const int2 part = head_part(nh);
      float w[8];
      if (kKind < 2 && gain) load_row<VEC>(gain, s, c, w);
      Raw<T, VEC> nx[kGradRows];
      Raw<TG, VEC> ng[kGradRows];
      auto fetch = [&](int h) {
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) {
          if (live && h + u < part.y) {
            ng[u].load(dz + (h + u) * pitch, s, c);
            if (kKind < 2) nx[u].load(X + static_cast<size_t>(h0 + h + u) * a.d, s, c);
          } else {
            ng[u].zero();
            if (kKind < 2) nx[u].zero();
          }
        }
      };
      fetch(part.x);
      for (int h = part.x; h < part.y; h += kGradRows) {
        Raw<T, VEC> rx[kGradRows];
        Raw<TG, VEC> rg[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) {
          rg[u] = ng[u];
          if (kKind < 2) rx[u] = nx[u];
        }
        fetch(h + kGradRows);
        if (kKind < 2 && !turned) {
          token_turns(cs, steps, a, c, tokens, live ? token : 0, static_cast<long long>(n));
          turned = true;
        }
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) {
          float g[8];
          rg[u].get(g, s, c);
          if (kKind < 2) {
            float x[8];
            rx[u].get(x, s, c);
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
            const float r = rsqrtf(fmaf(row_sum<LPR>(sq), inv_d, a.eps));
            rotate<-1>(g, cs);
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] *= r;
              if (gain) {
                dw[kKind & 1][e] = fmaf(g[e], x[e], dw[kKind & 1][e]);
                g[e] *= w[e];
              }
              dot = fmaf(g[e], x[e], dot);
            }
            dot = row_sum<LPR>(dot) * inv_d;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * (g[e] - x[e] * dot);
          }
          if (live && h + u < part.y)
            store_row<VEC>(dX + static_cast<size_t>(h0 + h + u) * a.d, s, c, g);
        }
      }
    };
    const size_t row = (b * a.H * a.N + n) * a.d, kvrow = (b * a.Hkv * a.N + n) * a.d;
    run(std::integral_constant<int, 0>(), a.H, 0, static_cast<const TG*>(a.Q) + row, a.wq);
    run(std::integral_constant<int, 1>(), a.Hkv, a.H, static_cast<const TG*>(a.K) + kvrow, a.wk);
    run(std::integral_constant<int, 2>(), a.Hkv, a.H + a.Hkv, static_cast<const TG*>(a.V) + kvrow,
        nullptr);
  }
  if (a.dwq == nullptr) return;
  const size_t block = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part_dw[(slot * LPR + c) * 8 + e] = dw[k][e];
    __syncthreads();
    for (int x = threadIdx.x; x < LPR * 8; x += NT) {
      float sum = 0.f;
      for (int q = 0; q < kSlots; ++q) sum += part_dw[q * LPR * 8 + x];
      // Position x of the lanes' order; the sum kernel puts it in place.
      a.workspace[(block * 2 + k) * 128 + x] = sum;
    }
  }
}

// dw[k][element] = the sum of the blocks' partials in a fixed order: 8 columns
// a block, 128 runs of partials each, joined in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int blocks,
                                                       float* __restrict__ dwq,
                                                       float* __restrict__ dwk, int d, int half,
                                                       int interleaved) {
  __shared__ float s[128][9];
  const int k = blockIdx.y, run = threadIdx.x >> 3, x = blockIdx.x * 8 + (threadIdx.x & 7);
  float sum = 0.f;
  wait_ahead();
#pragma unroll 4
  for (int b = run; b < blocks; b += 128) sum += part[(static_cast<size_t>(b) * 2 + k) * 128 + x];
  s[run][threadIdx.x & 7] = sum;
  for (int n = 64; n > 0; n >>= 1) {
    __syncthreads();
    if (run < n) s[run][threadIdx.x & 7] += s[run + n][threadIdx.x & 7];
  }
  if (run) return;
  const Shape sh{d, half, interleaved != 0};
  // Element e = x % 8 of lane x / 8: pair 4 (x / 8) + e / 2.
  const int2 at = pair_at(sh, 4 * (x >> 3) + ((x & 7) >> 1));
  const int col = x & 1 ? at.y : at.x;
  if (col < d) (k ? dwk : dwq)[col] = s[0][threadIdx.x];
}

// Blocks: NT / LPR tokens each up to `most` blocks, and cut by heads (four at
// least of the larger group) up to kMostBlocks: a short call (the new tokens of
// a batch) spreads over the SMs, a long one leaves little of its last wave idle.
dim3 norm_grid(const NormArgs& a, int lpr, unsigned most) {
  constexpr unsigned kMostBlocks = 2 * kSMs;
  const size_t slots = NT / lpr, blocks = (static_cast<size_t>(a.B) * a.N + slots - 1) / slots;
  const unsigned x = static_cast<unsigned>(blocks < most ? blocks : most);
  const int heads = a.H > a.Hkv ? a.H : a.Hkv;
  unsigned y = kMostBlocks / x;
  if (y > static_cast<unsigned>((heads + 3) / 4)) y = (heads + 3) / 4;
  return dim3(x, y < 1 ? 1 : y);
}

template <typename T, int LPR, bool VEC>
cudaError_t forward(const NormArgs& a) {
  const size_t smem = static_cast<size_t>(a.R / 2) * 8 * a.axes;
  norm_kernel<T, LPR, VEC><<<norm_grid(a, LPR, kForwardBlocks), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const NormArgs& a) {
  if (a.d <= 64) return vec_ok(a) ? forward<T, 8, true>(a) : forward<T, 8, false>(a);
  return vec_ok(a) ? forward<T, 16, true>(a) : forward<T, 16, false>(a);
}

template <typename T, typename TG, int LPR, bool VEC>
cudaError_t backward(const NormArgs& a) {
  const dim3 grid = norm_grid(a, LPR, kGradBlocks);
  const size_t smem = static_cast<size_t>(a.R / 2) * 8 * a.axes;
  norm_grad_kernel<T, TG, LPR, VEC><<<grid, NT, smem, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.dwq == nullptr) return e;
  return launch_after(true, norm_dw_kernel, dim3(LPR, 2), 1024, 0, 1, a.stream, a.workspace,
                      static_cast<int>(grid.x * grid.y), a.dwq, a.dwk, a.d, a.R / 2,
                      a.interleaved ? 1 : 0);
}

template <typename T, typename TG>
cudaError_t backward(const NormArgs& a) {
  if (a.d <= 64) return vec_ok(a) ? backward<T, TG, 8, true>(a) : backward<T, TG, 8, false>(a);
  return vec_ok(a) ? backward<T, TG, 16, true>(a) : backward<T, TG, 16, false>(a);
}

}  // namespace

size_t norm_grad_workspace(const NormArgs& a) {
  if (!a.wq) return 0;
  const dim3 grid = norm_grid(a, a.d <= 64 ? 8 : 16, kGradBlocks);
  return static_cast<size_t>(grid.x) * grid.y * 2 * 128 * sizeof(float);
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
