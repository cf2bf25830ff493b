// fp32 CUDA-core kernels of attention with capped scores, a distance bias and
// key ranges, any head dim 1 <= d <= 128, fp32 or bf16 inputs:
//   z = tau q.k,  c = cap tanh(z / cap) (cap > 0),  s = c - slope |pos - j|,
//   P = softmax of s over the visible keys,  O = P V,
//   ds = P (dO V^T - D) (1 - tanh^2),  dQ = tau ds K,  dK = tau ds^T Q,
//   dV = P^T dO.
// The tensor-core kernels take bf16 with d = 64 and d = 128; everything else
// runs here, in fp32 throughout.
//
// A block holds 64 rows and streams tiles of 64: the forward and dQ hold
// group rows (queries) and stream keys, dK and dV hold keys and stream group
// rows, so every output is written once and no sum depends on an order of
// atomics.  256 threads; thread (ty, tx) owns rows ty + 16 i and columns
// tx + 16 j of a 64 x 64 score tile (i, j < 4), so that the 16 threads of a
// row sit in half a warp and row reductions are four shuffles.  A score step
// of 4 along d costs 8 16-byte shared loads for 64 multiply-adds, rows
// padded by 4 floats against bank conflicts: the multiply-adds bound it.
// Grids that leave SMs idle are cut along the streamed side: the forward into
// runs joined by a second launch, dQ and dK, dV into clusters whose blocks sum
// their parts through distributed shared memory in the order of the ranks
// (B2 H3 N333 d80: forward 59 -> 29 us, gradient 146 -> 60 us).
#include <math.h>

#include "paged.cuh"
#include "tc_common.cuh"

namespace flashbob {
namespace {
using namespace attn;

constexpr int BT = 64;        // rows of a block, rows of a streamed tile
constexpr int NT = 256;
constexpr int LP = BT + 4;    // pitch of a 64 x 64 tile

template <int DP>
constexpr int kLd = DP + 4;   // pitch of a 64 x DP tile

// dst[r][k] <- rows row0 .. row0 + 63 of src (pitch d), zero outside
// [first, last) and beyond d.
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const T* __restrict__ src, int row0,
                                          int first, int last, int d) {
  if ((d & 3) == 0) {
    for (int x = threadIdx.x; x < BT * (DP / 4); x += NT) {
      const int r = x / (DP / 4), k = 4 * (x % (DP / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row0 + r >= first && row0 + r < last && k < d)
        v = ld4(src + static_cast<size_t>(row0 + r) * d + k);
      *reinterpret_cast<float4*>(dst + r * kLd<DP> + k) = v;
    }
  } else {
    for (int x = threadIdx.x; x < BT * DP; x += NT) {
      const int r = x / DP, k = x % DP;
      float v = 0.f;
      if (row0 + r >= first && row0 + r < last && k < d)
        v = to_f(src[static_cast<size_t>(row0 + r) * d + k]);
      dst[r * kLd<DP> + k] = v;
    }
  }
}

// The same of a group's keys or values: whole rows in memory, or pages of T or of
// e4m3 codes (scaled), whose missing pages are zero.
template <typename T>
struct DenseKeys {
  __device__ __forceinline__ explicit DenseKeys(const AttnArgs&) {}
  template <int DP>
  __device__ __forceinline__ void load(float* dst, const AttnArgs& a, bool values, int row0,
                                       int first, int last) const {
    const size_t g = static_cast<size_t>(blockIdx.z) * a.Hkv + blockIdx.y;
    load_tile<T, DP>(dst, static_cast<const T*>(values ? a.V : a.K) + g * a.Nk * a.d, row0, first,
                     last, a.d);
  }
};

template <typename T, bool CODES>
struct PagedKeys {
  const PageArgs& p;
  __device__ __forceinline__ explicit PagedKeys(const PagedAttnArgs& a) : p(a.page) {}
  template <int DP>
  __device__ __forceinline__ void load(float* dst, const AttnArgs& a, bool values, int row0,
                                       int first, int last) const {
    const void* pool = values ? a.V : a.K;
    const float* scales = values ? p.v_scale : p.k_scale;
    for (int x = threadIdx.x; x < BT * DP; x += NT) {
      const int r = x / DP, k = x % DP, j = row0 + r;
      float v = 0.f;
      if (j >= first && j < last && k < a.d) {
        const int page = paged::page_at(p, blockIdx.z, j);
        if (paged::page_ok(p, page)) {
          const size_t at = paged::page_row(p, page, a.Hkv, blockIdx.y, j) * a.d + k;
          if (CODES)
            v = paged::from_codes(static_cast<const uint8_t*>(pool)[at]).x *
                scales[static_cast<size_t>(page) * a.Hkv + blockIdx.y];
          else v = to_f(static_cast<const T*>(pool)[at]);
        }
      }
      dst[r * kLd<DP> + k] = v;
    }
  }
};

// acc[i][j] = A[ty + 16 i] . B[tx + 16 j]
template <int DP>
__device__ __forceinline__ void score_tile(const float* A, const float* Bm, int ty, int tx,
                                           float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int k = 0; k < DP; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kLd<DP> + k);
      b[i] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * i) * kLd<DP> + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(a[i].x, b[j].x,
                         fmaf(a[i].y, b[j].y,
                              fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
  }
}

// acc[i][2 c + e] += sum_k P[ty + 16 i][k] B[k][2 tx + 32 c + e]
template <int DP>
__device__ __forceinline__ void out_tile(const float* P, const float* Bm, int ty, int tx,
                                         float (&acc)[4][DP / 16]) {
#pragma unroll 2
  for (int k = 0; k < BT; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * LP + k);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        const float2 b = *reinterpret_cast<const float2*>(Bm + (k + u) * kLd<DP> + 2 * tx + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float pv = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
          acc[i][2 * c] = fmaf(pv, b.x, acc[i][2 * c]);
          acc[i][2 * c + 1] = fmaf(pv, b.y, acc[i][2 * c + 1]);
        }
      }
  }
}

__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The score in log2 units of a raw product, and tanh of it when capped.
__device__ __forceinline__ float score_log2(float raw, float tau, float cap, float inv_cap,
                                            float slope2, int pos, int j, float* th) {
  float z = raw * tau;
  if (cap > 0.f) {
    *th = tanhf(z * inv_cap);
    z = cap * *th;
  }
  z *= kLog2e;
  if (slope2 != 0.f) z = fmaf(-slope2, fabsf(static_cast<float>(pos - j)), z);
  return z;
}

// Range, position, slope of the block's 64 group rows in shared memory, and
// the hull of their ranges.
struct Rows {
  int lo[BT], hi[BT], pos[BT];
  float slope2[BT];
  int hull[2];
};

__device__ __forceinline__ void load_rows(Rows& s, const AttnArgs& a, int row0, int rows) {
  if (threadIdx.x < 32) {
    int lo = INT_MAX, hi = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = threadIdx.x + 32 * u;
      RowView v = empty_view();
      float slope = 0.f;
      if (row0 + r < rows) {
        v = row_view(a.ranges, a.q_pos, static_cast<size_t>(blockIdx.z) * a.Nq,
                     (row0 + r) % a.Nq, a.Nk, a.causal);
        if (a.slopes)
          slope = a.slopes[blockIdx.y * (a.H / a.Hkv) + (row0 + r) / a.Nq] * kLog2e;
      }
      s.lo[r] = v.lo;
      s.hi[r] = v.hi;
      s.pos[r] = v.pos;
      s.slope2[r] = slope;
      lo = min(lo, v.lo);
      hi = max(hi, v.hi);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    if (threadIdx.x == 0) {
      s.hull[0] = lo;
      s.hull[1] = hi;
    }
  }
  __syncthreads();
}

// The block's 64 x d sums (times scale) to global rows row0 .. of `rows`.  In a
// cluster of S blocks each stages its part in shared memory (pitch kLd) and
// writes the rows of its rank.
template <typename T, int DP>
__device__ __forceinline__ void stage_rows(float* stage, const float (&acc)[4][DP / 16], int ty,
                                           int tx, float scale) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 32; ++c)
      *reinterpret_cast<float2*>(stage + (ty + 16 * i) * kLd<DP> + 2 * tx + 32 * c) =
          make_float2(scale * acc[i][2 * c], scale * acc[i][2 * c + 1]);
}
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const float* stage, T* __restrict__ out, int live, int d,
                                           int rank, int S) {
  const int rb = BT * rank / S, re = min(BT * (rank + 1) / S, live);
  const uint32_t base = tc::smem_u32(stage);
  for (int x = threadIdx.x; x < (re - rb) * (DP / 4); x += NT) {
    const int r = rb + x / (DP / 4), k = 4 * (x % (DP / 4));
    if (k >= d) continue;
    float4 sum = *reinterpret_cast<const float4*>(stage + r * kLd<DP> + k);
    if (S > 1) {
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < S; ++p) {
        const float4 v = tc::ld_shared_cluster_f4(
            tc::mapa_shared(base + static_cast<uint32_t>((r * kLd<DP> + k) * 4), p));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
    }
    T* o = out + static_cast<size_t>(r) * d + k;
    put(o, sum.x);
    if (k + 1 < d) put(o + 1, sum.y);
    if (k + 2 < d) put(o + 2, sum.z);
    if (k + 3 < d) put(o + 3, sum.w);
  }
}

// ---------------------------------------------------------------------------
// Forward: one pass over the key tiles of the hull with the running maximum
// and sum; with splits > 1 the block takes one run of those tiles and leaves
// its unnormalised sums in the workspace.
// ---------------------------------------------------------------------------
template <typename T, int DP, typename KEYS, typename ARGS>
__global__ void __launch_bounds__(NT) attn_kernel(const __grid_constant__ ARGS a, int splits) {
  extern __shared__ float sm[];
  float* Qs = sm;
  float* Ks = Qs + BT * kLd<DP>;
  float* Vs = Ks + BT * kLd<DP>;
  float* Ps = Vs + BT * kLd<DP>;
  __shared__ Rows rs;
  const int rows = a.H / a.Hkv * a.Nq;
  const int split = blockIdx.x % splits, row0 = blockIdx.x / splits * BT;
  const int g = blockIdx.z * a.Hkv + blockIdx.y;
  const T* Q = static_cast<const T*>(a.Q) + static_cast<size_t>(g) * rows * a.d;
  const KEYS keys(a);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;

  if (splits > 1) release_next();
  load_rows(rs, a, row0, rows);
  const int first = rs.hull[0], last = rs.hull[1];
  const int t0 = first < last ? first / BT : 0, t1 = first < last ? (last + BT - 1) / BT : 0;
  const int tb = t0 + static_cast<int>(static_cast<long long>(t1 - t0) * split / splits);
  const int te = t0 + static_cast<int>(static_cast<long long>(t1 - t0) * (split + 1) / splits);

  load_tile<T, DP>(Qs, Q, row0, 0, rows, a.d);
  float m[4], l[4], acc[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  for (int t = tb; t < te; ++t) {
    __syncthreads();
    // Rows outside the hull are zero: what they hold must not reach O.
    keys.template load<DP>(Ks, a, false, t * BT, first, last);
    keys.template load<DP>(Vs, a, true, t * BT, first, last);
    __syncthreads();
    float s[4][4];
    score_tile<DP>(Qs, Ks, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      const int lo = rs.lo[r], hi = rs.hi[r], pos = rs.pos[r];
      const float slope2 = rs.slope2[r];
      float mx = -INFINITY;
      float th;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = t * BT + tx + 16 * j;
        s[i][j] = key >= lo && key < hi
                      ? score_log2(s[i][j], a.tau, a.cap, inv_cap, slope2, pos, key, &th)
                      : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], max16(mx));
      const float base = mn == -INFINITY ? 0.f : mn;  // nothing visible so far
      const float scale = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        Ps[r * LP + tx + 16 * j] = p;
      }
      l[i] = fmaf(l[i], scale, sum16(sum));
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) acc[i][c] *= scale;
    }
    __syncwarp();  // a row of P is written and read by the same half warp
    out_tile<DP>(Ps, Vs, ty, tx, acc);
  }

  const size_t all = static_cast<size_t>(a.B) * a.H * a.Nq;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + ty + 16 * i;
    if (r >= rows) continue;
    const size_t row = static_cast<size_t>(g) * rows + r;
    if (splits > 1) {
      const Partials p = partials(a.workspace, all, a.d, splits);
      const size_t at = split * all + row;
      if (tx == 0) p.ml[at] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < DP / 32; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = 2 * tx + 32 * c + e;
          if (k < a.d) p.o[at * a.d + k] = acc[i][2 * c + e];
        }
    } else {
      const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
      if (tx == 0) a.L[row] = (m[i] + log2f(l[i])) * kLn2;  // -inf where nothing is visible
#pragma unroll
      for (int c = 0; c < DP / 32; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = 2 * tx + 32 * c + e;
          if (k < a.d) put(static_cast<T*>(a.O) + row * a.d + k, acc[i][2 * c + e] * inv);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// dQ: 64 group rows resident, key tiles of the hull stream past.  Starts when
// every block of dK and dV runs and reads nothing that they or the row state's
// launch write (D is formed here); the last block outlasts them.
// ---------------------------------------------------------------------------
template <typename T, int DP>
__global__ void __launch_bounds__(NT)
    attn_dq_kernel(const __grid_constant__ AttnArgs a, int S) {
  extern __shared__ float sm[];
  float* Qs = sm;
  float* dOs = Qs + BT * kLd<DP>;
  float* Ks = dOs + BT * kLd<DP>;
  float* Vs = Ks + BT * kLd<DP>;
  float* Ps = Vs + BT * kLd<DP>;
  __shared__ Rows rs;
  __shared__ float2 lds[BT];
  const int rank = blockIdx.x % S;
  const int rows = a.H / a.Hkv * a.Nq, row0 = blockIdx.x / S * BT;
  const int g = blockIdx.z * a.Hkv + blockIdx.y;
  const T* Q = static_cast<const T*>(a.Q) + static_cast<size_t>(g) * rows * a.d;
  const T* dO = static_cast<const T*>(a.dO) + static_cast<size_t>(g) * rows * a.d;
  const T* K = static_cast<const T*>(a.K) + static_cast<size_t>(g) * a.Nk * a.d;
  const T* V = static_cast<const T*>(a.V) + static_cast<size_t>(g) * a.Nk * a.d;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;

  load_rows(rs, a, row0, rows);
  const int first = rs.hull[0], last = rs.hull[1];
  const int t0 = first < last ? first / BT : 0, t1 = first < last ? (last + BT - 1) / BT : 0;
  load_tile<T, DP>(Qs, Q, row0, 0, rows, a.d);
  load_tile<T, DP>(dOs, dO, row0, 0, rows, a.d);
  float2 ld[4];
  float acc[4][DP / 16];
  // L log2 e and D, eight lanes a row; a row that sees nothing may hold anything.
  const T* O = static_cast<const T*>(a.O) + static_cast<size_t>(g) * rows * a.d;
#pragma unroll
  for (int u = 0; u < BT / (NT / 8); ++u) {
    const int r = u * (NT / 8) + (threadIdx.x >> 3);
    const size_t at = static_cast<size_t>(row0 + r) * a.d;
    const float dot = sum8(row0 + r < rows ? dot_part<T, 0>(O + at, dO + at, a.d, threadIdx.x & 7)
                                           : 0.f);
    if ((threadIdx.x & 7) == 0)
      lds[r] = rs.hi[r] > 0
                   ? make_float2(a.L[static_cast<size_t>(g) * rows + row0 + r] * kLog2e, dot)
                   : make_float2(INFINITY, 0.f);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ld[i] = lds[ty + 16 * i];
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  for (int t = t0 + rank; t < t1; t += S) {
    __syncthreads();
    load_tile<T, DP>(Ks, K, t * BT, first, last, a.d);
    load_tile<T, DP>(Vs, V, t * BT, first, last, a.d);
    __syncthreads();
    float s[4][4], dp[4][4];
    score_tile<DP>(Qs, Ks, ty, tx, s);
    score_tile<DP>(dOs, Vs, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      const int lo = rs.lo[r], hi = rs.hi[r], pos = rs.pos[r];
      const float slope2 = rs.slope2[r];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = t * BT + tx + 16 * j;
        float ds = 0.f;
        if (key >= lo && key < hi) {
          float th = 0.f;
          const float z = score_log2(s[i][j], a.tau, a.cap, inv_cap, slope2, pos, key, &th);
          ds = exp2f(z - ld[i].x) * (dp[i][j] - ld[i].y) * fmaf(-th, th, 1.f);
        }
        Ps[r * LP + tx + 16 * j] = ds;
      }
    }
    __syncwarp();
    out_tile<DP>(Ps, Ks, ty, tx, acc);
  }
  __syncthreads();
  stage_rows<T, DP>(Qs, acc, ty, tx, a.tau);
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  write_rows<T, DP>(Qs, static_cast<T*>(a.dQ) + (static_cast<size_t>(g) * rows + row0) * a.d,
                    rows - row0, a.d, rank, S);
  if (S > 1) tc::cluster_sync();  // the staged rows stay until all are read
  if (blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y && blockIdx.z + 1 == gridDim.z)
    wait_ahead();
}

// ---------------------------------------------------------------------------
// dK, dV: 64 keys resident, the group rows that see any of them stream past
// in tiles of 64 (their bounds say which), so a shared head's gradient sums
// its query heads on chip.  Starts beside the row state's launch and waits for it
// before it reads any of it.
// ---------------------------------------------------------------------------
template <typename T, int DP>
__global__ void __launch_bounds__(NT)
    attn_dkv_kernel(const __grid_constant__ AttnArgs a, int S) {
  extern __shared__ float sm[];
  float* Ks = sm;
  float* Vs = Ks + BT * kLd<DP>;
  float* Qs = Vs + BT * kLd<DP>;
  float* dOs = Qs + BT * kLd<DP>;
  float* Ps = dOs + BT * kLd<DP>;
  float* Ss = Ps + BT * LP;
  __shared__ int4 info[BT];
  __shared__ float2 lds[BT];
  const int rank = blockIdx.x % S;
  const int rows = a.H / a.Hkv * a.Nq, key0 = blockIdx.x / S * BT;
  const int g = blockIdx.z * a.Hkv + blockIdx.y;
  const T* Q = static_cast<const T*>(a.Q) + static_cast<size_t>(g) * rows * a.d;
  const T* dO = static_cast<const T*>(a.dO) + static_cast<size_t>(g) * rows * a.d;
  const T* K = static_cast<const T*>(a.K) + static_cast<size_t>(g) * a.Nk * a.d;
  const T* V = static_cast<const T*>(a.V) + static_cast<size_t>(g) * a.Nk * a.d;
  const GradRows gr = grad_rows(a.workspace, a.B * a.Hkv, rows);
  const int4* bounds = gr.bounds + static_cast<size_t>(g) * (gr.pitch / kBoundRows);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;

  load_tile<T, DP>(Ks, K, key0, 0, a.Nk, a.d);
  load_tile<T, DP>(Vs, V, key0, 0, a.Nk, a.d);
  release_next();
  wait_ahead();  // the row state is written and visible
  float ak[4][DP / 16], av[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) ak[i][c] = av[i][c] = 0.f;
  int hit = 0;
  for (int t = 0; t * BT < rows; ++t) {
    const int4 b = __ldcg(bounds + t);
    if (b.x >= key0 + BT || b.y <= key0) continue;  // no row of the tile sees a key of the block
    if (hit++ % S != rank) continue;
    __syncthreads();
    if (threadIdx.x < BT) {
      const size_t at = static_cast<size_t>(g) * gr.pitch + t * BT + threadIdx.x;
      info[threadIdx.x] = __ldcg(gr.info + at);
      lds[threadIdx.x] = make_float2(__ldcg(gr.l2 + at), __ldcg(gr.dd + at));
    }
    load_tile<T, DP>(Qs, Q, t * BT, 0, rows, a.d);
    load_tile<T, DP>(dOs, dO, t * BT, 0, rows, a.d);
    __syncthreads();
    if (threadIdx.x < BT && info[threadIdx.x].y == 0) {  // sees nothing: may hold anything
      for (int k = 0; k < DP; ++k)
        Qs[threadIdx.x * kLd<DP> + k] = dOs[threadIdx.x * kLd<DP> + k] = 0.f;
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    score_tile<DP>(Ks, Qs, ty, tx, s);
    score_tile<DP>(Vs, dOs, ty, tx, dp);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int4 in = info[tx + 16 * j];
      const float2 ld = lds[tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + ty + 16 * i;
        float p = 0.f, ds = 0.f;
        if (key >= in.x && key < in.y) {
          float th = 0.f;
          const float z = score_log2(s[i][j], a.tau, a.cap, inv_cap, __int_as_float(in.w), in.z,
                                     key, &th);
          p = exp2f(z - ld.x);
          ds = p * (dp[i][j] - ld.y) * fmaf(-th, th, 1.f);
        }
        Ps[(ty + 16 * i) * LP + tx + 16 * j] = p;
        Ss[(ty + 16 * i) * LP + tx + 16 * j] = ds;
      }
    }
    __syncwarp();
    out_tile<DP>(Ps, dOs, ty, tx, av);
    out_tile<DP>(Ss, Qs, ty, tx, ak);
  }
  __syncthreads();
  stage_rows<T, DP>(Qs, ak, ty, tx, a.tau);
  stage_rows<T, DP>(dOs, av, ty, tx, 1.f);
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  const size_t at = (static_cast<size_t>(g) * a.Nk + key0) * a.d;
  write_rows<T, DP>(Qs, static_cast<T*>(a.dK) + at, a.Nk - key0, a.d, rank, S);
  write_rows<T, DP>(dOs, static_cast<T*>(a.dV) + at, a.Nk - key0, a.d, rank, S);
  if (S > 1) tc::cluster_sync();
}

// Blocks of a cluster that share one block's streamed tiles: 4 at most (the
// gradient of B1 H2 N500 d64 fp32 50 us with up to 8, 40 with 4, 62 with 2).
int cluster_size(const AttnArgs& a, long long blocks, long long tiles) {
  int S = 1;
  while (S < 4 && blocks * a.Hkv * a.B * S * 2 <= 2 * kSMs && tiles >= S * 2) S *= 2;
  return S;
}

template <typename K>
cudaError_t launch(K kernel, size_t smem, int blocks, int S, const AttnArgs& a) {
  const cudaError_t e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_after(true, kernel, dim3(blocks * S, a.Hkv, a.B), NT, smem, S, a.stream, a, S);
}

template <int DP>
constexpr size_t kTileBytes = BT * kLd<DP> * sizeof(float);
constexpr size_t kSquareBytes = BT * LP * sizeof(float);

template <typename T, int DP, typename KEYS, typename ARGS>
cudaError_t forward(const ARGS& a, int splits) {
  const int blocks = static_cast<int>((static_cast<long long>(a.H / a.Hkv) * a.Nq + BT - 1) / BT);
  const size_t smem = 3 * kTileBytes<DP> + kSquareBytes;
  const auto kernel = attn_kernel<T, DP, KEYS, ARGS>;
  cudaError_t e = tc_set_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kernel<<<dim3(blocks * splits, a.Hkv, a.B), NT, smem, a.stream>>>(a, splits);
  e = cudaGetLastError();
  return e == cudaSuccess && splits > 1 ? attn_join(a, splits) : e;
}

template <typename T, typename KEYS, typename ARGS>
cudaError_t forward(const ARGS& a, int splits) {
  return a.d <= 32   ? forward<T, 32, KEYS>(a, splits)
         : a.d <= 64 ? forward<T, 64, KEYS>(a, splits)
         : a.d <= 96 ? forward<T, 96, KEYS>(a, splits)
                     : forward<T, 128, KEYS>(a, splits);
}

template <typename T, int DP>
cudaError_t backward(const AttnArgs& a) {
  constexpr size_t tile = kTileBytes<DP>, square = kSquareBytes;
  const int blocks = static_cast<int>((static_cast<long long>(a.H / a.Hkv) * a.Nq + BT - 1) / BT);
  const int key_blocks = (a.Nk + BT - 1) / BT;
  cudaError_t e = launch(attn_dkv_kernel<T, DP>, 4 * tile + 2 * square, key_blocks,
                         cluster_size(a, key_blocks, blocks), a);
  if (e == cudaSuccess)
    e = launch(attn_dq_kernel<T, DP>, 4 * tile + square, blocks,
               cluster_size(a, blocks, key_blocks), a);
  return e;
}

template <typename T>
cudaError_t backward(const AttnArgs& a) {
  return a.d <= 32   ? backward<T, 32>(a)
         : a.d <= 64 ? backward<T, 64>(a)
         : a.d <= 96 ? backward<T, 96>(a)
                     : backward<T, 128>(a);
}

}  // namespace

cudaError_t simt_attn(const AttnArgs& a) {
  const int splits = simt_splits(a);
  return a.bf16 ? forward<__nv_bfloat16, DenseKeys<__nv_bfloat16>>(a, splits)
                : forward<float, DenseKeys<float>>(a, splits);
}

cudaError_t simt_paged(const PagedAttnArgs& a, int splits) {
  if (a.page.e4m3)
    return a.bf16 ? forward<__nv_bfloat16, PagedKeys<__nv_bfloat16, true>>(a, splits)
                  : forward<float, PagedKeys<float, true>>(a, splits);
  return a.bf16 ? forward<__nv_bfloat16, PagedKeys<__nv_bfloat16, false>>(a, splits)
                : forward<float, PagedKeys<float, false>>(a, splits);
}

cudaError_t simt_attn_grad(const AttnArgs& a) {
  return a.bf16 ? backward<__nv_bfloat16>(a) : backward<float>(a);
}

}  // namespace flashbob
