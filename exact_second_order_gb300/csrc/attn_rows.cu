// Row-wise kernels around attention with key ranges: the ranges themselves
// (from document offsets and prefixes), the row state of the gradient, and
// the join of a forward that was split over the keys.
#include <math.h>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace flashbob {
namespace {
using namespace attn;

// ---------------------------------------------------------------------------
// Key ranges.  Query i of batch entry b sits at p = q_start[b] + i; its
// document is the last one that starts at or before p (binary search over the
// M + 1 sorted offsets, in shared memory where they fit).
// ---------------------------------------------------------------------------
constexpr int kRangeThreads = 256;
constexpr int kRangeRows = 1024;       // rows per block
constexpr int kRangeOffsets = 8192;    // offsets that are kept in shared memory

__global__ void __launch_bounds__(kRangeThreads)
    ranges_kernel(const int* __restrict__ off, const int* __restrict__ prefix,
                  const int* __restrict__ q_start, int* __restrict__ ranges,
                  int* __restrict__ q_pos, int M, int Nq, int Nk, int causal) {
  __shared__ int s_off[kRangeOffsets];
  const int b = blockIdx.y;
  const int start = q_start ? q_start[b] : 0;
  const int* o = off ? off + static_cast<size_t>(b) * (M + 1) : nullptr;
  const int* pre = prefix ? prefix + static_cast<size_t>(b) * M : nullptr;
  if (o && M < kRangeOffsets) {
    for (int k = threadIdx.x; k <= M; k += kRangeThreads) s_off[k] = o[k];
    __syncthreads();
    o = s_off;
  }
  for (int u = 0; u < kRangeRows / kRangeThreads; ++u) {
    const long long i = static_cast<long long>(blockIdx.x) * kRangeRows + u * kRangeThreads +
                        threadIdx.x;
    if (i >= Nq) return;
    const int p = static_cast<int>(static_cast<unsigned>(start) + static_cast<unsigned>(i));
    int lo = 0, hi = 0;
    bool inside = p >= 0;
    if (o) {
      int a = 0, z = M + 1;  // first offset above p lies in [a, z]
      while (a < z) {
        const int mid = a + ((z - a) >> 1);
        if (o[mid] <= p) a = mid + 1;
        else z = mid;
      }
      const int m = a - 1;  // the document
      inside = inside && m >= 0 && m < M;
      if (inside) {
        lo = o[m];
        hi = o[m + 1];
        // lo <= p, so lo + prefix cannot pass p + 1 by more than the prefix:
        // compared as a difference it cannot overflow.
        if (causal) {
          const int after = pre ? max(p - lo, pre[m] - 1) : p - lo;
          hi = after < hi - lo ? lo + after + 1 : hi;
        }
      }
    } else if (inside) {
      hi = causal && p < Nk ? p + 1 : Nk;
    }
    hi = min(hi, Nk);
    const size_t at = static_cast<size_t>(b) * Nq + i;
    reinterpret_cast<int2*>(ranges)[at] = inside ? make_int2(lo, hi) : make_int2(0, 0);
    if (q_pos) q_pos[at] = p;
  }
}

// ---------------------------------------------------------------------------
// Row state that dK and dV read.  Eight lanes take a row: D = dO . O in fp32,
// the row's range, position and slope, and the bounds of 64 rows.  O is the one
// that the caller has, of the inputs' type: with bf16 its rounding leaves an error of
// up to 2^-8 |dO| |O| in D (another pass over the keys would be needed to avoid it).
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256)
    grad_rows_kernel(const T* __restrict__ O, const T* __restrict__ dO,
                     const float* __restrict__ L, const int* __restrict__ ranges,
                     const int* __restrict__ q_pos, const float* __restrict__ slopes,
                     void* workspace, int B, int H, int Hkv, int Nq, int Nk, int d, int causal,
                     float inv_tau, int ex) {
  __shared__ int s_bound[4][8];
  __shared__ int2 s_row[kBoundRows];  // position and slope
  release_next();
  const int G = H / Hkv, rows = G * Nq;
  const int g = blockIdx.z * Hkv + blockIdx.y;
  const GradRows out = grad_rows(workspace, B * Hkv, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lane8 = lane & 7;
  int b_lo = INT_MAX, b_hi = 0, i_lo = 0, i_hi = INT_MAX;
  // All loads of both rows first: none waits for another.
  float dots[2] = {0.f, 0.f}, ls[2] = {0.f, 0.f};
  RowView views[2] = {empty_view(), empty_view()};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = blockIdx.x * kBoundRows + warp * 8 + u * 4 + (lane >> 3);
    const size_t row = static_cast<size_t>(g) * rows + r;
    if (r < rows) {
      dots[u] = dot_part<T, D>(O + row * d, dO + row * d, d, lane8);
      ls[u] = L[row];
      views[u] = row_view(ranges, q_pos, static_cast<size_t>(blockIdx.z) * Nq, r % Nq, Nk, causal);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = blockIdx.x * kBoundRows + warp * 8 + u * 4 + (lane >> 3);
    const bool live = r < rows;
    const RowView v = views[u];
    const float l = ls[u];
    const float dot = sum8(dots[u]);  // used only where v.hi > 0: else the row may hold anything
    if (live) {
      b_lo = min(b_lo, v.lo);
      b_hi = max(b_hi, v.hi);
      i_lo = max(i_lo, v.lo);
      i_hi = min(i_hi, v.hi);
    }
    if (lane8 == 0) {
      const size_t at = static_cast<size_t>(g) * out.pitch + r;
      const float slope = slopes && live ? slopes[blockIdx.y * G + r / Nq] * kLog2e : 0.f;
      out.info[at] = make_int4(v.lo, v.hi, v.pos, __float_as_int(slope));
      s_row[warp * 8 + u * 4 + (lane >> 3)] = make_int2(v.pos, __float_as_int(slope));
      out.l2[at] = v.hi > 0 ? l * kLog2e : INFINITY;
      out.dd[at] = v.hi > 0 ? dot : 0.f;
      if (ex) {  // inv_tau = 0 for capped scores
        const uint2 el = tc::split3_bf16(v.hi > 0 && inv_tau != 0.f ? -l * inv_tau : 0.f);
        const uint2 ed = tc::split3_bf16(v.hi > 0 ? -dot : 0.f);
        uint8_t* row = out.ex + (at / kRowPad) * kRowPad * kExRow + (at % kRowPad / 8) * 256 +
                       (at % 8) * 16;
        *reinterpret_cast<uint4*>(row) =
            make_uint4(el.x, el.y | (ed.x << 16), (ed.x >> 16) | (ed.y << 16), 0u);
        *reinterpret_cast<uint4*>(row + 128) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  b_lo = warp_min(b_lo);
  b_hi = warp_max(b_hi);
  i_lo = warp_max(i_lo);
  i_hi = warp_min(i_hi);
  if (lane == 0) {
    s_bound[0][warp] = b_lo;
    s_bound[1][warp] = b_hi;
    s_bound[2][warp] = i_lo;
    s_bound[3][warp] = i_hi;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int4 x = make_int4(INT_MAX, 0, 0, INT_MAX);
    for (int w = 0; w < 8; ++w) {
      x.x = min(x.x, s_bound[0][w]);
      x.y = max(x.y, s_bound[1][w]);
      x.z = max(x.z, s_bound[2][w]);
      x.w = min(x.w, s_bound[3][w]);
    }
    out.bounds[static_cast<size_t>(g) * (out.pitch / kBoundRows) + blockIdx.x] = x;
  }
  if (warp == 1) {
    bool line = true;
    for (int q = lane; q < kBoundRows; q += 32)
      if (blockIdx.x * kBoundRows + q < static_cast<unsigned>(rows))
        line = line && s_row[q].y == s_row[0].y &&
               static_cast<unsigned>(s_row[q].x) == static_cast<unsigned>(s_row[0].x) + q;
    line = __all_sync(0xffffffffu, line);
    const int kind = blockIdx.x * kBoundRows >= static_cast<unsigned>(rows) ? 2 : line ? 1 : 0;
    if (lane == 0)
      out.lines[static_cast<size_t>(g) * (out.pitch / kBoundRows) + blockIdx.x] =
          make_int4(kind, s_row[0].x, s_row[0].y, 0);
  }
}

// ---------------------------------------------------------------------------
// Join of a split forward: with the splits' maxima m_s and sums l_s (log2
// units) and unnormalised O_s, m = max m_s, w_s = exp2(m_s - m),
// O = sum w_s O_s / sum w_s l_s, L = (m + log2 sum w_s l_s) ln 2.  One block a
// row; its warps take every kJoinWarps-th split and their sums meet in shared
// memory, always in the same order (one warp a row took 40 us for 128 splits,
// one after the other).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
    join_kernel(void* workspace, T* __restrict__ O, float* __restrict__ L, size_t rows, int d,
                int splits) {
  __shared__ float s_acc[kJoinWarps][128];
  __shared__ float s_l[kJoinWarps];
  const size_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const Partials p = partials(workspace, rows, d, splits);
  wait_ahead();
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, p.ml[s * rows + row].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = warp; s < splits; s += warps) {
    const float2 ml = p.ml[s * rows + row];
    // A split that saw no key has m_s = -inf and O_s = 0.
    const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
    // The reference of a cache in 8 bits holds its pages' scales, so that sums of weights
    // that count may be further apart than fp32's least 2^-126: far factors in two steps.
    // (Elsewhere such a part does not reach the sum's last bit.)
    const float far = fminf(ml.x - m + 100.f, 0.f);
    l = far < 0.f && ml.x != -INFINITY ? fmaf(0x1p-100f, ml.y * exp2f(far), l) : fmaf(w, ml.y, l);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < d) acc[c] = fmaf(w, p.o[(s * rows + row) * d + lane + 32 * c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) s_acc[warp][lane + 32 * c] = acc[c];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int k = 0; k < warps; ++k) l += s_l[k];
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float o = 0.f;
    for (int k = 0; k < warps; ++k) o += s_acc[k][c];
    put(O + row * d + c, o * inv);
  }
  if (threadIdx.x == 0) L[row] = (m + log2f(l)) * kLn2;  // -inf for a row that sees nothing
}

template <typename T, int D>
cudaError_t launch_grad_rows(const AttnArgs& a) {
  const int rows = a.H / a.Hkv * a.Nq;
  const dim3 grid(padded_rows(rows) / kBoundRows, a.Hkv, a.B);
  grad_rows_kernel<T, D><<<grid, 256, 0, a.stream>>>(
      static_cast<const T*>(a.O), static_cast<const T*>(a.dO), a.L, a.ranges, a.q_pos, a.slopes,
      a.workspace, a.B, a.H, a.Hkv, a.Nq, a.Nk, a.d, a.causal ? 1 : 0,
      a.cap > 0.f ? 0.f : 1.f / a.tau, a.bf16 && a.d == 64 ? 1 : 0);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_join(const AttnArgs& a, int splits) {
  const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq;
  const int warps = splits < kJoinWarps ? splits : kJoinWarps;
  return launch_after(true, join_kernel<T>, dim3(static_cast<unsigned>(rows)), 32 * warps, 0, 1,
                      a.stream, a.workspace, static_cast<T*>(a.O), a.L, rows, a.d, splits);
}

}  // namespace

cudaError_t attn_grad_rows(const AttnArgs& a) {
  if (!a.bf16) return launch_grad_rows<float, 0>(a);
  return a.d == 64    ? launch_grad_rows<__nv_bfloat16, 64>(a)
         : a.d == 128 ? launch_grad_rows<__nv_bfloat16, 128>(a)
                      : launch_grad_rows<__nv_bfloat16, 0>(a);
}

cudaError_t attn_join(const AttnArgs& a, int splits) {
  return a.bf16 ? launch_join<__nv_bfloat16>(a, splits) : launch_join<float>(a, splits);
}

cudaError_t attn_ranges(const int* doc_offsets, const int* prefix, const int* q_start, int* ranges,
                        int* q_pos, int B, int M, int Nq, int Nk, bool causal,
                        cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(Nq) + kRangeRows - 1) / kRangeRows),
                  B);
  ranges_kernel<<<grid, kRangeThreads, 0, stream>>>(doc_offsets, prefix, q_start, ranges, q_pos, M,
                                                    Nq, Nk, causal ? 1 : 0);
  return cudaGetLastError();
}

size_t attn_forward_workspace(const AttnArgs& a) {
  const int splits = attn_splits(a);
  return splits == 1 ? 0 : partial_bytes(static_cast<size_t>(a.B) * a.H * a.Nq, a.d, splits);
}

size_t attn_grad_workspace(const AttnArgs& a) {
  const int rows = a.H / a.Hkv * a.Nq, groups = a.B * a.Hkv;
  const GradRows g = grad_rows(nullptr, groups, rows);
  return reinterpret_cast<size_t>(g.ex) +
         (a.bf16 && a.d == 64 ? static_cast<size_t>(groups) * g.pitch * kExRow : 0);
}

// A grid that leaves SMs idle is cut along the keys, so that the tiles of one
// row block run side by side and are joined afterwards.
int attn_splits(const AttnArgs& a) {
  return tc_attn_supported(a) ? tc_attn_splits(a) : simt_splits(a);
}

int simt_splits(const AttnArgs& a) {
  const long long blocks = static_cast<long long>(a.B) * a.Hkv *
                           ((static_cast<long long>(a.H / a.Hkv) * a.Nq + 63) / 64);
  const long long tiles = (a.Nk + 63) / 64, s = kSMs / blocks;
  return s < 2 || tiles < 2 ? 1 : static_cast<int>(s < tiles ? s : tiles);
}

}  // namespace flashbob
