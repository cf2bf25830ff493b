// Shared by the kernels of attention with key ranges: what a query row sees,
// the group-row numbering and the gradient's row state in the workspace.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "internal.h"

namespace flashbob {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 152;          // grids are sized for the GB300
constexpr int kBoundRows = 64;     // group rows summarised by one bounds entry
constexpr int kRowPad = 128;       // group rows are padded to this in the workspace

// The keys lo <= j < hi that a query sees and its position; an empty range
// is lo = INT_MAX, hi = 0, so that it never widens a hull.
struct RowView {
  int lo, hi, pos;
};

__device__ __forceinline__ RowView empty_view() { return {INT_MAX, 0, 0}; }

__device__ __forceinline__ RowView row_view(const int* __restrict__ ranges,
                                            const int* __restrict__ q_pos, size_t bq, int i,
                                            int Nk, int causal) {
  RowView v{0, Nk, q_pos ? q_pos[bq + i] : i};
  if (ranges) {  // clamped: whatever the array holds, no key outside 0 .. Nk - 1 is read
    const int2 r = reinterpret_cast<const int2*>(ranges)[bq + i];
    v.lo = max(r.x, 0);
    v.hi = min(r.y, Nk);
  }
  if (causal && v.pos < v.hi) v.hi = v.pos + 1;
  if (v.lo >= v.hi) v.lo = INT_MAX, v.hi = 0;
  return v;
}

// Minimum and maximum over a warp.
__device__ __forceinline__ int warp_min(int v) { return __reduce_min_sync(0xffffffffu, v); }
__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Row state that the dK, dV kernels read, one entry for each group row,
// rows padded to a multiple of kRowPad per (batch, key/value head):
//   info  {lo, hi, pos, slope log2 e (as bits)},
//   l2, dd  L log2 e and D; +inf in place of L for rows that see nothing and
//         for the padding,
//   ex      (bf16 with d = 64 only) -L / tau and -D as sums of three bf16 parts
//         (exact to 2^-24), the B operand of one more K step of the score
//         products: columns 0 - 2 and 3 - 5 of 16, in core matrices of 8 rows
//         x 16 bytes (row r of 128: (r / 8) 256 + (r % 8) 16, columns 8 - 15
//         128 bytes further); the L columns are 0 for capped scores, and for
//         rows that see nothing and the padding (their tiles run masked),
// and for each kBoundRows rows {min lo, max hi, max lo, min hi}, the hull of
// their ranges and their intersection (the padding takes no part), and
//   lines   {kind, pos, slope log2 e (as bits), 0}: kind 1 where the positions of
//         the rows count up by one from pos and their slopes are equal, 2 where
//         there are no rows, else 0.
struct GradRows {
  int4* bounds;
  int4* lines;
  int4* info;
  float *l2, *dd;
  uint8_t* ex;  // kExRow bytes a row
  int pitch;  // padded rows per (batch, key/value head)
};

__host__ __device__ inline int padded_rows(int rows) {
  return (rows + kRowPad - 1) / kRowPad * kRowPad;
}

constexpr int kExRow = 32;

__host__ __device__ inline GradRows grad_rows(void* workspace, int groups, int rows) {
  GradRows g;
  g.pitch = padded_rows(rows);
  const size_t n = static_cast<size_t>(groups) * g.pitch;
  g.bounds = static_cast<int4*>(workspace);
  g.lines = g.bounds + n / kBoundRows;
  g.info = g.lines + n / kBoundRows;
  g.l2 = reinterpret_cast<float*>(g.info + n);
  g.dd = g.l2 + n;
  g.ex = reinterpret_cast<uint8_t*>(g.dd + n);
  return g;
}

// Partial results of a split forward: for split s and global row r (row-major
// [B, H, Nq]) the unnormalised sum over its keys [s][r][d], its maximum and
// its sum of weights (log2 units).
struct Partials {
  float* o;
  float2* ml;
};

__host__ __device__ inline Partials partials(void* workspace, size_t rows, int d, int splits) {
  Partials p;
  p.ml = static_cast<float2*>(workspace);
  p.o = reinterpret_cast<float*>(p.ml + ((rows * splits + 1) & ~static_cast<size_t>(1)));
  return p;
}

// A call's later launches may start before the launch ahead has ended
// (launch_after): wait_ahead returns when it has, with all that it wrote;
// release_next lets the next launch start once every block has come here.
// Only wait_ahead makes writes visible, and only those of the launch directly
// ahead: what an early launch reads without it, or past it, has to be complete
// before the call's first launch, which is never early.  So a gradient runs the
// row state, then dK and dV (which wait for it), then dQ, which reads the call's
// inputs alone.  Whatever follows a call on the stream waits for its last launch
// alone, so the last block of an early launch always waits for the launch ahead.
__device__ __forceinline__ void wait_ahead() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with clusters of S blocks along x.  `early`: right behind the kernel
// ahead on the stream, as soon as that releases it.
template <typename... P, typename... A>
cudaError_t launch_after(bool early, void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                         int S, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (S > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = S;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four consecutive elements, aligned to their size.
__device__ __forceinline__ float4 ld4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}

// Lane `lane8` of eight: its part of the dot product of two rows.
template <typename T, int D>
__device__ __forceinline__ float dot_part(const T* __restrict__ x, const T* __restrict__ y, int d,
                                          int lane8) {
  float s = 0.f;
  if (D > 0) {  // bf16, d = D: 16-byte loads
    uint4 a[D / 64 + 1], b[D / 64 + 1];
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      a[k] = reinterpret_cast<const uint4*>(x)[8 * k + lane8];
      b[k] = reinterpret_cast<const uint4*>(y)[8 * k + lane8];
    }
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const uint32_t u[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
      const uint32_t v[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), s);
        s = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), __uint_as_float(v[e] & 0xFFFF0000u), s);
      }
    }
  } else if ((d & 3) == 0) {
    for (int k = 4 * lane8; k < d; k += 32) {
      const float4 a = ld4(x + k), b = ld4(y + k);
      s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
    }
  } else {
    for (int k = lane8; k < d; k += 8) s = fmaf(to_f(x[k]), to_f(y[k]), s);
  }
  return s;
}

// The same sum in all eight lanes (of a whole warp).
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace attn
}  // namespace flashbob
