// The paged cache's own traffic: new tokens into pages, and pages back to
// head-major tensors.
#include <math.h>

#include "norm_rope.cuh"
#include "paged.cuh"

namespace flashbob {
namespace {
using namespace rope;
using namespace paged;

// ---------------------------------------------------------------------------
// Append.  From the packed projection [B, N, H + 2 Hkv, d]: queries to head-major
// Q, keys and values into the pages; queries and keys normed (eps > 0) and turned.
// In e4m3 a page and head has one scale,
//   s = max(scale_for(largest magnitude of the new tokens), s of what it holds),
// and where that grows the codes that the page holds move to it: code' =
// nearest(code s_old / s).  A page whose first row is among the new ones starts anew.
//
// A block takes one page's tokens of one batch entry and a part of the heads (all
// H + 2 Hkv are one list of rows), so that it alone decides the page's scales: TS
// token slots of LPR lanes (8 elements each), TG tokens a slot, and where the tokens
// are few HS slots beside each other for different heads.  A lane keeps its tokens'
// angles in registers and walks the heads with TG HB = 4 rows in flight and the next
// four behind them; the page's largest magnitude meets in shuffles and, across warps,
// in shared memory.  Every element is read and written once: memory bounds it.
// ---------------------------------------------------------------------------
constexpr int kInFlight = 4;
constexpr int kMostWarps = 16;

// The lane's eight codes of a row.
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* x, const Shape& s, int c,
                                            const float (&v)[8], float inv) {
  if (VEC) {
    if (8 * c >= s.d) return;
    const bool apart = 4 * c < s.half && !s.interleaved;
    uint32_t w[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float e0 = apart ? v[u] : v[4 * u], e1 = apart ? v[2 + u] : v[4 * u + 1];
      const float e2 = apart ? v[4 + u] : v[4 * u + 2], e3 = apart ? v[6 + u] : v[4 * u + 3];
      w[u] = to_codes(e0 * inv, e1 * inv) | (to_codes(e2 * inv, e3 * inv) << 16);
    }
    *reinterpret_cast<uint32_t*>(x + (apart ? 4 * c : 8 * c)) = w[0];
    *reinterpret_cast<uint32_t*>(x + (apart ? s.half + 4 * c : 8 * c + 4)) = w[1];
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int2 at = pair_at(s, 4 * c + u);
      const uint32_t w = to_codes(v[2 * u] * inv, v[2 * u + 1] * inv);
      if (at.x < s.d) x[at.x] = static_cast<uint8_t>(w);
      if (at.y < s.d) x[at.y] = static_cast<uint8_t>(w >> 8);
    }
  }
}

// Its share of a row that the page holds already, moved to another scale.
template <bool VEC>
__device__ __forceinline__ void move_codes(uint8_t* x, int d, int c, float factor) {
  constexpr int kRun = VEC ? 4 : 1;
#pragma unroll
  for (int u = 0; u < 8 / kRun; ++u) {
    const int at = 8 * c + kRun * u;
    if (at >= d) return;
    if (VEC) {
      uint32_t* p = reinterpret_cast<uint32_t*>(x + at);
      const float2 a = from_codes(*p & 0xFFFFu), b = from_codes(*p >> 16);
      *p = to_codes(a.x * factor, a.y * factor) | (to_codes(b.x * factor, b.y * factor) << 16);
    } else {
      x[at] = static_cast<uint8_t>(to_codes(from_codes(x[at]).x * factor, 0.f));
    }
  }
}

template <typename T, bool CODES, int LPR, bool VEC, int TG>
__global__ void __launch_bounds__(32 * kMostWarps)
    append_kernel(const __grid_constant__ AppendArgs a, int TS, int pages) {
  extern __shared__ unsigned long long steps[];
  constexpr int HB = kInFlight / TG;
  __shared__ float s_most[2][kMostWarps * HB];
  const PageArgs& pg = a.page;
  const int b = blockIdx.x / pages, s = blockIdx.x % pages;
  const int heads = a.H + 2 * a.Hkv, HS = blockDim.x / LPR / TS;
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, ts = slot % TS, hs = slot / TS;
  const Shape shape{a.d, a.R / 2, a.interleaved};

  // Tokens nb .. ne - 1 lie on page `index` of the table, from row `first` on.
  const int start = a.kv_start ? a.kv_start[b] : 0;
  const int off = start & (pg.T - 1);
  const int nb = s == 0 ? 0 : s * pg.T - off;
  const int ne = static_cast<int>(min(static_cast<long long>(a.N),
                                      static_cast<long long>(s + 1) * pg.T - off));
  if (nb >= ne) return;
  const int index = (start >> pg.shift) + s, first = s == 0 ? off : 0;
  const int count = a.counts ? min(a.counts[b], a.N) : a.N;
  const int page = index >= 0 && index < pg.M ? pg.table[static_cast<size_t>(b) * pg.M + index] : -1;
  const int kept = page_ok(pg, page) ? min(ne, count) : 0;  // tokens below it enter the cache

  const int r0 = static_cast<int>(static_cast<long long>(heads) * blockIdx.y / gridDim.y);
  const int r1 = static_cast<int>(static_cast<long long>(heads) * (blockIdx.y + 1) / gridDim.y);
  const size_t tokens = static_cast<size_t>(a.B) * a.N, token0 = static_cast<size_t>(b) * a.N + nb;
  const T* X = static_cast<const T*>(a.QKV) + token0 * heads * a.d;
  auto load = [&](Raw<T, VEC> (&x)[kInFlight], int base) {
#pragma unroll
    for (int k = 0; k < HB; ++k)
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        const int row = base + hs + HS * k, n = ts + TS * g;
        if (row < r1 && nb + n < ne)
          x[k * TG + g].load(X + (static_cast<size_t>(n) * heads + row) * a.d, shape, c);
        else x[k * TG + g].zero();
      }
  };
  Raw<T, VEC> next[kInFlight];
  load(next, r0);
  fill_steps(steps, a);
  float2 cs[TG][4];
#pragma unroll
  for (int g = 0; g < TG; ++g) {
    const int n = min(nb + ts + TS * g, ne - 1);
    token_turns(cs[g], steps, a, c, tokens, static_cast<size_t>(b) * a.N + n,
                static_cast<long long>(start) + n);
  }
  const float inv_d = 1.f / a.d;
  const int span = TS * LPR, wpr = span / 32;  // lanes, and whole warps, that share a head's rows
  int parity = 0;
  for (int base = r0; base < r1; base += HS * HB, parity ^= 1) {
    float v[kInFlight][8];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) next[u].get(v[u], shape, c);
    if (base + HS * HB < r1) load(next, base + HS * HB);
    float most[HB], old[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int row = base + hs + HS * k;
      most[k] = old[k] = 0.f;
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        float(&x)[8] = v[k * TG + g];
        if (a.eps > 0.f) {  // the lanes of a warp stay together: the shuffles need them all
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
          const float r = rsqrtf(fmaf(row_sum<LPR>(sq), inv_d, a.eps));
          if (row < a.H + a.Hkv) {
            const float* gain = row < a.H ? a.wq : a.wk;
            float w[8];
            if (gain) load_row<VEC>(gain, shape, c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = gain ? x[e] * r * w[e] : x[e] * r;
          }
        }
        // Pairs that do not turn are left alone: 0 times an infinity beside it is NaN.
        if (row < a.H + a.Hkv && 4 * c < shape.half) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e];
          rotate<1>(y, cs[g]);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (4 * c + u < shape.half) x[2 * u] = y[2 * u], x[2 * u + 1] = y[2 * u + 1];
        }
        if (CODES && nb + ts + TS * g < kept) {
#pragma unroll
          for (int e = 0; e < 8; ++e) most[k] = fmaxf(most[k], finite_abs(x[e]));
        }
      }
    }
    const bool any_kv = base + HS * HB > a.H && kept > nb;
    if (CODES && any_kv) {
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        const int row = base + hs + HS * k, h = row - a.H;
        for (int o = 1; o < 32 && o < span; o <<= 1)
          most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
        if (first > 0 && h >= 0 && row < r1)
          old[k] = held_scale((h < a.Hkv ? pg.k_scale : pg.v_scale)[
              static_cast<size_t>(page) * a.Hkv + (h < a.Hkv ? h : h - a.Hkv)]);
        if (wpr > 1 && (threadIdx.x & 31) == 0)
          s_most[parity][(threadIdx.x >> 5) + kMostWarps * k] = most[k];
      }
      if (wpr > 1) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < HB; ++k)
          for (int w = 0; w < wpr; ++w)
            most[k] = fmaxf(most[k], s_most[parity][hs * wpr + w + kMostWarps * k]);
      }
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int row = base + hs + HS * k, h = row - a.H, kv = h < a.Hkv ? h : h - a.Hkv;
      if (row >= r1) continue;
      if (row < a.H) {
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int n = nb + ts + TS * g;
          if (n < ne)
            store_row<VEC>(static_cast<T*>(a.Q) +
                               ((static_cast<size_t>(b) * a.H + row) * a.N + n) * a.d,
                           shape, c, v[k * TG + g]);
        }
        continue;
      }
      if (kept <= nb) continue;
      const size_t at = page_row(pg, page, a.Hkv, kv, 0);
      if (CODES) {
        uint8_t* pool = static_cast<uint8_t*>(h < a.Hkv ? a.K : a.V) + at * a.d;
        const float scale = fmaxf(scale_for(most[k]), old[k]), inv = 1.f / scale;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int n = ts + TS * g;
          if (nb + n < kept)
            store_codes<VEC>(pool + static_cast<size_t>(first + n) * a.d, shape, c, v[k * TG + g],
                             inv);
        }
        if (first > 0 && scale != old[k])
          for (int r = ts; r < first; r += TS)
            move_codes<VEC>(pool + static_cast<size_t>(r) * a.d, a.d, c, old[k] * inv);
        if (ts == 0 && c == 0 && scale != old[k])
          (h < a.Hkv ? pg.k_scale : pg.v_scale)[static_cast<size_t>(page) * a.Hkv + kv] = scale;
      } else {
        T* pool = static_cast<T*>(h < a.Hkv ? a.K : a.V) + at * a.d;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int n = ts + TS * g;
          if (nb + n < kept)
            store_row<VEC>(pool + static_cast<size_t>(first + n) * a.d, shape, c, v[k * TG + g]);
        }
      }
    }
  }
}

template <typename T, bool CODES, int LPR, bool VEC, int TG>
cudaError_t append(const AppendArgs& a, int threads, int TS) {
  const long long pages = (static_cast<long long>(a.N) + 2LL * a.page.T - 2) >> a.page.shift;
  const long long blocks = pages * a.B;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const int heads = a.H + 2 * a.Hkv, HS = threads / LPR / TS;
  // Parts of the heads: as many as fill the GPU a few times over, each with one row
  // of a slot at least.
  long long y = (8LL * kSMs + blocks - 1) / blocks;
  const long long most = (heads + HS - 1) / HS;
  y = y > most ? most : y;
  const size_t smem = static_cast<size_t>(a.R / 2) * 8 * a.axes;
  append_kernel<T, CODES, LPR, VEC, TG>
      <<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y)), threads, smem, a.stream>>>(
          a, TS, static_cast<int>(pages));
  return cudaGetLastError();
}

template <typename T, bool CODES, int LPR>
cudaError_t append(const AppendArgs& a) {
  int window = 1;  // tokens of a page that a call can bring
  while (window < a.page.T && window < a.N) window *= 2;
  // 256 threads, or 512 where four tokens a slot would not cover the page.
  const int threads = window > 4 * (256 / LPR) ? 512 : 256, slots = threads / LPR;
  if (!vec_ok(a)) return append<T, CODES, LPR, false, 4>(a, threads, window < 4 ? 1 : window / 4);
  const int TS = window < slots ? window : slots;
  switch (window / TS) {
    case 1: return append<T, CODES, LPR, true, 1>(a, threads, TS);
    case 2: return append<T, CODES, LPR, true, 2>(a, threads, TS);
    default: return append<T, CODES, LPR, true, 4>(a, threads, TS);
  }
}

template <typename T>
cudaError_t append(const AppendArgs& a) {
  if (a.d <= 64) return a.page.e4m3 ? append<T, true, 8>(a) : append<T, false, 8>(a);
  return a.page.e4m3 ? append<T, true, 16>(a) : append<T, false, 16>(a);
}

// ---------------------------------------------------------------------------
// Read.  A thread takes runs of 16 codes, or of 16 bytes of a 16- or 32-bit cache
// (single elements where rows do not divide into them); blockIdx.y = 1 the values.
// ---------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadRuns = 4;  // in flight of each thread

template <typename T, bool CODES, bool VEC>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(const __grid_constant__ ReadArgs a, int runs, int blocks) {
  constexpr int E = !VEC ? 1 : CODES ? 16 : 16 / static_cast<int>(sizeof(T));
  const int g = blockIdx.x / blocks, b = g / a.Hkv, hkv = g % a.Hkv;
  const int per = kReadThreads / runs, r = threadIdx.x / runs, k = threadIdx.x % runs * E;
  if (r >= per) return;
  const bool values = blockIdx.y == 1;
  const void* pool = values ? a.V : a.K;
  const float* scales = values ? a.page.v_scale : a.page.k_scale;
  T* out = static_cast<T*>(values ? a.Vd : a.Kd) + static_cast<size_t>(g) * a.Nk * a.d + k;
  const int len = a.lens ? min(a.lens[b], a.Nk) : a.Nk;
  const long long row0 = static_cast<long long>(blockIdx.x % blocks) * per * kReadRuns + r;
  uint4 w[kReadRuns];
  float scale[kReadRuns];
#pragma unroll
  for (int u = 0; u < kReadRuns; ++u) {
    const long long j = row0 + u * per;
    w[u] = make_uint4(0u, 0u, 0u, 0u);
    scale[u] = 1.f;
    const int page = j < len ? page_at(a.page, b, static_cast<int>(j)) : -1;
    if (!page_ok(a.page, page)) continue;
    const size_t at = page_row(a.page, page, a.Hkv, hkv, static_cast<int>(j)) * a.d + k;
    if (CODES) scale[u] = scales[static_cast<size_t>(page) * a.Hkv + hkv];
    if (VEC) w[u] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) +
                                                    at * (CODES ? 1 : sizeof(T)));
    else if (CODES) w[u].x = static_cast<const uint8_t*>(pool)[at];
    else *reinterpret_cast<T*>(&w[u].x) = static_cast<const T*>(pool)[at];
  }
#pragma unroll
  for (int u = 0; u < kReadRuns; ++u) {
    const long long j = row0 + u * per;
    if (j >= a.Nk) return;
    T* o = out + static_cast<size_t>(j) * a.d;
    if (!CODES) {
      if (VEC) *reinterpret_cast<uint4*>(o) = w[u];
      else *o = *reinterpret_cast<const T*>(&w[u].x);
      continue;
    }
    const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    if (!VEC) {
      put(o, from_codes(x[0]).x * scale[u]);
      continue;
    }
    // 16 values: one run of 32 bytes, or of 64.
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 lo = from_codes(x[q] & 0xFFFFu), hi = from_codes(x[q] >> 16);
      st4(o + 4 * q, lo.x * scale[u], lo.y * scale[u], hi.x * scale[u], hi.y * scale[u]);
    }
  }
}

template <typename T, bool CODES, bool VEC>
cudaError_t read(const ReadArgs& a) {
  const int E = !VEC ? 1 : CODES ? 16 : 16 / static_cast<int>(sizeof(T));
  const int runs = a.d / E, rows = kReadThreads / runs * kReadRuns;
  const long long blocks = (static_cast<long long>(a.Nk) + rows - 1) / rows;
  const long long grid = blocks * a.B * a.Hkv;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  read_kernel<T, CODES, VEC><<<dim3(static_cast<unsigned>(grid), 2), kReadThreads, 0, a.stream>>>(
      a, runs, static_cast<int>(blocks));
  return cudaGetLastError();
}

template <typename T>
cudaError_t read(const ReadArgs& a) {
  if (a.page.e4m3) return a.d % 16 == 0 ? read<T, true, true>(a) : read<T, true, false>(a);
  return a.d * sizeof(T) % 16 == 0 ? read<T, false, true>(a) : read<T, false, false>(a);
}

}  // namespace

cudaError_t cache_append(const AppendArgs& a) {
  return a.bf16 ? append<__nv_bfloat16>(a) : append<float>(a);
}

cudaError_t cache_read(const ReadArgs& a) {
  return a.bf16 ? read<__nv_bfloat16>(a) : read<float>(a);
}

}  // namespace flashbob
