// The paged cache's own traffic: new tokens into pages, and pages back to
// head-major tensors.
#include <math.h>

#include "norm_rope.cuh"
#include "paged.cuh"
#include "tc_common.cuh"

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
// token slots of eight lanes (E8 times eight elements each), TG tokens a slot, and where
// the tokens are few HS slots beside each other for different heads.  A lane keeps its
// tokens' angles in shared memory and walks the heads with E8 TG HB = 4 such eights in
// flight; the page's largest magnitude meets in shuffles and, across warps, in shared
// memory, and the rows are turned again for their codes (cheaper than to keep them: 64
// registers and two blocks an SM).  Every element is read and written once.
// Measured (two prompts of 8192 tokens, H32 Hkv8 d128, e4m3): 87 to 88 us, 4.2 TB/s of the
// 369 MB, 62% of the copy rate, with neither DRAM (48% of its peak) nor issue (53% of the
// slots) full: a block asks for its next heads at the top of a round, and nothing is under
// way while its warps meet, turn the rows again and write, in 2.5 waves of blocks.  Four
// eights with the next four behind them and 119 registers took 118 us, sixteen lanes a row
// 107.  Questions asked lane by lane (KIND 1): 93 with half of each head turning, 101 with
// neighbouring pairs; normed 106; pages of 128 tokens, two tokens a slot, 105; a bf16 cache
// 75, fp32 projections 168.
// ---------------------------------------------------------------------------
constexpr int kThreads = 512;
constexpr int kInFlight = 4;
constexpr int kWarps = kThreads / 32;
constexpr int LPR = 8;  // lanes a row

// Which eight elements of a row a lane has, as two runs of four: pair k is (a[k], b[k])
// (`apart`), or two neighbours of the runs in order.  VEC: see vec_ok; otherwise element
// by element, absent ones 0.
struct Lane {
  int a, b;     // first elements of the runs (VEC)
  int p;        // first pair
  int turning;  // of its four pairs
  bool apart, live;
};

template <bool VEC>
__device__ __forceinline__ Lane lane_of(const Shape& s, int c) {
  Lane n;
  n.p = 4 * c;
  n.turning = min(4, s.half - 4 * c);
  n.apart = !VEC || (4 * c < s.half && !s.interleaved);
  n.a = n.apart ? 4 * c : 8 * c;
  n.b = n.apart ? s.half + 4 * c : 8 * c + 4;
  n.live = 8 * c < s.d;
  return n;
}

template <typename T, bool VEC>
struct Eight {
  float4 a, b;
  __device__ __forceinline__ void load(const T* x, const Shape& s, const Lane& n) {
    if (VEC) {
      a = ld4(x + n.a);
      b = ld4(x + n.b);
    } else {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int2 at = pair_at(s, n.p + k);
        v[k] = at.x < s.d ? to_f(x[at.x]) : 0.f;
        v[4 + k] = at.y < s.d ? to_f(x[at.y]) : 0.f;
      }
      a = make_float4(v[0], v[1], v[2], v[3]);
      b = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float4& x, float4& y) const { x = a, y = b; }
};
template <>
struct Eight<__nv_bfloat16, true> {  // as loaded: fewer registers for rows in flight
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* x, const Shape&, const Lane& n) {
    a = *reinterpret_cast<const uint2*>(x + n.a);
    b = *reinterpret_cast<const uint2*>(x + n.b);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(float4& x, float4& y) const {
    x = make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
                    __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u));
    y = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u),
                    __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_eight(T* x, const Shape& s, const Lane& n, const float4& a,
                                            const float4& b) {
  if (VEC) {
    st4(x + n.a, a.x, a.y, a.z, a.w);
    st4(x + n.b, b.x, b.y, b.z, b.w);
  } else {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int2 at = pair_at(s, n.p + k);
      if (at.x < s.d) put(x + at.x, v[k]);
      if (at.y < s.d) put(x + at.y, v[4 + k]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* x, const Shape& s, const Lane& n,
                                            const float4& a, const float4& b, float inv) {
  const uint32_t w[4] = {to_codes(a.x * inv, a.y * inv), to_codes(a.z * inv, a.w * inv),
                         to_codes(b.x * inv, b.y * inv), to_codes(b.z * inv, b.w * inv)};
  if (VEC) {
    *reinterpret_cast<uint32_t*>(x + n.a) = w[0] | (w[1] << 16);
    *reinterpret_cast<uint32_t*>(x + n.b) = w[2] | (w[3] << 16);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int2 at = pair_at(s, n.p + k);
      const int by = 8 * (k & 1);
      if (at.x < s.d) x[at.x] = static_cast<uint8_t>(w[k / 2] >> by);
      if (at.y < s.d) x[at.y] = static_cast<uint8_t>(w[2 + k / 2] >> by);
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

// (x, y) turned by the angle with cosine c and sine s.
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float u = x * c - y * s, v = y * c + x * s;
  x = u;
  y = v;
}

// KIND 0: any head; 1: vec_ok; 2: and every lane has whole eights of pairs apart that
// turn (halves, R = d, d = 64 or 128), so nothing is asked lane by lane.
template <typename T, bool CODES, int E8, int KIND, int TG>
__global__ void __launch_bounds__(kThreads, KIND > 0 && sizeof(T) == 2 ? 2 : 1)
    append_kernel(const __grid_constant__ AppendArgs a, int TS, int pages) {
  extern __shared__ __align__(16) unsigned long long steps[];
  constexpr int HB = kInFlight / (E8 * TG);
  constexpr bool VEC = KIND > 0, WHOLE = KIND == 2;
  __shared__ float s_most[2][kWarps * HB];
  const PageArgs& pg = a.page;
  const int b = blockIdx.x / pages, s = blockIdx.x % pages;
  const int heads = a.H + 2 * a.Hkv, HS = kThreads / LPR / TS;
  const int c = threadIdx.x % LPR, slot = threadIdx.x / LPR, ts = slot % TS, hs = slot / TS;
  const Shape shape{a.d, a.R / 2, a.interleaved};
  Lane own[E8];
#pragma unroll
  for (int e = 0; e < E8; ++e) own[e] = lane_of<VEC>(shape, c + LPR * e);

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
  const size_t slab = static_cast<size_t>(kept > nb ? page : 0) * a.Hkv;  // of the page's head 0

  const int r0 = static_cast<int>(static_cast<long long>(heads) * blockIdx.y / gridDim.y);
  const int r1 = static_cast<int>(static_cast<long long>(heads) * (blockIdx.y + 1) / gridDim.y);
  const size_t tokens = static_cast<size_t>(a.B) * a.N;
  const T* X = static_cast<const T*>(a.QKV) +
               (static_cast<size_t>(b) * a.N + nb) * heads * static_cast<size_t>(a.d);
  T* Q = static_cast<T*>(a.Q) + (static_cast<size_t>(b) * a.H * a.N + nb) * a.d;
  const size_t q_head = static_cast<size_t>(a.N) * a.d, q_token = static_cast<size_t>(heads) * a.d;
  const T* x_of[TG];
  T* q_of[TG];
#pragma unroll
  for (int g = 0; g < TG; ++g) {
    const int n = min(ts + TS * g, ne - nb - 1);
    x_of[g] = X + n * q_token;
    q_of[g] = Q + n * a.d;
  }
  Eight<T, VEC> x[HB][TG][E8];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < HB; ++k)
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        const int row = base + hs + HS * k, n = ts + TS * g;
        const bool there = row < r1 && nb + n < ne;
        const T* p = x_of[g] + (row < r1 ? row : 0) * a.d;
#pragma unroll
        for (int e = 0; e < E8; ++e) {
          if (there && (WHOLE || own[e].live)) x[k][g][e].load(p, shape, own[e]);
          else x[k][g][e].zero();
        }
      }
  };
  load(r0);
  fill_steps(steps, a);
  // The lane's angles: cosines and sines of an eight's four pairs.
  float4* turns = reinterpret_cast<float4*>(steps + ((a.R / 2 * a.axes + 1) & ~1)) + threadIdx.x;
#pragma unroll
  for (int g = 0; g < TG; ++g) {
    const int n = min(nb + ts + TS * g, ne - 1);
#pragma unroll
    for (int e = 0; e < E8; ++e) {
      float2 cs[4];
      token_turns(cs, steps, a, c + LPR * e, tokens, static_cast<size_t>(b) * a.N + n,
                  static_cast<long long>(start) + n);
      turns[2 * (g * E8 + e) * kThreads] = make_float4(cs[0].x, cs[1].x, cs[2].x, cs[3].x);
      turns[(2 * (g * E8 + e) + 1) * kThreads] = make_float4(cs[0].y, cs[1].y, cs[2].y, cs[3].y);
    }
  }
  const float inv_d = 1.f / a.d;
  // 1 / rms of a row.  All lanes of a warp come here together, for the shuffles.
  auto norm_of = [&](const Eight<T, VEC> (&raw)[E8]) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < E8; ++e) {
      float4 u, v;
      raw[e].get(u, v);
      sq = fmaf(u.x, u.x, sq), sq = fmaf(u.y, u.y, sq), sq = fmaf(u.z, u.z, sq);
      sq = fmaf(u.w, u.w, sq), sq = fmaf(v.x, v.x, sq), sq = fmaf(v.y, v.y, sq);
      sq = fmaf(v.z, v.z, sq), sq = fmaf(v.w, v.w, sq);
    }
    return rsqrtf(fmaf(row_sum<LPR>(sq), inv_d, a.eps));
  };
  // Eight values of a row as they enter Q or the cache.
  auto finish = [&](const Eight<T, VEC>& raw, const Lane& o, int row, int at, float r, float4& u,
                    float4& v) {
    raw.get(u, v);
    if (row >= a.H + a.Hkv) return;
    if (a.eps > 0.f) {
      u = make_float4(u.x * r, u.y * r, u.z * r, u.w * r);
      v = make_float4(v.x * r, v.y * r, v.z * r, v.w * r);
      const float* gain = row < a.H ? a.wq : a.wk;
      if (gain && (WHOLE || o.live)) {
        Eight<float, VEC> w;
        w.load(gain, shape, o);
        u = make_float4(u.x * w.a.x, u.y * w.a.y, u.z * w.a.z, u.w * w.a.w);
        v = make_float4(v.x * w.b.x, v.y * w.b.y, v.z * w.b.z, v.w * w.b.w);
      }
    }
    if (!WHOLE && o.turning <= 0) return;
    const float4 co = turns[2 * at * kThreads], si = turns[(2 * at + 1) * kThreads];
    if (WHOLE || (o.turning == 4 && o.apart)) {
      turn_pair(u.x, v.x, co.x, si.x), turn_pair(u.y, v.y, co.y, si.y);
      turn_pair(u.z, v.z, co.z, si.z), turn_pair(u.w, v.w, co.w, si.w);
    } else if (o.apart) {  // a pair that does not turn is left alone: 0 times an infinity
      turn_pair(u.x, v.x, co.x, si.x);  // beside it would be NaN
      if (o.turning > 1) turn_pair(u.y, v.y, co.y, si.y);
      if (o.turning > 2) turn_pair(u.z, v.z, co.z, si.z);
    } else {
      turn_pair(u.x, u.y, co.x, si.x);
      if (o.turning > 1) turn_pair(u.z, u.w, co.y, si.y);
      if (o.turning > 2) turn_pair(v.x, v.y, co.z, si.z);
      if (o.turning > 3) turn_pair(v.z, v.w, co.w, si.w);
    }
  };
  const int span = TS * LPR, wpr = span / 32;  // lanes, and whole warps, that share a head's rows
  int parity = 0;
  for (int base = r0; base < r1; base += HS * HB, parity ^= 1) {
    if (base > r0) load(base);
    float r[HB][TG];
    if (a.eps > 0.f) {
#pragma unroll
      for (int k = 0; k < HB; ++k)
#pragma unroll
        for (int g = 0; g < TG; ++g) r[k][g] = norm_of(x[k][g]);
    }
    // Queries leave, and the keys and values of a cache without scales; the others are
    // looked through for their largest magnitude.
    float most[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int row = base + hs + HS * k, h = row - a.H;
      most[k] = 0.f;
      if (row >= r1) continue;
      if (row < a.H) {
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int n = ts + TS * g;
          if (nb + n >= ne) continue;
          T* out = q_of[g] + row * q_head;
#pragma unroll
          for (int e = 0; e < E8; ++e) {
            float4 u, v;
            finish(x[k][g][e], own[e], row, g * E8 + e, r[k][g], u, v);
            if (WHOLE || own[e].live) store_eight<T, VEC>(out, shape, own[e], u, v);
          }
        }
        continue;
      }
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        const int n = ts + TS * g;
        if (nb + n >= kept) continue;
        T* out = static_cast<T*>(h < a.Hkv ? a.K : a.V) +
                 (((slab + (h < a.Hkv ? h : h - a.Hkv)) << pg.shift) + first + n) * a.d;
#pragma unroll
        for (int e = 0; e < E8; ++e) {
          float4 u, v;
          finish(x[k][g][e], own[e], row, g * E8 + e, r[k][g], u, v);
          if (!WHOLE && !own[e].live) continue;
          if (!CODES) {
            store_eight<T, VEC>(out, shape, own[e], u, v);
            continue;
          }
          float m = fmaxf(fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))),
                          fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
          if (!(m <= 3.402823466e38f))  // passes over NaN; infinities do not count either
            m = fmaxf(fmaxf(fmaxf(finite_abs(u.x), finite_abs(u.y)),
                            fmaxf(finite_abs(u.z), finite_abs(u.w))),
                      fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)),
                            fmaxf(finite_abs(v.z), finite_abs(v.w))));
          most[k] = fmaxf(most[k], m);
        }
      }
    }
    if (!CODES || base + HS * HB <= a.H || kept <= nb) continue;
    float old[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int row = base + hs + HS * k, h = row - a.H;
      for (int o = 1; o < 32 && o < span; o <<= 1)
        most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
      old[k] = 0.f;
      if (first > 0 && h >= 0 && row < r1)
        old[k] = held_scale((h < a.Hkv ? pg.k_scale : pg.v_scale)[
            slab + (h < a.Hkv ? h : h - a.Hkv)]);
      if (wpr > 1 && (threadIdx.x & 31) == 0)
        s_most[parity][(threadIdx.x >> 5) + kWarps * k] = most[k];
    }
    if (wpr > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < HB; ++k)
        for (int w = 0; w < wpr; ++w)
          most[k] = fmaxf(most[k], s_most[parity][hs * wpr + w + kWarps * k]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int row = base + hs + HS * k, h = row - a.H, kv = h < a.Hkv ? h : h - a.Hkv;
      const bool mine = row < r1 && h >= 0;
      uint8_t* pool = static_cast<uint8_t*>(h < a.Hkv ? a.K : a.V) +
                      ((slab + (mine ? kv : 0)) << pg.shift) * a.d;
      const float scale = fmaxf(scale_for(most[k]), old[k]), inv = 1.f / scale;
      if (!mine) continue;
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        const int n = ts + TS * g;
        if (nb + n >= kept) continue;
#pragma unroll
        for (int e = 0; e < E8; ++e) {
          float4 u, v;
          finish(x[k][g][e], own[e], row, g * E8 + e, r[k][g], u, v);
          if (WHOLE || own[e].live)
            store_codes<VEC>(pool + (first + n) * a.d, shape, own[e], u, v, inv);
        }
      }
      if (scale == old[k]) continue;
      for (int q = ts; q < first; q += TS)
#pragma unroll
        for (int e = 0; e < E8; ++e)
          move_codes<VEC>(pool + q * a.d, a.d, c + LPR * e, old[k] * inv);
      if (ts == 0 && c == 0) (h < a.Hkv ? pg.k_scale : pg.v_scale)[slab + kv] = scale;
    }
  }
}

template <typename T, bool CODES, int E8, int KIND, int TG>
cudaError_t append(const AppendArgs& a, int TS) {
  const long long pages = (static_cast<long long>(a.N) + 2LL * a.page.T - 2) >> a.page.shift;
  const long long blocks = pages * a.B;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const int heads = a.H + 2 * a.Hkv, HS = kThreads / LPR / TS;
  // Parts of the heads: as many as fill the GPU twice over, each with one row of a slot
  // at least.
  long long y = (4LL * kSMs + blocks - 1) / blocks;
  const long long most = (heads + HS - 1) / HS;
  y = y > most ? most : y;
  // The frequencies' steps and the lanes' angles.
  const size_t smem = static_cast<size_t>((a.R / 2 * a.axes + 1) & ~1) * 8 +
                      kThreads * TG * E8 * 32;
  const auto kernel = append_kernel<T, CODES, E8, KIND, TG>;
  if (smem > 48 * 1024) {
    const cudaError_t e = tc_set_smem(reinterpret_cast<const void*>(kernel), 80 * 1024);
    if (e != cudaSuccess) return e;
  }
  kernel<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y)), kThreads, smem,
           a.stream>>>(a, TS, static_cast<int>(pages));
  return cudaGetLastError();
}

// Eights a lane by the head, tokens a slot by how many tokens of a page a call can bring;
// fp32 and odd heads in one form.
template <bool CODES>
cudaError_t append(const AppendArgs& a) {
  int window = 1;
  while (window < a.page.T && window < a.N) window *= 2;
  const int half = window < 2 ? 1 : window / 2;
  const bool vec = vec_ok(a), whole = !a.interleaved && a.R == a.d && (a.d == 64 || a.d == 128);
  if (!a.bf16)
    return vec ? append<float, CODES, 2, 1, 2>(a, half) : append<float, CODES, 2, 0, 2>(a, half);
  using B = __nv_bfloat16;
  if (!vec) return append<B, CODES, 2, 0, 2>(a, half);
  if (a.d <= 64 && whole)
    return window <= 64 ? append<B, CODES, 1, 2, 1>(a, window) : append<B, CODES, 1, 2, 2>(a, half);
  if (whole)
    return window <= 64 ? append<B, CODES, 2, 2, 1>(a, window) : append<B, CODES, 2, 2, 2>(a, half);
  if (a.d <= 64)
    return window <= 64 ? append<B, CODES, 1, 1, 1>(a, window) : append<B, CODES, 1, 1, 2>(a, half);
  return window <= 64 ? append<B, CODES, 2, 1, 1>(a, window) : append<B, CODES, 2, 1, 2>(a, half);
}

// ---------------------------------------------------------------------------
// Read.  A thread takes runs of 16 codes, or of 16 bytes of a 16- or 32-bit cache
// (single elements where rows do not divide into them); blockIdx.y = 1 the values.
// ---------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadRuns = 4;  // in flight of each thread

// 32 bytes at p, which is 32-byte aligned (`wide`) or 16-byte aligned.
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void st16(__nv_bfloat16* p, const float (&f)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = tc::pack_bf16x2(f[2 * k], f[2 * k + 1]);
  st32(p, w, wide);
}
__device__ __forceinline__ void st16(float* p, const float (&f)[16], bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(f[8 * h + k]);
    st32(p + 8 * h, w, wide);
  }
}

template <typename T, bool CODES, bool VEC>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(const __grid_constant__ ReadArgs a, int runs, int blocks, bool wide) {
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
    // 16 values: one store of 32 bytes, or two (four of 8 bytes, a quarter of each sector
    // at a time: 221 us for four requests of 32768 tokens of 8 heads of 128, now 116, 94%
    // of the copy rate); 16 bytes a store where Kd or Vd is only that far aligned.
    float f[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 lo = from_codes(x[q] & 0xFFFFu), hi = from_codes(x[q] >> 16);
      f[4 * q] = lo.x * scale[u], f[4 * q + 1] = lo.y * scale[u];
      f[4 * q + 2] = hi.x * scale[u], f[4 * q + 3] = hi.y * scale[u];
    }
    st16(o, f, wide);
  }
}

template <typename T, bool CODES, bool VEC>
cudaError_t read(const ReadArgs& a) {
  const int E = !VEC ? 1 : CODES ? 16 : 16 / static_cast<int>(sizeof(T));
  const int runs = a.d / E, rows = kReadThreads / runs * kReadRuns;
  const long long blocks = (static_cast<long long>(a.Nk) + rows - 1) / rows;
  const long long grid = blocks * a.B * a.Hkv;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  // Rows of 16 values keep the alignment of the first one.
  const bool wide = ((reinterpret_cast<uintptr_t>(a.Kd) | reinterpret_cast<uintptr_t>(a.Vd)) & 31) == 0;
  read_kernel<T, CODES, VEC><<<dim3(static_cast<unsigned>(grid), 2), kReadThreads, 0, a.stream>>>(
      a, runs, static_cast<int>(blocks), wide);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read(const ReadArgs& a) {
  if (a.page.e4m3) return a.d % 16 == 0 ? read<T, true, true>(a) : read<T, true, false>(a);
  return a.d * sizeof(T) % 16 == 0 ? read<T, false, true>(a) : read<T, false, false>(a);
}

}  // namespace

cudaError_t cache_append(const AppendArgs& a) {
  return a.page.e4m3 ? append<true>(a) : append<false>(a);
}

cudaError_t cache_read(const ReadArgs& a) {
  return a.bf16 ? read<__nv_bfloat16>(a) : read<float>(a);
}

}  // namespace flashbob
