// C ABI of libflashbob: argument checks, dispatch and the device error word.
// The declarations and their contracts are in include/flashbob.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "../../include/flashbob.h"
#include "internal.h"

namespace flashbob {
namespace {

// One error word per device that loads the library; kernels receive its
// device address (taken with cudaGetSymbolAddress while that device is
// current) and write a nonzero code when a bounded wait gives up.
__device__ unsigned int g_error_word;

constexpr int kMaxDevices = 64;
unsigned int* g_error_ptr[kMaxDevices];
std::mutex g_error_mu;

struct Range {
  uintptr_t lo, hi;
};

bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

flashbob_status check_sizes(int B, int H, int Hkv, int Nq, int Nk, int d, float tau) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || d <= 0)
    return FLASHBOB_ERR_INVALID_ARG;
  if (H % Hkv != 0) return FLASHBOB_ERR_INVALID_ARG;
  if (!(isfinite(tau) && tau > 0.f)) return FLASHBOB_ERR_INVALID_ARG;
  if (d > 128 || B > kMaxGridY || H > kMaxGridY) return FLASHBOB_ERR_UNSUPPORTED;
  // Kernels index a (batch, head) pair with a 32-bit integer.
  if (static_cast<long long>(B) * H > INT_MAX) return FLASHBOB_ERR_UNSUPPORTED;
  return FLASHBOB_OK;
}

// One buffer of a call: `bytes` from p, read or written; p may be null where
// the call allows it.
struct Buf {
  const void* p;
  size_t bytes;
  bool out;
  bool optional = false;
};

// Null pointers, alignment, and outputs that overlap an input or another output.
flashbob_status check_buffers(const Buf* bufs, int n) {
  for (int i = 0; i < n; ++i)
    if (!bufs[i].p && !bufs[i].optional) return FLASHBOB_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!aligned16(bufs[i].p)) return FLASHBOB_ERR_MISALIGNED;
  for (int i = 0; i < n; ++i) {
    if (!bufs[i].out || !bufs[i].p) continue;
    const Range o{(uintptr_t)bufs[i].p, (uintptr_t)bufs[i].p + bufs[i].bytes};
    for (int j = 0; j < n; ++j) {
      if (j == i || !bufs[j].p) continue;
      const Range r{(uintptr_t)bufs[j].p, (uintptr_t)bufs[j].p + bufs[j].bytes};
      if (overlaps(o, r)) return FLASHBOB_ERR_INVALID_ARG;
    }
  }
  return FLASHBOB_OK;
}

flashbob_status check_dtype(flashbob_dtype t) {
  return (t == FLASHBOB_F32 || t == FLASHBOB_BF16) ? FLASHBOB_OK : FLASHBOB_ERR_INVALID_ARG;
}

}  // namespace

cudaError_t error_word_ptr(unsigned int** ptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_error_mu);
  if (g_error_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_error_word);
    if (e != cudaSuccess) return e;
    g_error_ptr[dev] = static_cast<unsigned int*>(p);
  }
  *ptr = g_error_ptr[dev];
  return cudaSuccess;
}

namespace {

// Checks shared by flashbob_bob and its two passes: which buffers a pass
// reads and writes follows from a.passes.
flashbob_status run_bob(BobArgs& a, int causal, flashbob_dtype in_dtype) {
  flashbob_status st = check_dtype(in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (causal != 0 && causal != 1) return FLASHBOB_ERR_INVALID_ARG;
  a.causal = causal == 1;
  a.bf16 = in_dtype == FLASHBOB_BF16;
  const bool p1 = a.passes & kPass1, p2 = a.passes & kPass2;
  const size_t B = a.B > 0 ? a.B : 0, dd = a.d > 0 ? a.d : 0;
  const size_t Nq = a.Nq > 0 ? a.Nq : 0, Nk = a.Nk > 0 ? a.Nk : 0;
  const size_t rows = B * (a.H > 0 ? a.H : 0) * Nq;      // query-side rows
  const size_t krows = B * (a.Hkv > 0 ? a.Hkv : 0) * Nk; // key-side rows
  const size_t esz = a.bf16 ? 2 : 4;
  const size_t inb = rows * dd * esz, mat = rows * dd * 4, vec = rows * 4;
  const size_t kinb = krows * dd * esz, kmat = krows * dd * 4;
  struct Buf {
    const void* p;
    size_t bytes;
    bool out;
  };
  Buf bufs[16];
  int n = 0;
  auto add = [&](const void* p, size_t bytes, bool out) { bufs[n++] = Buf{p, bytes, out}; };
  add(a.Q, inb, false);
  add(a.K, kinb, false);
  add(a.V, kinb, false);
  add(a.dO, inb, false);
  add(a.L, vec, false);
  add(a.D, vec, false);
  add(a.UQ, inb, false);
  add(a.UK, kinb, false);
  add(a.UV, kinb, false);
  if (p1) {
    add(a.O, mat, false);
    add(a.dQt, mat, true);
    add(a.ddOt, mat, true);
  }
  if (p2) {
    add(a.dKt, kmat, true);
    add(a.dVt, kmat, true);
  }
  add(a.alpha, vec, p1);  // written by pass 1, read by pass 2
  add(a.E, vec, p1);
  for (int i = 0; i < n; ++i)
    if (!bufs[i].p) return FLASHBOB_ERR_INVALID_ARG;
  st = check_sizes(a.B, a.H, a.Hkv, a.Nq, a.Nk, a.d, a.tau);
  if (st != FLASHBOB_OK) return st;
  for (int i = 0; i < n; ++i)
    if (!aligned16(bufs[i].p)) return FLASHBOB_ERR_MISALIGNED;
  for (int i = 0; i < n; ++i) {
    if (!bufs[i].out) continue;
    const Range o{(uintptr_t)bufs[i].p, (uintptr_t)bufs[i].p + bufs[i].bytes};
    for (int j = 0; j < n; ++j) {
      if (j == i) continue;
      const Range r{(uintptr_t)bufs[j].p, (uintptr_t)bufs[j].p + bufs[j].bytes};
      if (overlaps(o, r)) return FLASHBOB_ERR_INVALID_ARG;
    }
  }
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  const cudaError_t e = tc_supported(a) ? tc_bob(a) : simt_bob(a);
  return e == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}
}  // namespace

}  // namespace flashbob

using namespace flashbob;

extern "C" {

const char* flashbob_status_string(flashbob_status s) {
  switch (s) {
    case FLASHBOB_OK: return "FLASHBOB_OK";
    case FLASHBOB_ERR_INVALID_ARG: return "FLASHBOB_ERR_INVALID_ARG";
    case FLASHBOB_ERR_UNSUPPORTED: return "FLASHBOB_ERR_UNSUPPORTED";
    case FLASHBOB_ERR_MISALIGNED: return "FLASHBOB_ERR_MISALIGNED";
    case FLASHBOB_ERR_CUDA: return "FLASHBOB_ERR_CUDA";
    case FLASHBOB_ERR_TIMEOUT: return "FLASHBOB_ERR_TIMEOUT";
  }
  return "FLASHBOB_UNKNOWN_STATUS";
}

flashbob_status flashbob_prep(const void* Q, const void* K, const void* V, const void* dO,
                              float* O, float* L, float* D, int B, int H, int Hkv, int Nq,
                              int Nk, int d, float tau, int causal, flashbob_dtype in_dtype,
                              void* stream) {
  flashbob_status st = check_dtype(in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (causal != 0 && causal != 1) return FLASHBOB_ERR_INVALID_ARG;
  // dO and D are both given (the BoB's row state) or both null (forward only).
  if (!Q || !K || !V || !O || !L || (!dO != !D)) return FLASHBOB_ERR_INVALID_ARG;
  st = check_sizes(B, H, Hkv, Nq, Nk, d, tau);
  if (st != FLASHBOB_OK) return st;
  const void* ptrs[] = {Q, K, V, dO, O, L, D};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return FLASHBOB_ERR_MISALIGNED;
  const size_t rows = (size_t)B * H * Nq, krows = (size_t)B * Hkv * Nk;
  const size_t esz = in_dtype == FLASHBOB_BF16 ? 2 : 4;
  // A null dO / D gets an empty range.
  const size_t dob = dO ? rows * d * esz : 0, db = D ? rows * 4 : 0;
  const Range ins[] = {{(uintptr_t)Q, (uintptr_t)Q + rows * d * esz},
                       {(uintptr_t)K, (uintptr_t)K + krows * d * esz},
                       {(uintptr_t)V, (uintptr_t)V + krows * d * esz},
                       {(uintptr_t)dO, (uintptr_t)dO + dob}};
  const Range outs[] = {{(uintptr_t)O, (uintptr_t)O + rows * d * 4},
                        {(uintptr_t)L, (uintptr_t)L + rows * 4},
                        {(uintptr_t)D, (uintptr_t)D + db}};
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (overlaps(o, i)) return FLASHBOB_ERR_INVALID_ARG;
    for (const Range& o2 : outs)
      if (&o != &o2 && overlaps(o, o2)) return FLASHBOB_ERR_INVALID_ARG;
  }
  PrepArgs a{Q,  K,  V, dO,  O,  L, D, B, H, Hkv, Nq, Nk, d, tau, causal == 1,
             in_dtype == FLASHBOB_BF16, (cudaStream_t)stream, nullptr};
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  const cudaError_t e = tc_prep_supported(a) ? tc_prep(a) : simt_prep(a);
  return e == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_bob(const void* Q, const void* K, const void* V, const float* O,
                             const void* dO, const float* L, const float* D, const void* UQ,
                             const void* UK, const void* UV, float tau, float* dQt, float* dKt,
                             float* dVt, float* ddOt, float* alpha, float* E, int B, int H,
                             int Hkv, int Nq, int Nk, int d, int causal, flashbob_dtype in_dtype,
                             void* stream) {
  BobArgs a{Q,  K,  V,     O, dO, L,     D,     UQ,    UK, UV, tau, dQt, dKt, dVt,
            ddOt, alpha, E, B, H,  Hkv, Nq, Nk, d, false, false, (cudaStream_t)stream,
            nullptr, kPass1 | kPass2};
  return run_bob(a, causal, in_dtype);
}

flashbob_status flashbob_bob_pass1(const void* Q, const void* K, const void* V, const float* O,
                                   const void* dO, const float* L, const float* D,
                                   const void* UQ, const void* UK, const void* UV, float tau,
                                   float* dQt, float* ddOt, float* alpha, float* E, int B, int H,
                                   int Hkv, int Nq, int Nk, int d, int causal,
                                   flashbob_dtype in_dtype, void* stream) {
  BobArgs a{Q,    K,     V, O, dO, L,   D,  UQ, UK, UV,    tau,   dQt, nullptr, nullptr,
            ddOt, alpha, E, B, H,  Hkv, Nq, Nk, d,  false, false, (cudaStream_t)stream,
            nullptr, kPass1};
  return run_bob(a, causal, in_dtype);
}

flashbob_status flashbob_bob_pass2(const void* Q, const void* K, const void* V, const void* dO,
                                   const float* L, const float* D, const float* alpha,
                                   const float* E, const void* UQ, const void* UK,
                                   const void* UV, float tau, float* dKt, float* dVt, int B,
                                   int H, int Hkv, int Nq, int Nk, int d, int causal,
                                   flashbob_dtype in_dtype, void* stream) {
  // alpha and E are inputs of pass 2; the BobArgs fields keep their names.
  BobArgs a{Q,       K,   V,   nullptr, dO, L, D, UQ, UK, UV, tau, nullptr, dKt, dVt, nullptr,
            (float*)alpha, (float*)E, B, H, Hkv, Nq, Nk, d, false, false, (cudaStream_t)stream,
            nullptr, kPass2};
  return run_bob(a, causal, in_dtype);
}

flashbob_status flashbob_bob_launches(int B, int H, int Hkv, int Nq, int Nk, int d,
                                      flashbob_dtype in_dtype, int* launches) {
  if (check_dtype(in_dtype) != FLASHBOB_OK || launches == nullptr)
    return FLASHBOB_ERR_INVALID_ARG;
  const flashbob_status st = check_sizes(B, H, Hkv, Nq, Nk, d, 1.0f);
  if (st != FLASHBOB_OK) return st;
  BobArgs a{};
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.Nq = Nq;
  a.Nk = Nk;
  a.d = d;
  a.bf16 = in_dtype == FLASHBOB_BF16;
  a.passes = kPass1 | kPass2;
  // Per head group: pass 1 (d = 128: the JVP launch and the rows launch) and pass 2.
  *launches = tc_supported(a) ? (d == 128 ? 3 : 2) * tc_bob_streams(a) : 2;
  return FLASHBOB_OK;
}

flashbob_status flashbob_bob_tile_sizes(int d, flashbob_dtype in_dtype, int* Br1, int* Bc1,
                                        int* Br2, int* Bc2, size_t* smem_bytes_pass1,
                                        size_t* smem_bytes_pass2) {
  if (check_dtype(in_dtype) != FLASHBOB_OK) return FLASHBOB_ERR_INVALID_ARG;
  if (d <= 0 || d > 128) return FLASHBOB_ERR_UNSUPPORTED;
  BobArgs probe{};
  probe.d = d;
  probe.Nq = probe.Nk = 1;
  probe.bf16 = in_dtype == FLASHBOB_BF16;
  const bool tc = tc_supported(probe), wide = tc && d == 128;
  const int br1 = tc ? kTcRows : kSimtTile, bc1 = tc ? kTcStream : kSimtTile;
  const int bc2 = tc ? kTcRows : kSimtTile;
  const int br2 = wide ? kTcStream : tc ? kTcStream2 : kSimtTile;
  if (Br1) *Br1 = br1;
  if (Bc1) *Bc1 = bc1;
  if (Br2) *Br2 = br2;
  if (Bc2) *Bc2 = bc2;
  if (smem_bytes_pass1)
    *smem_bytes_pass1 = wide ? tc_pass1_d128_smem() : tc ? tc_pass1_smem() : simt_pass1_smem(d);
  if (smem_bytes_pass2)
    *smem_bytes_pass2 = wide ? tc_pass2_d128_smem() : tc ? tc_pass2_smem() : simt_pass2_smem(d);
  return FLASHBOB_OK;
}

flashbob_status flashbob_attention_jvp(const void* Q, const void* K, const void* V,
                                       const float* O, const float* L, const void* UQ,
                                       const void* UK, const void* UV, float tau, float* Od,
                                       float* Ld, int B, int H, int Hkv, int Nq, int Nk, int d,
                                       int causal, flashbob_dtype in_dtype, void* stream) {
  flashbob_status st = check_dtype(in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (causal != 0 && causal != 1) return FLASHBOB_ERR_INVALID_ARG;
  const void* ptrs[] = {Q, K, V, O, L, UQ, UK, UV, Od, Ld};
  for (const void* p : ptrs)
    if (!p) return FLASHBOB_ERR_INVALID_ARG;
  st = check_sizes(B, H, Hkv, Nq, Nk, d, tau);
  if (st != FLASHBOB_OK) return st;
  for (const void* p : ptrs)
    if (!aligned16(p)) return FLASHBOB_ERR_MISALIGNED;
  const size_t rows = (size_t)B * H * Nq, krows = (size_t)B * Hkv * Nk;
  const size_t esz = in_dtype == FLASHBOB_BF16 ? 2 : 4;
  const Range ins[] = {{(uintptr_t)Q, (uintptr_t)Q + rows * d * esz},
                       {(uintptr_t)K, (uintptr_t)K + krows * d * esz},
                       {(uintptr_t)V, (uintptr_t)V + krows * d * esz},
                       {(uintptr_t)O, (uintptr_t)O + rows * d * 4},
                       {(uintptr_t)L, (uintptr_t)L + rows * 4},
                       {(uintptr_t)UQ, (uintptr_t)UQ + rows * d * esz},
                       {(uintptr_t)UK, (uintptr_t)UK + krows * d * esz},
                       {(uintptr_t)UV, (uintptr_t)UV + krows * d * esz}};
  const Range outs[] = {{(uintptr_t)Od, (uintptr_t)Od + rows * d * 4},
                        {(uintptr_t)Ld, (uintptr_t)Ld + rows * 4}};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlaps(o, i)) return FLASHBOB_ERR_INVALID_ARG;
  if (overlaps(outs[0], outs[1])) return FLASHBOB_ERR_INVALID_ARG;
  JvpArgs a{Q,  K,  V,  O,  L,   UQ,  UK, UV, tau, Od, Ld, B, H, Hkv, Nq, Nk, d, causal == 1,
            in_dtype == FLASHBOB_BF16, (cudaStream_t)stream, nullptr};
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  const cudaError_t e = tc_jvp_supported(a) ? tc_jvp(a) : simt_jvp(a);
  return e == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

}  // extern "C"

namespace flashbob {
namespace {

// Sizes and scalars of the attention calls with key ranges.
flashbob_status check_attention(const AttnArgs& a, int causal, flashbob_dtype in_dtype) {
  flashbob_status st = check_dtype(in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (causal != 0 && causal != 1) return FLASHBOB_ERR_INVALID_ARG;
  if (!(isfinite(a.cap) && a.cap >= 0.f)) return FLASHBOB_ERR_INVALID_ARG;
  st = check_sizes(a.B, a.H, a.Hkv, a.Nq, a.Nk, a.d, a.tau);
  if (st != FLASHBOB_OK) return st;
  // The kernels work with L / tau, 1 / cap, tau / cap and multiples of cap:
  // none of them may overflow or lose bits to underflow.
  auto in_reach = [](float x) { return x >= 0x1p-120f && x <= 0x1p120f; };
  if (!in_reach(a.tau) || (a.cap > 0.f && !(in_reach(a.cap) && in_reach(a.tau / a.cap))))
    return FLASHBOB_ERR_INVALID_ARG;
  // The rows of a group of query heads are counted in 32 bits, padding
  // included, and so are the keys with the tile beyond the last.
  if (static_cast<long long>(a.H / a.Hkv) * a.Nq > INT_MAX - 1024 || a.Nk > INT_MAX - 1024)
    return FLASHBOB_ERR_UNSUPPORTED;
  return FLASHBOB_OK;
}

// Sizes of the norm-and-rotation calls.  R may be 0 (no rotation); B * N
// counts grid blocks.  eps = 0, no norm, where `bare` allows it.
flashbob_status check_norm(const NormArgs& a, flashbob_dtype in_dtype, int interleaved,
                           bool bare = false) {
  flashbob_status st = check_dtype(in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (interleaved != 0 && interleaved != 1) return FLASHBOB_ERR_INVALID_ARG;
  if (a.B <= 0 || a.N <= 0 || a.H <= 0 || a.Hkv <= 0 || a.Nk <= 0 || a.d <= 0 || a.R < 0 ||
      a.R > a.d || a.R % 2 != 0 || a.axes < 1)
    return FLASHBOB_ERR_INVALID_ARG;
  if (!(isfinite(a.eps) && (a.eps > 0.f || (bare && a.eps == 0.f && !a.wq && !a.wk))))
    return FLASHBOB_ERR_INVALID_ARG;
  if (!a.wq != !a.wk) return FLASHBOB_ERR_INVALID_ARG;
  if (a.R > 0 && !a.freqs) return FLASHBOB_ERR_INVALID_ARG;
  if (!a.positions && a.axes != 1) return FLASHBOB_ERR_INVALID_ARG;
  if (a.d > 128 || a.axes > 4 || a.H > kMaxGridY || a.Hkv > kMaxGridY ||
      static_cast<long long>(a.B) * a.N > INT_MAX)
    return FLASHBOB_ERR_UNSUPPORTED;
  return FLASHBOB_OK;
}

// A paged cache beside tensors of `dtype`; fills the sizes in.
flashbob_status check_pages(PageArgs& p, int P, int T, int M, flashbob_dtype dtype,
                            flashbob_dtype cache_dtype) {
  const flashbob_status st = check_dtype(dtype);
  if (st != FLASHBOB_OK) return st;
  if (cache_dtype != dtype && cache_dtype != FLASHBOB_E4M3) return FLASHBOB_ERR_INVALID_ARG;
  if (P <= 0 || T <= 0 || M <= 0) return FLASHBOB_ERR_INVALID_ARG;
  p.P = P, p.T = T, p.M = M, p.e4m3 = cache_dtype == FLASHBOB_E4M3;
  p.shift = T == 16 ? 4 : T == 32 ? 5 : T == 64 ? 6 : T == 128 ? 7 : 0;
  if (p.shift == 0 || static_cast<long long>(M) * T > INT_MAX - 1024)
    return FLASHBOB_ERR_UNSUPPORTED;
  return FLASHBOB_OK;
}

// Scales come with an 8-bit cache and with no other; a page and head is counted in 32
// bits, one beyond the last included.
flashbob_status check_pools(const PageArgs& p, int Hkv) {
  if (!p.k_scale == p.e4m3 || !p.v_scale == p.e4m3) return FLASHBOB_ERR_INVALID_ARG;
  return static_cast<long long>(p.P) * Hkv >= INT_MAX ? FLASHBOB_ERR_UNSUPPORTED : FLASHBOB_OK;
}

size_t pool_bytes(const PageArgs& p, int Hkv, int d, int element) {
  return static_cast<size_t>(p.P) * Hkv * p.T * d * (p.e4m3 ? 1 : element);
}

}  // namespace
}  // namespace flashbob

extern "C" {

flashbob_status flashbob_attention_workspace(int B, int H, int Hkv, int Nq, int Nk, int d,
                                             flashbob_dtype in_dtype, size_t* forward,
                                             size_t* gradient) {
  AttnArgs a{};
  a.B = B, a.H = H, a.Hkv = Hkv, a.Nq = Nq, a.Nk = Nk, a.d = d, a.tau = 1.f;
  a.bf16 = in_dtype == FLASHBOB_BF16;
  const flashbob_status st = check_attention(a, 0, in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (forward) *forward = attn_forward_workspace(a);
  if (gradient) *gradient = attn_grad_workspace(a);
  return FLASHBOB_OK;
}

flashbob_status flashbob_attention(const void* Q, const void* K, const void* V, const int* ranges,
                                   const int* q_pos, const float* slopes, float tau, float cap,
                                   void* O, float* L, void* workspace, size_t workspace_bytes,
                                   int B, int H, int Hkv, int Nq, int Nk, int d, int causal,
                                   flashbob_dtype in_dtype, void* stream) {
  AttnArgs a{};
  a.Q = Q, a.K = K, a.V = V, a.ranges = ranges, a.q_pos = q_pos, a.slopes = slopes;
  a.tau = tau, a.cap = cap, a.O = O, a.L = L, a.workspace = workspace;
  a.B = B, a.H = H, a.Hkv = Hkv, a.Nq = Nq, a.Nk = Nk, a.d = d;
  a.causal = causal == 1, a.bf16 = in_dtype == FLASHBOB_BF16, a.stream = (cudaStream_t)stream;
  flashbob_status st = check_attention(a, causal, in_dtype);
  if (st != FLASHBOB_OK) return st;
  const size_t rows = (size_t)B * H * Nq, krows = (size_t)B * Hkv * Nk, e = a.bf16 ? 2 : 4;
  const size_t need = attn_forward_workspace(a);
  const Buf bufs[] = {{Q, rows * d * e, false},
                      {K, krows * d * e, false},
                      {V, krows * d * e, false},
                      {ranges, (size_t)B * Nq * 8, false, true},
                      {q_pos, (size_t)B * Nq * 4, false, true},
                      {slopes, (size_t)H * 4, false, true},
                      {O, rows * d * e, true},
                      {L, rows * 4, true},
                      {workspace, need, true, need == 0}};
  st = check_buffers(bufs, 9);
  if (st != FLASHBOB_OK) return st;
  if (workspace_bytes < need) return FLASHBOB_ERR_INVALID_ARG;
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  const cudaError_t ce = tc_attn_supported(a) ? tc_attn(a) : simt_attn(a);
  return ce == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_attention_grad(const void* Q, const void* K, const void* V, const void* O,
                                        const float* L, const void* dO, const int* ranges,
                                        const int* q_pos, const float* slopes, float tau,
                                        float cap, void* dQ, void* dK, void* dV, void* workspace,
                                        size_t workspace_bytes, int B, int H, int Hkv, int Nq,
                                        int Nk, int d, int causal, flashbob_dtype in_dtype,
                                        void* stream) {
  AttnArgs a{};
  a.Q = Q, a.K = K, a.V = V, a.ranges = ranges, a.q_pos = q_pos, a.slopes = slopes;
  a.tau = tau, a.cap = cap, a.O = const_cast<void*>(O), a.L = const_cast<float*>(L), a.dO = dO;
  a.dQ = dQ, a.dK = dK, a.dV = dV, a.workspace = workspace;
  a.B = B, a.H = H, a.Hkv = Hkv, a.Nq = Nq, a.Nk = Nk, a.d = d;
  a.causal = causal == 1, a.bf16 = in_dtype == FLASHBOB_BF16, a.stream = (cudaStream_t)stream;
  flashbob_status st = check_attention(a, causal, in_dtype);
  if (st != FLASHBOB_OK) return st;
  const size_t rows = (size_t)B * H * Nq, krows = (size_t)B * Hkv * Nk, e = a.bf16 ? 2 : 4;
  const size_t need = attn_grad_workspace(a);
  const Buf bufs[] = {{Q, rows * d * e, false},
                      {K, krows * d * e, false},
                      {V, krows * d * e, false},
                      {O, rows * d * e, false},
                      {L, rows * 4, false},
                      {dO, rows * d * e, false},
                      {ranges, (size_t)B * Nq * 8, false, true},
                      {q_pos, (size_t)B * Nq * 4, false, true},
                      {slopes, (size_t)H * 4, false, true},
                      {dQ, rows * d * e, true},
                      {dK, krows * d * e, true},
                      {dV, krows * d * e, true},
                      {workspace, need, true}};
  st = check_buffers(bufs, 13);
  if (st != FLASHBOB_OK) return st;
  if (workspace_bytes < need) return FLASHBOB_ERR_INVALID_ARG;
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  cudaError_t ce = attn_grad_rows(a);
  if (ce == cudaSuccess) {
    if (!tc_attn_grad_supported(a)) ce = simt_attn_grad(a);
    else if ((ce = tc_attn_dkv(a)) == cudaSuccess) ce = tc_attn_dq(a);
  }
  return ce == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_attention_ranges(const int* doc_offsets, const int* prefix,
                                          const int* q_start, int* ranges, int* q_pos, int B,
                                          int M, int Nq, int Nk, int causal, void* stream) {
  if (causal != 0 && causal != 1) return FLASHBOB_ERR_INVALID_ARG;
  if (B <= 0 || Nq <= 0 || Nk <= 0 || M < 0) return FLASHBOB_ERR_INVALID_ARG;
  if (doc_offsets ? M < 1 : M != 0 || prefix) return FLASHBOB_ERR_INVALID_ARG;
  if (B > kMaxGridY || M > INT_MAX - 1) return FLASHBOB_ERR_UNSUPPORTED;
  const Buf bufs[] = {{doc_offsets, (size_t)B * (M + 1) * 4, false, true},
                      {prefix, (size_t)B * M * 4, false, true},
                      {q_start, (size_t)B * 4, false, true},
                      {ranges, (size_t)B * Nq * 8, true},
                      {q_pos, (size_t)B * Nq * 4, true, true}};
  const flashbob_status st = check_buffers(bufs, 5);
  if (st != FLASHBOB_OK) return st;
  return attn_ranges(doc_offsets, prefix, q_start, ranges, q_pos, B, M, Nq, Nk, causal == 1,
                     (cudaStream_t)stream) == cudaSuccess
             ? FLASHBOB_OK
             : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_qk_norm_rope(const void* QKV, const float* wq, const float* wk,
                                      const float* freqs, const int* positions,
                                      const int* kv_start, float eps, void* Q, void* K, void* V,
                                      int B, int N, int H, int Hkv, int Nk, int d, int R, int axes,
                                      int interleaved, flashbob_dtype in_dtype, void* stream) {
  NormArgs a{};
  a.QKV = QKV, a.wq = wq, a.wk = wk, a.freqs = freqs, a.positions = positions, a.eps = eps;
  a.Q = Q, a.K = K, a.V = V, a.kv_start = kv_start;
  a.B = B, a.N = N, a.H = H, a.Hkv = Hkv, a.Nk = Nk, a.d = d, a.R = R, a.axes = axes;
  a.interleaved = interleaved == 1, a.bf16 = in_dtype == FLASHBOB_BF16;
  a.stream = (cudaStream_t)stream;
  flashbob_status st = check_norm(a, in_dtype, interleaved);
  if (st != FLASHBOB_OK) return st;
  // Without kv_start every token needs its row of K and V.
  if (!kv_start && Nk < N) return FLASHBOB_ERR_INVALID_ARG;
  const size_t e = a.bf16 ? 2 : 4, tokens = (size_t)B * N, cache = (size_t)B * Hkv * Nk * d * e;
  const Buf bufs[] = {{QKV, tokens * (H + 2 * (size_t)Hkv) * d * e, false},
                      {wq, (size_t)d * 4, false, true},
                      {wk, (size_t)d * 4, false, true},
                      {freqs, (size_t)axes * (R / 2) * 4, false, true},
                      {positions, axes * tokens * 4, false, true},
                      {kv_start, (size_t)B * 4, false, true},
                      {Q, tokens * H * d * e, true},
                      {K, cache, true},
                      {V, cache, true}};
  st = check_buffers(bufs, 9);
  if (st != FLASHBOB_OK) return st;
  return qk_norm(a) == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_qk_norm_rope_workspace(int B, int N, int H, int Hkv, int d,
                                                flashbob_dtype in_dtype, size_t* gradient) {
  NormArgs a{};
  const float one = 1.f;
  a.wq = a.wk = &one;
  a.B = B, a.N = N, a.H = H, a.Hkv = Hkv, a.Nk = 1, a.d = d, a.axes = 1, a.eps = 1.f;
  const flashbob_status st = check_norm(a, in_dtype, 0);
  if (st != FLASHBOB_OK) return st;
  if (gradient) *gradient = norm_grad_workspace(a);
  return FLASHBOB_OK;
}

flashbob_status flashbob_qk_norm_rope_grad(const void* QKV, const float* wq, const float* wk,
                                           const float* freqs, const int* positions, float eps,
                                           const void* dQ, const void* dK, const void* dV,
                                           void* dQKV, float* dwq, float* dwk, void* workspace,
                                           size_t workspace_bytes, int B, int N, int H, int Hkv,
                                           int d, int R, int axes, int interleaved,
                                           flashbob_dtype in_dtype, flashbob_dtype grad_dtype,
                                           void* stream) {
  NormArgs a{};
  a.QKV = QKV, a.wq = wq, a.wk = wk, a.freqs = freqs, a.positions = positions, a.eps = eps;
  a.Q = const_cast<void*>(dQ), a.K = const_cast<void*>(dK), a.V = const_cast<void*>(dV);
  a.dQKV = dQKV, a.dwq = dwq, a.dwk = dwk, a.workspace = static_cast<float*>(workspace);
  a.B = B, a.N = N, a.H = H, a.Hkv = Hkv, a.Nk = N, a.d = d, a.R = R, a.axes = axes;
  a.interleaved = interleaved == 1, a.bf16 = in_dtype == FLASHBOB_BF16;
  a.grad_bf16 = grad_dtype == FLASHBOB_BF16, a.stream = (cudaStream_t)stream;
  flashbob_status st = check_dtype(grad_dtype);
  if (st == FLASHBOB_OK) st = check_norm(a, in_dtype, interleaved);
  if (st != FLASHBOB_OK) return st;
  // The gains' gradients exist exactly where the gains do.
  if (!dwq != !wq || !dwk != !wk) return FLASHBOB_ERR_INVALID_ARG;
  const size_t e = a.bf16 ? 2 : 4, ge = a.grad_bf16 ? 2 : 4, tokens = (size_t)B * N;
  const size_t all = tokens * (H + 2 * (size_t)Hkv) * d * e, need = norm_grad_workspace(a);
  const Buf bufs[] = {{QKV, all, false},
                      {wq, (size_t)d * 4, false, true},
                      {wk, (size_t)d * 4, false, true},
                      {freqs, (size_t)axes * (R / 2) * 4, false, true},
                      {positions, axes * tokens * 4, false, true},
                      {dQ, tokens * H * d * ge, false},
                      {dK, tokens * Hkv * d * ge, false},
                      {dV, tokens * Hkv * d * ge, false},
                      {dQKV, all, true},
                      {dwq, (size_t)d * 4, true, true},
                      {dwk, (size_t)d * 4, true, true},
                      {workspace, need, true, need == 0}};
  st = check_buffers(bufs, 12);
  if (st != FLASHBOB_OK) return st;
  if (workspace_bytes < need) return FLASHBOB_ERR_INVALID_ARG;
  return qk_norm_grad(a) == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_cache_append(const void* QKV, const float* wq, const float* wk,
                                      const float* freqs, const int* positions,
                                      const int* kv_start, const int* counts, const int* table,
                                      float eps, void* Q, void* K, void* V, float* k_scale,
                                      float* v_scale, int B, int N, int H, int Hkv, int P, int T,
                                      int M, int d, int R, int axes, int interleaved,
                                      flashbob_dtype in_dtype, flashbob_dtype cache_dtype,
                                      void* stream) {
  AppendArgs a{};
  a.QKV = QKV, a.wq = wq, a.wk = wk, a.freqs = freqs, a.positions = positions, a.eps = eps;
  a.Q = Q, a.K = K, a.V = V, a.kv_start = kv_start, a.counts = counts;
  a.page.table = table, a.page.k_scale = k_scale, a.page.v_scale = v_scale;
  flashbob_status st = check_pages(a.page, P, T, M, in_dtype, cache_dtype);
  if (st != FLASHBOB_OK) return st;
  a.B = B, a.N = N, a.H = H, a.Hkv = Hkv, a.Nk = M * T, a.d = d, a.R = R, a.axes = axes;
  a.interleaved = interleaved == 1, a.bf16 = in_dtype == FLASHBOB_BF16;
  a.stream = (cudaStream_t)stream;
  st = check_norm(a, in_dtype, interleaved, true);
  if (st == FLASHBOB_OK) st = check_pools(a.page, Hkv);
  if (st != FLASHBOB_OK) return st;
  // Tokens and their pages are counted in 32 bits, a page beyond the last included.
  if (N > INT_MAX - 1024) return FLASHBOB_ERR_UNSUPPORTED;
  const size_t e = a.bf16 ? 2 : 4, tokens = (size_t)B * N, pool = pool_bytes(a.page, Hkv, d, (int)e);
  const size_t scales = (size_t)P * Hkv * 4;
  const Buf bufs[] = {{QKV, tokens * (H + 2 * (size_t)Hkv) * d * e, false},
                      {wq, (size_t)d * 4, false, true},
                      {wk, (size_t)d * 4, false, true},
                      {freqs, (size_t)axes * (R / 2) * 4, false, true},
                      {positions, axes * tokens * 4, false, true},
                      {kv_start, (size_t)B * 4, false, true},
                      {counts, (size_t)B * 4, false, true},
                      {table, (size_t)B * M * 4, false},
                      {Q, tokens * H * d * e, true},
                      {K, pool, true},
                      {V, pool, true},
                      {k_scale, scales, true, true},
                      {v_scale, scales, true, true}};
  st = check_buffers(bufs, 13);
  if (st != FLASHBOB_OK) return st;
  return cache_append(a) == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_cache_read(const void* K, const void* V, const float* k_scale,
                                    const float* v_scale, const int* table, const int* lens,
                                    void* Kd, void* Vd, int B, int Hkv, int P, int T, int M,
                                    int Nk, int d, flashbob_dtype cache_dtype,
                                    flashbob_dtype out_dtype, void* stream) {
  ReadArgs a{};
  a.K = K, a.V = V, a.lens = lens, a.Kd = Kd, a.Vd = Vd;
  a.page.table = table;
  a.page.k_scale = const_cast<float*>(k_scale), a.page.v_scale = const_cast<float*>(v_scale);
  flashbob_status st = check_pages(a.page, P, T, M, out_dtype, cache_dtype);
  if (st != FLASHBOB_OK) return st;
  a.B = B, a.Hkv = Hkv, a.Nk = Nk, a.d = d, a.bf16 = out_dtype == FLASHBOB_BF16;
  a.stream = (cudaStream_t)stream;
  if (B <= 0 || Hkv <= 0 || Nk <= 0 || d <= 0 || Nk > M * T) return FLASHBOB_ERR_INVALID_ARG;
  if (d > 128 || B > kMaxGridY || Hkv > kMaxGridY) return FLASHBOB_ERR_UNSUPPORTED;
  st = check_pools(a.page, Hkv);
  if (st != FLASHBOB_OK) return st;
  const size_t e = a.bf16 ? 2 : 4, pool = pool_bytes(a.page, Hkv, d, (int)e);
  const size_t scales = (size_t)P * Hkv * 4, out = (size_t)B * Hkv * Nk * d * e;
  const Buf bufs[] = {{K, pool, false},
                      {V, pool, false},
                      {k_scale, scales, false, true},
                      {v_scale, scales, false, true},
                      {table, (size_t)B * M * 4, false},
                      {lens, (size_t)B * 4, false, true},
                      {Kd, out, true},
                      {Vd, out, true}};
  st = check_buffers(bufs, 8);
  if (st != FLASHBOB_OK) return st;
  return cache_read(a) == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_attention_paged_workspace(int B, int H, int Hkv, int Nq, int T, int M,
                                                   int d, flashbob_dtype in_dtype,
                                                   flashbob_dtype cache_dtype, size_t* forward) {
  PagedAttnArgs a{};
  flashbob_status st = check_pages(a.page, 1, T, M, in_dtype, cache_dtype);
  if (st != FLASHBOB_OK) return st;
  a.B = B, a.H = H, a.Hkv = Hkv, a.Nq = Nq, a.Nk = M * T, a.d = d, a.tau = 1.f;
  a.bf16 = in_dtype == FLASHBOB_BF16;
  st = check_attention(a, 0, in_dtype);
  if (st != FLASHBOB_OK) return st;
  if (forward) *forward = paged_workspace(a);
  return FLASHBOB_OK;
}

flashbob_status flashbob_attention_paged(const void* Q, const void* K, const void* V,
                                         const float* k_scale, const float* v_scale,
                                         const int* table, const int* ranges, const int* q_pos,
                                         const float* slopes, float tau, float cap, void* O,
                                         float* L, void* workspace, size_t workspace_bytes, int B,
                                         int H, int Hkv, int Nq, int P, int T, int M, int d,
                                         int causal, flashbob_dtype in_dtype,
                                         flashbob_dtype cache_dtype, void* stream) {
  PagedAttnArgs a{};
  a.page.table = table;
  a.page.k_scale = const_cast<float*>(k_scale), a.page.v_scale = const_cast<float*>(v_scale);
  flashbob_status st = check_pages(a.page, P, T, M, in_dtype, cache_dtype);
  if (st != FLASHBOB_OK) return st;
  a.Q = Q, a.K = K, a.V = V, a.ranges = ranges, a.q_pos = q_pos, a.slopes = slopes;
  a.tau = tau, a.cap = cap, a.O = O, a.L = L, a.workspace = workspace;
  a.B = B, a.H = H, a.Hkv = Hkv, a.Nq = Nq, a.Nk = M * T, a.d = d;
  a.causal = causal == 1, a.bf16 = in_dtype == FLASHBOB_BF16, a.stream = (cudaStream_t)stream;
  st = check_attention(a, causal, in_dtype);
  if (st == FLASHBOB_OK) st = check_pools(a.page, Hkv);
  if (st != FLASHBOB_OK) return st;
  const size_t rows = (size_t)B * H * Nq, e = a.bf16 ? 2 : 4, need = paged_workspace(a);
  const size_t pool = pool_bytes(a.page, Hkv, d, (int)e), scales = (size_t)P * Hkv * 4;
  const Buf bufs[] = {{Q, rows * d * e, false},
                      {K, pool, false},
                      {V, pool, false},
                      {k_scale, scales, false, true},
                      {v_scale, scales, false, true},
                      {table, (size_t)B * M * 4, false},
                      {ranges, (size_t)B * Nq * 8, false, true},
                      {q_pos, (size_t)B * Nq * 4, false, true},
                      {slopes, (size_t)H * 4, false, true},
                      {O, rows * d * e, true},
                      {L, rows * 4, true},
                      {workspace, need, true, need == 0}};
  st = check_buffers(bufs, 12);
  if (st != FLASHBOB_OK) return st;
  if (workspace_bytes < need) return FLASHBOB_ERR_INVALID_ARG;
  if (error_word_ptr(&a.err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  return paged_attn(a) == cudaSuccess ? FLASHBOB_OK : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_check_wait_timeout(void* stream) {
  unsigned int* err = nullptr;
  if (error_word_ptr(&err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  return launch_wait_timeout((cudaStream_t)stream, err) == cudaSuccess ? FLASHBOB_OK
                                                                       : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_mma_cycles(int n, int a_in_tmem, void* stream, double* cycles_per_mma) {
  if (cycles_per_mma == nullptr || n < 16 || n > 256 || n % 16 != 0)
    return FLASHBOB_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  if (error_word_ptr(&err) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  return mma_cycles(n, a_in_tmem != 0, (cudaStream_t)stream, err, cycles_per_mma) == cudaSuccess
             ? FLASHBOB_OK
             : FLASHBOB_ERR_CUDA;
}

flashbob_status flashbob_last_device_error(void) {
  unsigned int* p = nullptr;
  if (error_word_ptr(&p) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return FLASHBOB_ERR_CUDA;
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v)) != cudaSuccess) return FLASHBOB_ERR_CUDA;
  if (v != 0) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) != cudaSuccess)
      return FLASHBOB_ERR_CUDA;
    return FLASHBOB_ERR_TIMEOUT;
  }
  return FLASHBOB_OK;
}

}  // extern "C"
