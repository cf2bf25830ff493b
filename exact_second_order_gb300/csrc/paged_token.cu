// Attention over a paged cache: which kernel takes a call.
#include "paged.cuh"

namespace flashbob {

size_t paged_workspace(const PagedAttnArgs& a) {
  const int splits = simt_splits(a);
  return splits == 1 ? 0
                     : attn::partial_bytes(static_cast<size_t>(a.B) * a.H * a.Nq, a.d, splits);
}

cudaError_t paged_attn(const PagedAttnArgs& a) { return simt_paged(a); }

}  // namespace flashbob
