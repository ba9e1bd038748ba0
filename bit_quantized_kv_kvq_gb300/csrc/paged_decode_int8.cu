// Decode attention over int8 pages, and the dispatch by code type.
#include "paged_decode.cuh"

namespace kvq {

cudaError_t launch_paged_decode_e4m3(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st);

size_t paged_decode_workspace(int dim, int group, int requests, int sm_count) {
  const int nt = pdec::nt_of(group), passes = (group + 8 * nt - 1) / (8 * nt);
  return pdec::prefix_bytes(requests) +
         (size_t)sm_count * pdec::ctas_per_sm(nt) * 2 * passes * 8 * nt * (dim + 2) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st) {
  if (c.code == KVQ_PAGE_E4M3) return launch_paged_decode_e4m3(c, a, st);
  return c.dim == 64 ? pdec::by_type<64, KVQ_PAGE_INT8>(c, a, st) : pdec::by_type<128, KVQ_PAGE_INT8>(c, a, st);
}

}  // namespace kvq
