// Decode attention over e4m3 pages.
#include "paged_decode.cuh"

namespace kvq {
cudaError_t launch_paged_decode_e4m3(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st) {
  return c.dim == 64 ? pdec::by_type<64, KVQ_PAGE_E4M3>(c, a, st) : pdec::by_type<128, KVQ_PAGE_E4M3>(c, a, st);
}
}  // namespace kvq
