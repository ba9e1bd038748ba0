// Chunk attention over e4m3 pages.
#include "paged_attn.cuh"

namespace kvq {

cudaError_t launch_paged_attention_e4m3(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  return c.dim == 64 ? patt::by_type<64, KVQ_PAGE_E4M3>(c, a, st) : patt::by_type<128, KVQ_PAGE_E4M3>(c, a, st);
}

}  // namespace kvq
