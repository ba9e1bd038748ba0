// Chunk attention over int8 pages.
#include "paged_attn.cuh"

namespace kvq {

cudaError_t launch_paged_attention_e4m3(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st);

cudaError_t launch_paged_attention_int8(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  return c.dim == 64 ? patt::by_type<64, KVQ_PAGE_INT8>(c, a, st) : patt::by_type<128, KVQ_PAGE_INT8>(c, a, st);
}

size_t paged_attn_workspace(int dim, int sm_count) {
  return patt::pos_bytes(sm_count) + (size_t)sm_count * 4 * patt::kRows * (dim + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  return c.code == KVQ_PAGE_INT8 ? launch_paged_attention_int8(c, a, st) : launch_paged_attention_e4m3(c, a, st);
}

}  // namespace kvq
