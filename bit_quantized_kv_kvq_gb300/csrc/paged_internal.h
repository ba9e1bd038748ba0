// Structures shared by the paged cache's host side and its kernels.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace kvq {

// Status bits of the paged calls, beside kStatusTimeout and kStatusBadState.
constexpr uint32_t kStatusNoRoom = 1u << 2;   // a reserve did not fit
constexpr uint32_t kStatusBadIndex = 1u << 3; // a length, slot, page or count out of range

constexpr int kMaxRequests = 4096;

// One layer of a paged cache, device side.
struct PagedDev {
  uint8_t* pages;   // [num_pages][H][2][P][D]
  float* scales;    // [num_pages][H][2]
  uint16_t* tails;  // [max_requests][H][2][P][D]
  int heads;        // kv-heads
  int dim;          // 64 or 128
  int page_shift;   // log2(page_tokens)
  int num_pages;
  int max_pages;    // entries of a table row
  int code;         // kvq_page_code
  int dtype;        // KVQ_F16 or KVQ_BF16
  uint32_t* status;
};

struct ReserveArgs {
  int requests, page_shift, num_pages, max_pages, max_tokens;
  const int32_t *lens, *add, *free_pages, *free_count;
  int32_t *table, *cu, *slots, *positions, *lens_out, *free_count_out;
  uint32_t* status;
};
int reserve_launches(int max_tokens);
cudaError_t launch_reserve(const ReserveArgs& a, cudaStream_t st);

struct ReleaseArgs {
  int requests, page_shift, num_pages, max_pages;
  const int32_t *done, *table;
  int32_t *lens, *free_pages, *free_count;
  uint32_t* status;
};
cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t st);

struct PagedWriteArgs {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;  // elements between tokens
  int max_tokens, requests;
  const int32_t *cu, *slots, *lens;  // lens: after the step
};
cudaError_t launch_paged_write(const PagedDev& c, const PagedWriteArgs& a, cudaStream_t st);

struct PagedDecodeArgs {
  const uint16_t* q;
  int64_t q_stride;
  int requests, q_heads, group;  // group: query heads per kv-head
  const int32_t *table, *lens;
  float scale_log2;
  void* out;
  int out_f32;
  void* ws;
  int sm_count;
};
size_t paged_decode_workspace(int dim, int group, int requests, int sm_count);
cudaError_t launch_paged_decode(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st);

struct PromptArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int tokens, seqs, q_heads, kv_heads, dim, dtype;
  const int32_t* cu;
  float scale_log2;
  uint16_t* out;
  uint32_t* status;
};
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t st);

// The last index b in [0, n) with key(b) <= x, for keys in ascending order and
// key(0) <= x. A whole warp calls it: 32 probes a step, so that the search
// costs one memory latency per factor of 32.
template <typename F>
__device__ __forceinline__ int warp_last_le(int n, int x, F key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && key(lo + at) <= x;
    const int c = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    const int skip = (c < 0 ? 0 : c) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return lo;
}

}  // namespace kvq
