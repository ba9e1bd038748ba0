// What the attention kernels on the 5th-generation tensor cores share.
#pragma once

#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvq {

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A box of 16-bit rows [token][head][channel], 64 channels wide.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int ch, int head, int token,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ch), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// acc + 0 * x for a pair: +-0 where x is finite.
template <bool BF16>
__device__ __forceinline__ uint32_t fma_zero(uint32_t x, uint32_t acc) {
  if (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  return acc;
}

template <int N>
__device__ __forceinline__ float max_of(const uint32_t* s) {
  float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
  for (int c = 0; c < N; c += 8) {
    t0 = fmaxf(fmaxf(t0, __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
    t1 = fmaxf(fmaxf(t1, __uint_as_float(s[c + 2])), __uint_as_float(s[c + 3]));
    t2 = fmaxf(fmaxf(t2, __uint_as_float(s[c + 4])), __uint_as_float(s[c + 5]));
    t3 = fmaxf(fmaxf(t3, __uint_as_float(s[c + 6])), __uint_as_float(s[c + 7]));
  }
  return fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
}

// 64 bytes of an output row: whole 32-byte sectors where `out` is so aligned.
__device__ __forceinline__ void store_row(uint16_t* to, const uint32_t* w, bool wide) {
  if (wide) {
#pragma unroll
    for (int q = 0; q < 16; q += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 2 * q), "r"(w[q]), "r"(w[q + 1]),
                   "r"(w[q + 2]), "r"(w[q + 3]), "r"(w[q + 4]), "r"(w[q + 5]), "r"(w[q + 6]), "r"(w[q + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int q = 0; q < 16; q += 4)
      *reinterpret_cast<uint4*>(to + 2 * q) = make_uint4(w[q], w[q + 1], w[q + 2], w[q + 3]);
  }
}

// 16-bit rows [tokens][heads][dim], `stride` elements between tokens, in boxes
// of 64 channels with the 128-byte swizzle.
inline cudaError_t encode_heads(CUtensorMap* m, const void* base, int dim, int heads, int tokens, int64_t stride,
                                bool bf16, int box_heads, int box_tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace kvq
