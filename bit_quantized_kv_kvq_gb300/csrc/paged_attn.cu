// Attention of several new tokens per request over the paged 8-bit cache
// (kvq_paged_attention).
//
//   e_t = c <q_i, k_hat_t>,  o_i = sum_{t <= p_i} softmax(e)_t v_hat_t,  x_hat = code * s(page, head)
//
// One CTA per (token, query head), a quarter of the keys to each of four warps,
// a key at a time: the plainest form, all of it in fp32.
#include "paged_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;

template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x) {
  if (BF16) return __uint_as_float((uint32_t)x << 16);
  return __half2float(__ushort_as_half(x));
}

template <int D, int CODE, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const PagedDev c, const PagedAttnArgs a) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, token = blockIdx.x, hq = blockIdx.y, h = hq / a.group;
  const int P = 1 << c.page_shift;
  int b = -1;
  for (int i0 = 0; i0 < a.requests && b < 0; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t mine = __ballot_sync(0xffffffffu, i < a.requests && a.cu[i] <= token && token < a.cu[i + 1]);
    if (mine) b = i0 + __ffs(mine) - 1;
  }
  if (b < 0) return;
  const int c0 = a.cu[b], m = a.cu[b + 1] - c0, n = a.lens[b];
  if (c0 < 0 || m > a.tokens - c0 || n < m || n > (int64_t)c.max_pages << c.page_shift) {
    if (threadIdx.x == 0) raise_status(c.status, kStatusBadIndex);
    return;
  }
  const int seen = n - m + (token - c0) + 1, full = n & ~(P - 1);
  float q[kPer], o[kPer], top = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = widen<BF16>(a.q[token * a.q_stride + (int64_t)hq * D + lane * kPer + i]);
    o[i] = 0.0f;
  }
  for (int t = warp; t < seen; t += kWarps) {
    float k[kPer], v[kPer];
    if (t < full) {
      const int page = a.table[(int64_t)b * c.max_pages + (t >> c.page_shift)];
      if (page < 0 || page >= c.num_pages) {
        if (lane == 0) raise_status(c.status, kStatusBadIndex);
        continue;
      }
      const int64_t ph = ((int64_t)page * c.heads + h) * 2;
      const float sk = c.scales[ph], sv = c.scales[ph + 1];
      const uint8_t* at = c.pages + (ph << c.page_shift) * D + (t & (P - 1)) * D + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint8_t x = at[i], y = at[P * D + i];
        if (CODE == KVQ_PAGE_INT8) {
          k[i] = (float)(int8_t)x * sk, v[i] = (float)(int8_t)y * sv;
        } else {
          uint32_t w;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"((uint16_t)(x | (y << 8))));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
          k[i] = f.x * sk, v[i] = f.y * sv;
        }
      }
    } else {
      const uint16_t* at = c.tails + (((((int64_t)b * c.heads + h) * 2) << c.page_shift) + (t - full)) * D + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; ++i) k[i] = widen<BF16>(at[i]), v[i] = widen<BF16>(at[P * D + i]);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float now = fmaxf(top, s), f = top == -INFINITY ? 0.0f : exp2f(top - now);
    const float p = now == -INFINITY ? 0.0f : exp2f(s - now);
    top = now;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + p * v[i];
  }
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  if (lane == 0) sm[warp] = top, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < kPer; ++i) so[warp][lane * kPer + i] = o[i];
  __syncthreads();
  if (threadIdx.x >= D) return;
  top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float r = 0.0f, sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    const float f = sm[w] == -INFINITY ? 0.0f : exp2f(sm[w] - top);
    r = sm[w] == -INFINITY && sl[w] == 0.0f ? r : r + f * so[w][threadIdx.x];
    sum += f * sl[w];
  }
  r /= sum;
  uint16_t* to = a.out + ((int64_t)token * a.q_heads + hq) * D + threadIdx.x;
  if (BF16) *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16(r);
  else *reinterpret_cast<__half*>(to) = __float2half(r);
}

template <int D, int CODE>
cudaError_t launch(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  const dim3 grid(a.tokens, a.q_heads);
  if (c.dtype == KVQ_BF16) paged_attn_kernel<D, CODE, true><<<grid, kWarps * 32, 0, st>>>(c, a);
  else paged_attn_kernel<D, CODE, false><<<grid, kWarps * 32, 0, st>>>(c, a);
  return cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace(int, int) { return 16; }

cudaError_t launch_paged_attention(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  if (c.code == KVQ_PAGE_INT8) return c.dim == 64 ? launch<64, KVQ_PAGE_INT8>(c, a, st) : launch<128, KVQ_PAGE_INT8>(c, a, st);
  return c.dim == 64 ? launch<64, KVQ_PAGE_E4M3>(c, a, st) : launch<128, KVQ_PAGE_E4M3>(c, a, st);
}

}  // namespace kvq
