// Writing a step's packed keys and values into the paged 8-bit cache
// (kvq_paged_write).
//
// A page's scale is absmax / Q over its P tokens x D channels, so a page can be
// coded only when its last token is there; one CTA then holds the page's tile
// of one head in registers (K in one half of the threads, V in the other),
// reduces the absmax, and stores the codes: every input row is read once and
// every code written once. Rows of the page that came in earlier steps are in
// the request's tail; the rows of the new open page go there, by the CTA of
// the request's first item, which is the only one that reads that tail.
//
// Bound by bytes: 131072 fp16 tokens of 8 heads x 128 channels (805 MB) take
// 128 us, 6.27 TB/s, 0.92 of the measured copy rate. With an IEEE division a
// value it was bound by those (193 us); with 20 warps an SM by latency (151 us).
#include "paged_internal.h"

namespace kvq {
namespace {

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes of x / s, packed, by the IEEE quotient.
template <int CODE>
__device__ __forceinline__ uint32_t code4(const float* x, float s) {
  if (s == 0.0f) return 0u;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __fdiv_rn(x[i], s);
  if (CODE == KVQ_PAGE_E4M3) return e4m3_pair(y[0], y[1]) | (e4m3_pair(y[2], y[3]) << 16);
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (uint32_t)(max(-127, min(127, __float2int_rn(y[i]))) & 255) << (8 * i);
  return r;
}

// The same codes without a division: lo and hi are 1 / s less and more 2^-21
// of it, so the quotient, rounded however it may be, lies between x lo and
// x hi (1 / s and the product are within 2^-23). Rounding is monotone: where
// the codes of both ends are the same one it is the quotient's; `differ`
// collects where they are not (about one value in 10^5), and those take code4.
template <int CODE>
__device__ __forceinline__ uint32_t code4_fast(const float* x, float lo, float hi, uint32_t& differ) {
  if (CODE == KVQ_PAGE_E4M3) {
    const uint32_t a = e4m3_pair(x[0] * lo, x[1] * lo) | (e4m3_pair(x[2] * lo, x[3] * lo) << 16);
    const uint32_t b = e4m3_pair(x[0] * hi, x[1] * hi) | (e4m3_pair(x[2] * hi, x[3] * hi) << 16);
    differ |= a ^ b;
    return a;
  }
  constexpr float kInt = 12582912.0f;  // 1.5 * 2^23: the sum's last bit is 1, its low byte the rounded integer
  uint32_t a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(__fmaf_rn(x[i], lo, kInt));
    differ |= a[i] ^ __float_as_uint(__fmaf_rn(x[i], hi, kInt));
  }
  return __byte_perm(__byte_perm(a[0], a[1], 0x0040), __byte_perm(a[2], a[3], 0x0040), 0x5410);
}

// P tokens, D channels. A granule is 16 channels of a row (32 bytes in, 16
// out); a thread holds kGran of them.
template <int P, int D, int CODE, bool BF16>
struct WriteCfg {
  static constexpr int kGranules = P * D / 16;
  static constexpr int kGran = P * D <= 4096 ? 2 : 4;
  static constexpr int kHalf = kGranules / kGran;  // threads per tensor
  static constexpr int kThreads = 2 * kHalf;
};

// 64 registers a thread: 1024 threads of an SM, 128 KB of rows on their way.
template <int P, int D, int CODE, bool BF16>
__global__ void __launch_bounds__(WriteCfg<P, D, CODE, BF16>::kThreads, 1024 / WriteCfg<P, D, CODE, BF16>::kThreads)
    paged_write_kernel(const PagedDev c, const PagedWriteArgs a) {
  using Cfg = WriteCfg<P, D, CODE, BF16>;
  constexpr int kRowGran = D / 16;
  // heads run fastest: CTAs that run together read whole token rows
  const int h = blockIdx.x % c.heads;
  const int32_t* cu = a.cu;
  // items of request b start at floor(cu[b] / P) + b: room for ceil(m / P) of them
  const int w = blockIdx.x / c.heads;
  const int b = warp_last_le(a.requests, w, [&](int i) { return (int)((uint32_t)cu[i] / P) + i; });
  const int c0 = cu[b], m = cu[b + 1] - c0;
  if (m <= 0) return;
  const int j = w - (c0 / P + b);
  const int new_len = a.lens[b], old = new_len - m;
  if (c0 < 0 || m > a.max_tokens - c0 || new_len < m) {
    if (threadIdx.x == 0) raise_status(c.status, kStatusBadIndex);
    return;
  }
  if (j < 0) return;  // before the first request's
  const int page0 = old / P, pages = new_len / P - page0;  // completed in this call
  const int half = threadIdx.x / Cfg::kHalf;               // 0: keys, 1: values
  const int tid = threadIdx.x - half * Cfg::kHalf;
  const uint16_t* in = half ? a.v : a.k;
  const int64_t stride = half ? a.v_stride : a.k_stride;
  uint16_t* tail = c.tails + (((int64_t)b * c.heads + h) * 2 + half) * (P * D);

  if (j < pages) {
    uint4 x[Cfg::kGran][2];
    uint32_t top = 0;
    const int start = (page0 + j) * P;  // position of the page's first token
    const int slot = a.slots[c0 + start + P - 1 - old];  // of the page's last token
#pragma unroll
    for (int i = 0; i < Cfg::kGran; ++i) {
      const int gr = i * Cfg::kHalf + tid, row = gr / kRowGran, ch = (gr % kRowGran) * 16;
      const int t = start + row - old;  // the row's place among the request's new tokens
      const uint16_t* src = t >= 0 ? in + (int64_t)(c0 + t) * stride + h * D + ch : tail + row * D + ch;
      x[i][0] = *reinterpret_cast<const uint4*>(src);
      x[i][1] = *reinterpret_cast<const uint4*>(src + 8);
      // |x| as an integer: NaN sorts above infinity, so it reaches the scale
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (uint32_t word : {x[i][q].x, x[i][q].y, x[i][q].z, x[i][q].w})
          top = __vmaxu2(top, word & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    __shared__ uint32_t wtop[32];
    if ((threadIdx.x & 31) == 0) wtop[threadIdx.x >> 5] = top;
    __syncthreads();  // also: every read of the tail is done
    constexpr int kWarps = Cfg::kHalf / 32;
    top = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = max(top, wtop[half * kWarps + i]);
    const float s = __fdiv_rn(unpack2<BF16>(top).x, CODE == KVQ_PAGE_INT8 ? 127.0f : 448.0f);
    const int page = slot >> c.page_shift;
    if (slot < 0 || page >= c.num_pages || (slot & (P - 1)) != P - 1) {
      if (threadIdx.x == 0) raise_status(c.status, kStatusBadIndex);
    } else {
      const int64_t ph = ((int64_t)page * c.heads + h) * 2 + half;
      uint8_t* dst = c.pages + ph * (P * D);
      // page-uniform: 1 / s and its products stay normal numbers
      const bool fast = s > 0x1p-100f && s < 0x1p100f;
      const float r = __frcp_rn(fast ? s : 1.0f), lo = r * (1.0f - 0x1p-21f), hi = r * (1.0f + 0x1p-21f);
#pragma unroll
      for (int i = 0; i < Cfg::kGran; ++i) {
        uint32_t o[4], differ = fast ? 0u : 1u;
        float f[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t u[4] = {x[i][q].x, x[i][q].y, x[i][q].z, x[i][q].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2<BF16>(u[k]);
            f[8 * q + 2 * k] = v.x;
            f[8 * q + 2 * k + 1] = v.y;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = code4_fast<CODE>(f + 4 * q, lo, hi, differ);
        if (differ) {
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = code4<CODE>(f + 4 * q, s);
        }
        *reinterpret_cast<uint4*>(dst + (i * Cfg::kHalf + tid) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (tid == 0) c.scales[ph] = s;
    }
  }
  if (j == 0) {  // the rows of the new open page
    const int open = new_len / P * P, from = open > old ? open : old;
    const int n8 = (new_len - from) * (D / 8);
    for (int i = tid; i < n8; i += Cfg::kHalf) {
      const int pos = from + i / (D / 8), ch = (i % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(tail + (pos - open) * D + ch) =
          *reinterpret_cast<const uint4*>(in + (int64_t)(c0 + pos - old) * stride + h * D + ch);
    }
  }
}

template <int P, int D, int CODE, bool BF16>
cudaError_t launch(const PagedDev& c, const PagedWriteArgs& a, cudaStream_t st) {
  const int64_t grid = (int64_t)(a.max_tokens / P + a.requests) * c.heads;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  paged_write_kernel<P, D, CODE, BF16><<<(unsigned)grid, WriteCfg<P, D, CODE, BF16>::kThreads, 0, st>>>(c, a);
  return cudaGetLastError();
}

template <int P, int D>
cudaError_t by_type(const PagedDev& c, const PagedWriteArgs& a, cudaStream_t st) {
  if (c.code == KVQ_PAGE_INT8)
    return c.dtype == KVQ_BF16 ? launch<P, D, KVQ_PAGE_INT8, true>(c, a, st) : launch<P, D, KVQ_PAGE_INT8, false>(c, a, st);
  return c.dtype == KVQ_BF16 ? launch<P, D, KVQ_PAGE_E4M3, true>(c, a, st) : launch<P, D, KVQ_PAGE_E4M3, false>(c, a, st);
}

template <int D>
cudaError_t by_page(const PagedDev& c, const PagedWriteArgs& a, cudaStream_t st) {
  switch (c.page_shift) {
    case 4: return by_type<16, D>(c, a, st);
    case 5: return by_type<32, D>(c, a, st);
    case 6: return by_type<64, D>(c, a, st);
    default: return by_type<128, D>(c, a, st);
  }
}

}  // namespace

cudaError_t launch_paged_write(const PagedDev& c, const PagedWriteArgs& a, cudaStream_t st) {
  return c.dim == 64 ? by_page<64>(c, a, st) : by_page<128>(c, a, st);
}

}  // namespace kvq
