// Norm of query and key heads and rotation by position in one pass
// (kvq_norm_rotate).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * f_j
//
// Bound by bytes: every row is read once and written once. D / 8 lanes hold a
// head's row, eight channels each, such that both channels of a pair are in one
// lane: two runs of four, `rot / 2` apart (or side by side for neighbouring
// pairs), so the rotation needs no exchange and the norm one sum over the
// lanes. A lane's four pairs are the same in every head: a warp makes a token's
// sines and cosines once and takes the token's heads in turn.
//
// The angle is kept in turns as a 64-bit fraction: position * turns[j] mod 2^64
// is exact, its upper half goes to sincospif (2^-25 of half a turn off), so a
// position of a million is as good as one of ten.
//
// 32768 tokens of 40 heads of 128 (671 MB): 123 us, 5460 GB/s, 0.82 of the copy rate (127.6
// with the loads behind the sines). 16 tokens: 4.9 us, one launch (6.2).
#include "paged_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// `passes`: passes over 256 / D heads each that a warp makes of its token;
// `parts`: warps of a token. The first rows' loads go out before anything else is
// known, so that a small call takes one memory latency and not four.
template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kWarps * 32, 7) norm_rotate_kernel(const RotateArgs a, const int passes, const int parts) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a pass
  constexpr int kBatch = 4;                            // passes whose loads are in flight together
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int token = (int)(task / parts), part = (int)(task % parts);
  if (token >= a.tokens) return;
  const int heads = a.q_heads + a.k_heads;

  // the lane's channels: ch0 .. + 3 and ch1 .. + 3
  const bool turn = l < a.rot / 8;
  const bool apart = !INTERLEAVED && turn;
  const int ch0 = apart ? 4 * l : 8 * l, ch1 = apart ? a.rot / 2 + 4 * l : 8 * l + 4;

  const int first = part * passes * kHeads, last = min(heads, first + passes * kHeads);
  uint2 x[kBatch][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * kHeads + sub;
      if (h >= last) continue;
      const uint16_t* row = h < a.q_heads ? a.q + token * a.q_stride + (int64_t)h * D
                                          : a.k + token * a.k_stride + (int64_t)(h - a.q_heads) * D;
      x[i][0] = *reinterpret_cast<const uint2*>(row + ch0);
      x[i][1] = *reinterpret_cast<const uint2*>(row + ch1);
    }
  };
  load(first);
  const int position = a.positions[token];
  uint64_t turns[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) turns[j] = turn ? a.turns[4 * l + j] : 0;
  if (position < 0) return;
  float c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t t = (uint64_t)(uint32_t)position * turns[j] + (1ull << 31);
    sincospif((float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f, &s[j], &c[j]);
    c[j] *= a.magnitude, s[j] *= a.magnitude;
  }
#pragma unroll 1
  for (int h0 = first; h0 < last; h0 += kBatch * kHeads) {
    if (h0 > first) load(h0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * kHeads + sub;
      const bool is_q = h < a.q_heads;
      float v[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 p = unpack2<BF16>(x[i][j].x), q = unpack2<BF16>(x[i][j].y);
        v[4 * j] = p.x, v[4 * j + 1] = p.y, v[4 * j + 2] = q.x, v[4 * j + 3] = q.y;
      }
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (h >= last) continue;
      const float* weight = is_q ? a.q_weight : a.k_weight;
      if (weight) {
        const float r = rsqrtf(sum * (1.0f / D) + a.eps);
        const float4 w0 = *reinterpret_cast<const float4*>(weight + ch0), w1 = *reinterpret_cast<const float4*>(weight + ch1);
        v[0] = v[0] * r * w0.x, v[1] = v[1] * r * w0.y, v[2] = v[2] * r * w0.z, v[3] = v[3] * r * w0.w;
        v[4] = v[4] * r * w1.x, v[5] = v[5] * r * w1.y, v[6] = v[6] * r * w1.z, v[7] = v[7] * r * w1.w;
      }
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float& p = INTERLEAVED ? v[2 * j] : v[j];
          float& q = INTERLEAVED ? v[2 * j + 1] : v[4 + j];
          const float y = p * c[j] - q * s[j];
          q = q * c[j] + p * s[j];
          p = y;
        }
      }
      uint16_t* to = is_q ? a.q_out + token * a.q_out_stride + (int64_t)h * D
                          : a.k_out + token * a.k_out_stride + (int64_t)(h - a.q_heads) * D;
      *reinterpret_cast<uint2*>(to + ch0) = make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
      *reinterpret_cast<uint2*>(to + ch1) = make_uint2(pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
    }
  }
}

template <int D, bool BF16>
cudaError_t launch(const RotateArgs& a, cudaStream_t st) {
  constexpr int kHeads = 256 / D;
  const int all = (a.q_heads + a.k_heads + kHeads - 1) / kHeads;
  // Few passes: a warp for each, for latency; many: the sines of a token serve all its
  // heads. us with a warp a pass / for four / for the token, 40 heads of 128 (20 passes a token):
  //   tokens    16           64           128          256          512          2048           4096           8192
  //          2.2/2.7/7.6  2.5/2.7/7.7  2.9/2.9/7.7  4.6/3.4/7.9  7.1/4.2/8.0  22.6/10.4/10.9  44.5/19.1/17.2  91/38.4/33.8
  const int64_t work = (int64_t)a.tokens * all;
  const int parts = work < 2560 ? all : work < 51200 ? (all + 3) / 4 : 1, passes = (all + parts - 1) / parts;
  const int64_t grid = ((int64_t)a.tokens * parts + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (a.interleaved) norm_rotate_kernel<D, BF16, true><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, passes, parts);
  else norm_rotate_kernel<D, BF16, false><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, passes, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs& a, cudaStream_t st) {
  if (a.dim == 64) return a.dtype == KVQ_BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return a.dtype == KVQ_BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace kvq
