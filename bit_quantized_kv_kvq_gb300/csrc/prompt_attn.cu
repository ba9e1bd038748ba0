// Causal attention over packed prompts on their own keys and values
// (kvq_prompt_attention).
//
//   o_i = sum_{t <= i} softmax(c <q_i, k_t>)_t v_t
//
// One pass over the keys per block of query rows, with the running maximum m
// and sum l of the exponentials: a tile's weights are 2^(e - m), and a tile
// that raises m scales o and l by 2^(m_old - m_new). The products run on the
// tensor cores in the input type with fp32 sums; P is rounded to that type,
// whose rounding (2^-12 or 2^-9 of each weight, zero mean) is that of an
// output element.
#include "paged_internal.h"

namespace kvq {
namespace {

constexpr int kRows = 64;    // query rows of a CTA
constexpr int kCols = 64;    // keys of a tile
constexpr int kThreads = 128;
constexpr int kNever = 0x7fffffff;

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const PromptArgs a) {
  constexpr int kPad = D + 8;
  __shared__ __align__(16) uint16_t ks[kCols][kPad];
  __shared__ __align__(16) uint16_t vs[kCols][kPad];
  // the first token of this CTA's masked tiles whose value is NaN, +inf, -inf, per channel
  __shared__ int first[3][D];
  __shared__ int any_nonfinite;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int w = gridDim.x - 1 - blockIdx.x, hq = blockIdx.y, h = hq / (a.q_heads / a.kv_heads);
  const int* cu = a.cu;
  // tiles of sequence s start at floor(cu[s] / rows) + s: room for all of them
  const int s = warp_last_le(a.seqs, w, [&](int i) { return (int)((uint32_t)cu[i] / kRows) + i; });
  const int c0 = cu[s], n = cu[s + 1] - c0;
  if (n <= 0) return;
  const int tile = w - (c0 / kRows + s);
  if (c0 < 0 || n > a.tokens - c0 || tile < 0) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(a.status, kStatusBadIndex);
    return;
  }
  const int q0 = tile * kRows;
  if (q0 >= n) return;
  const uint16_t* qp = a.q + (int64_t)c0 * a.q_stride + (int64_t)hq * D;
  const uint16_t* kp = a.k + (int64_t)c0 * a.k_stride + (int64_t)h * D;
  const uint16_t* vp = a.v + (int64_t)c0 * a.v_stride + (int64_t)h * D;

  for (int i = threadIdx.x; i < 3 * D; i += kThreads) first[i / D][i % D] = kNever;
  if (threadIdx.x == 0) any_nonfinite = 0;

  const int r0 = q0 + warp * 16 + g, r1 = r0 + 8;
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const int ch = i * 16 + 2 * t4;
    qf[i][0] = r0 < n ? *reinterpret_cast<const uint32_t*>(qp + r0 * a.q_stride + ch) : 0u;
    qf[i][1] = r1 < n ? *reinterpret_cast<const uint32_t*>(qp + r1 * a.q_stride + ch) : 0u;
    qf[i][2] = r0 < n ? *reinterpret_cast<const uint32_t*>(qp + r0 * a.q_stride + ch + 8) : 0u;
    qf[i][3] = r1 < n ? *reinterpret_cast<const uint32_t*>(qp + r1 * a.q_stride + ch + 8) : 0u;
  }
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) o[i][r] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  for (int k0 = 0; k0 < q0 + kRows && k0 < n; k0 += kCols) {
    const bool masked = k0 + kCols > q0;
    __syncthreads();
    for (int i = threadIdx.x; i < kCols * (D / 8); i += kThreads) {
      const int r = i / (D / 8), ch = i % (D / 8) * 8, tok = k0 + r;
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      if (tok < n) {
        x = *reinterpret_cast<const uint4*>(kp + tok * a.k_stride + ch);
        y = *reinterpret_cast<const uint4*>(vp + tok * a.v_stride + ch);
      }
      if (masked) {
        // 0 * inf would carry a later token's infinity or NaN to an earlier
        // row: the tensor cores get 0 there, the rows from it on are set at the end
        constexpr uint16_t kInf = BF16 ? 0x7f80 : 0x7c00;
        uint16_t* e = reinterpret_cast<uint16_t*>(&y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((e[j] & kInf) == kInf) {
            const int kind = (e[j] & 0x7fff) != kInf ? 0 : (e[j] >> 15) ? 2 : 1;
            atomicMin(&first[kind][ch + j], tok);
            any_nonfinite = 1;
            e[j] = 0;
          }
      }
      *reinterpret_cast<uint4*>(&ks[r][ch]) = x;
      *reinterpret_cast<uint4*>(&vs[r][ch]) = y;
    }
    __syncthreads();
    float sc[kCols / 8][4];
#pragma unroll
    for (int j = 0; j < kCols / 8; ++j) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sc[j][r] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t b[4];
        ldm4(b, &ks[j * 8 + (lane & 7)][i * 32 + (lane >> 3) * 8]);
        mma16816<BF16>(sc[j], qf[2 * i], b[0], b[1]);
        mma16816<BF16>(sc[j], qf[2 * i + 1], b[2], b[3]);
      }
    }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int j = 0; j < kCols / 8; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = k0 + j * 8 + 2 * t4 + (r & 1);
        float e = sc[j][r] * a.scale_log2;
        if (masked && tok > (r < 2 ? r0 : r1)) e = -INFINITY;
        sc[j][r] = e;
        top[r >> 1] = fmaxf(top[r >> 1], e);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float f = top[r] == -INFINITY ? 1.0f : exp2_fast(m[r] - top[r]);
      m[r] = top[r];
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][2 * r] *= f, o[i][2 * r + 1] *= f;
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j) {
      uint32_t p[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[r] = exp2_fast(sc[2 * j + q][r] - ref[r >> 1]);
          l[r >> 1] += e[r];
        }
        p[2 * q] = pack2<BF16>(e[0], e[1]);
        p[2 * q + 1] = pack2<BF16>(e[2], e[3]);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldm4t(b, &vs[j * 16 + (lane & 15)][i * 16 + (lane >> 4) * 8]);
        mma16816<BF16>(o[2 * i], p, b[0], b[1]);
        mma16816<BF16>(o[2 * i + 1], p, b[2], b[3]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = r ? r1 : r0;
    if (row >= n) continue;
    uint16_t* op = a.out + ((int64_t)(c0 + row) * a.q_heads + hq) * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      float x = o[i][2 * r] / l[r], y = o[i][2 * r + 1] / l[r];
      const int ch = i * 8 + 2 * t4;
      if (any_nonfinite) {
        if (row >= first[1][ch]) x += INFINITY;
        if (row >= first[2][ch]) x -= INFINITY;
        if (row >= first[0][ch]) x = NAN;
        if (row >= first[1][ch + 1]) y += INFINITY;
        if (row >= first[2][ch + 1]) y -= INFINITY;
        if (row >= first[0][ch + 1]) y = NAN;
      }
      *reinterpret_cast<uint32_t*>(op + ch) = pack2<BF16>(x, y);
    }
  }
}

template <int D>
cudaError_t launch(const PromptArgs& a, cudaStream_t st) {
  const dim3 grid(a.tokens / kRows + a.seqs, a.q_heads);
  if (a.dtype == KVQ_BF16) prompt_kernel<D, true><<<grid, kThreads, 0, st>>>(a);
  else prompt_kernel<D, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t st) {
  return a.dim == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace kvq
