// Decode attention over the paged 8-bit cache (kvq_paged_decode_attention).
//
//   e_t = c <q, k_hat_t>,  o = sum_t softmax(e)_t v_hat_t,  x_hat = code * s(page, head)
//
// The step is bound by the bytes of codes it reads: 2 L H D per request,
// against 4 L H_q D operations. So the codes go straight from global memory
// into the registers that the tensor cores read them from, and nothing is
// staged: per warp and 16 tokens,
//   S^T = K Q^T   A = K codes (16 tokens x 16 channels), B = Q (8 heads),
//   O^T += s_v V^T P^T   A = V codes (16 channels x 16 tokens), B = P^T,
// both m16n8k16 in fp16 with fp32 sums. Every code (int8 or e4m3) is an exact
// fp16 number, so only P is rounded (2^-11 of each weight). Tokens and
// channels may be summed in any order, so a lane loads 16 contiguous bytes
// and calls them the fragment's slots.
//
// The tiles (64 or 128 tokens of one request and kv-head) of all requests form one
// line that is cut into equal ranges, one per CTA: the kernel makes the line
// from the device lengths itself, so the grid needs no host knowledge and
// ragged batches stay even. A CTA's four warps take 16 tokens of a tile each
// (32 with 64 channels: as many bytes in flight) and keep their own running maximum and sums. A (request, head) that one CTA
// covers is finished there; the others leave partial sums, which a second
// kernel merges in the order of the CTAs.
#pragma once

#include "paged_internal.h"

namespace kvq {
namespace pdec {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

// Groups of 16 tokens that a warp takes of a tile, and the tile's tokens.
__host__ __device__ constexpr int sub_of(int dim) { return 128 / dim; }
__host__ __device__ constexpr int unit_of(int dim) { return kWarps * 16 * sub_of(dim); }

// Heads of one pass over the codes: 8 NT (NT column tiles of the products).
__host__ __device__ constexpr int nt_of(int group) { return group <= 8 ? 1 : 2; }
// CTAs per SM that the registers allow.
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 4 : 2; }

// Workspace: int prefix[requests + 1] of tiles (one kv-head), then partial
// rows [ctas][2][passes][8 NT][D + 2]: o[D], m, l.
__host__ __device__ inline size_t prefix_bytes(int requests) { return ((size_t)(requests + 1) * 4 + 255) / 256 * 256; }

struct Params {
  PagedDev c;
  PagedDecodeArgs a;
  int ctas, passes;
  int* prefix;
  float* part;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of fp16 pairs across the warp: lane 4r + c holds row r,
// columns 2c, 2c + 1; it gets column r, rows 2c, 2c + 1.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The four codes of a word as two fp16 pairs (bytes 0, 1 and bytes 2, 3).
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (CODE == KVQ_PAGE_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 0x6400 | u is 1024 + u in fp16; u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Exponent k with max |x| * 2^k in [2^14, 2^15), from the bits of max |x| in
// bf16: rows in bf16 go to the fp16 products scaled by 2^k. That is exact but
// for elements below 2^-29 of the row's largest, whose rounding (2^-40 of it)
// is far below the fp32 sums' own.
__device__ __forceinline__ int bf16_shift(uint32_t top_bits) {
  const int k = 14 - ((int)(top_bits >> 7) - 127);
  return k > 100 ? 100 : k;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A bf16 pair times f, as an fp16 pair.
__device__ __forceinline__ uint32_t bf2_to_h2(uint32_t w, float f) {
  return pack_h2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t both_halves(uint32_t top) {
  const uint32_t a = top & 0xffffu, b = top >> 16;
  return a > b ? a : b;
}

template <int D, int CODE, bool BF16, int NT>
struct Warp {
  static constexpr int kSteps = D / 16;   // k-steps of S, row tiles of O
  static constexpr int kChunks = D / 64;  // 16-byte chunks of a key row per lane
  static constexpr int kVw = D / 32;      // words of a value row per lane
  uint32_t qf[NT][kSteps][2];
  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2], qs[NT][2];  // heads 2 t4, 2 t4 + 1 of the column tile

  // Queries of heads [h0, h0 + heads) and the empty running state.
  __device__ __forceinline__ void begin(const uint16_t* q, int heads, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool live = nt * 8 + g < heads;
      const uint16_t* row = q + (int64_t)(live ? nt * 8 + g : 0) * D;
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + ((s >> 2) * 4 + t) * 16 + (s & 3) * 4);
        qf[nt][s][0] = live ? w.x : 0u;
        qf[nt][s][1] = live ? w.y : 0u;
        top = abs_max2(abs_max2(top, qf[nt][s][0]), qf[nt][s][1]);
      }
      float f = scale_log2;
      if (BF16) {
        top = both_halves(top);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int k = bf16_shift(top);
        const float up = exp2i(k);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          qf[nt][s][0] = bf2_to_h2(qf[nt][s][0], up);
          qf[nt][s][1] = bf2_to_h2(qf[nt][s][1], up);
        }
        f *= exp2i(-k);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[nt][i] = __shfl_sync(kFull, f, (2 * t + i) * 4);
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[nt][j][r] = 0.0f;
    }
  }

  // Weights of 16 tokens from their scores s (c0, c1: token g; c2, c3: token
  // g + 8), as the B operand of P^T. fa, fb: factors of the two token rows.
  __device__ __forceinline__ void weights(float (&s)[NT][4], float fa, float fb, bool va, bool vb,
                                          uint32_t (&p)[NT][2]) {
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[nt][i] = va ? s[nt][i] * (qs[nt][i] * fa) : -INFINITY;
        s[nt][2 + i] = vb ? s[nt][2 + i] * (qs[nt][i] * fb) : -INFINITY;
        up |= fmaxf(s[nt][i], s[nt][2 + i]) > m[nt][i] + 8.0f;
      }
    }
    // The reference of the exponentials moves only when a score passes it by
    // 8: weights stay below 2^8, and most tiles skip the reduction.
    if (__any_sync(kFull, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(s[nt][i], s[nt][2 + i]);
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
          const bool mine = x > m[nt][i] + 8.0f;  // each head by its own scores
          const float f = mine ? exp2_fast(m[nt][i] - x) : 1.0f;
          m[nt][i] = mine ? x : m[nt][i];
          l[nt][i] *= f;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) o[nt][j][i] *= f, o[nt][j][2 + i] *= f;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
        s[nt][i] = exp2_fast(s[nt][i] - ref);
        s[nt][2 + i] = exp2_fast(s[nt][2 + i] - ref);
        l[nt][i] += s[nt][i] + s[nt][2 + i];
      }
      p[nt][0] = movmatrix(pack_h2(s[nt][0], s[nt][1]));
      p[nt][1] = movmatrix(pack_h2(s[nt][2], s[nt][3]));
    }
  }

  // O^T += sv * V^T P^T for one 16-channel row tile.
  __device__ __forceinline__ void add_pv(int j, float sv, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t (&p)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma16816(d, a0, a1, a2, a3, p[nt][0], p[nt][1]);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[nt][j][r] = fmaf(sv, d[r], o[nt][j][r]);
    }
  }

  __device__ __forceinline__ void load_k(const uint8_t* k, uint4 (&kr)[2][kChunks]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        kr[r][c] = __ldcs(reinterpret_cast<const uint4*>(k + (g + 8 * r) * D + (c * 4 + t) * 16));
  }
  __device__ __forceinline__ void load_v(const uint8_t* v, uint32_t (&vr)[4][kVw]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* src = v + (2 * t + (r & 1) + (r >> 1) * 8) * D + g * (D / 8);
      if (D == 128) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src));
        vr[r][0] = w.x, vr[r][1] = w.y, vr[r][2 % kVw] = w.z, vr[r][3 % kVw] = w.w;
      } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
        vr[r][0] = w.x, vr[r][1] = w.y;
      }
    }
  }

  __device__ __forceinline__ void scores(const uint4 (&kr)[2][kChunks], float (&s)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nt][r] = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t wa[4] = {kr[0][c].x, kr[0][c].y, kr[0][c].z, kr[0][c].w};
      const uint32_t wb[4] = {kr[1][c].x, kr[1][c].y, kr[1][c].z, kr[1][c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a0, a1, a2, a3;
        codes_to_half<CODE>(wa[i], a0, a2);
        codes_to_half<CODE>(wb[i], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a0, a1, a2, a3, qf[nt][c * 4 + i][0], qf[nt][c * 4 + i][1]);
      }
    }
  }

  __device__ __forceinline__ void values(const uint32_t (&vr)[4][kVw], float sv, const uint32_t (&p)[NT][2]) {
#pragma unroll
    for (int w = 0; w < kVw; ++w) {
      // bytes of two token rows side by side: (r0.b0, r1.b0, r0.b1, r1.b1), ...
      const uint32_t x = __byte_perm(vr[0][w], vr[1][w], 0x5140), y = __byte_perm(vr[0][w], vr[1][w], 0x7362);
      const uint32_t z = __byte_perm(vr[2][w], vr[3][w], 0x5140), u = __byte_perm(vr[2][w], vr[3][w], 0x7362);
      uint32_t a0, a1, a2, a3;
      codes_to_half<CODE>(x, a0, a1);
      codes_to_half<CODE>(z, a2, a3);
      add_pv(2 * w, sv, a0, a1, a2, a3, p);
      codes_to_half<CODE>(y, a0, a1);
      codes_to_half<CODE>(u, a2, a3);
      add_pv(2 * w + 1, sv, a0, a1, a2, a3, p);
    }
  }

  // 16 rows of the tail, `live` of them cached: the same products on the
  // input type's rows. k, v: the tail's rows at the first of them.
  __device__ __forceinline__ void tail_rows(const uint16_t* k, const uint16_t* v, int live) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float s[NT][4];
    float f[2] = {1.0f, 1.0f};
    uint32_t kw[2][kChunks][8];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(k + row * D + (c * 4 + t) * 16);
        const uint4 x = row < live ? src[0] : zero, y = row < live ? src[1] : zero;
        kw[r][c][0] = x.x, kw[r][c][1] = x.y, kw[r][c][2] = x.z, kw[r][c][3] = x.w;
        kw[r][c][4] = y.x, kw[r][c][5] = y.y, kw[r][c][6] = y.z, kw[r][c][7] = y.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = abs_max2(top, kw[r][c][i]);
      }
      if (BF16) {
        top = both_halves(top);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int e = bf16_shift(top);
        const float up = exp2i(e);
        f[r] = exp2i(-e);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) kw[r][c][i] = bf2_to_h2(kw[r][c][i], up);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nt][r] = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(s[nt], kw[0][c][2 * i], kw[1][c][2 * i], kw[0][c][2 * i + 1], kw[1][c][2 * i + 1],
                   qf[nt][c * 4 + i][0], qf[nt][c * 4 + i][1]);
    uint32_t p[NT][2];
    weights(s, f[0], f[1], g < live, g + 8 < live, p);
    uint32_t vw[4][D / 16];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * t + (r & 1) + (r >> 1) * 8;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 x = row < live ? reinterpret_cast<const uint4*>(v + row * D + g * (D / 8))[c] : zero;
        vw[r][4 * c] = x.x, vw[r][4 * c + 1] = x.y, vw[r][4 * c + 2] = x.z, vw[r][4 * c + 3] = x.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = abs_max2(top, vw[r][4 * c + i]);
      }
    }
    float sv = 1.0f;
    if (BF16) {  // one power of two for the 16 rows
      const int e = bf16_shift(__reduce_max_sync(kFull, both_halves(top)));
      const float up = exp2i(e);
      sv = exp2i(-e);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) vw[r][i] = bf2_to_h2(vw[r][i], up);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)  // channels 2 j and 2 j + 1 of the lane's D / 8
      add_pv(j, sv, __byte_perm(vw[0][j], vw[1][j], 0x5410), __byte_perm(vw[0][j], vw[1][j], 0x7632),
             __byte_perm(vw[2][j], vw[3][j], 0x5410), __byte_perm(vw[2][j], vw[3][j], 0x7632), p);
  }
};

// A tile's codes of one head, and its scales.
struct TilePtr {
  const uint8_t* k;
  float ks, vs;
};

template <int D, int CODE, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) paged_decode_kernel(const Params prm) {
  using W = Warp<D, CODE, BF16, NT>;
  constexpr int kSub = sub_of(D), kUnit = unit_of(D);
  const PagedDev& c = prm.c;
  const PagedDecodeArgs& a = prm.a;
  extern __shared__ int prefix[];  // [requests + 1]
  __shared__ float so[kWarps][8 * NT][D + 1];
  __shared__ float sml[kWarps][8 * NT][2];
  __shared__ int wsum[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int R = a.requests, P = 1 << c.page_shift;
  const int most = c.max_pages << c.page_shift;

  // prefix sums of the requests' tiles
  const int per = (R + kThreads - 1) / kThreads;
  int sum = 0;
  bool bad = false;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    int n = b < R ? a.lens[b] : 0;
    if (n < 0 || n > most) bad = true, n = 0;
    sum += (n + kUnit - 1) / kUnit;
  }
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) raise_status(c.status, kStatusBadIndex);
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int i = 0; i < warp; ++i) at += wsum[i];
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b < R) {
      prefix[b] = at;
      int n = a.lens[b];
      if (n < 0 || n > most) n = 0;
      at += (n + kUnit - 1) / kUnit;
      if (b == R - 1) prefix[R] = at;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b <= R; b += kThreads) prm.prefix[b] = prefix[b];

  const long long units = (long long)prefix[R] * c.heads;
  const int ctas = units < prm.ctas ? (int)units : prm.ctas;  // each of these has a tile at least
  if ((int)blockIdx.x >= ctas) return;
  const long long u1 = units * (blockIdx.x + 1) / ctas;
  long long u = units * blockIdx.x / ctas;
  while (u < u1) {
    // the request, head and tiles [t0, t1) that start at unit u
    int b = 0;
    {
      int n = R;
      while (n > 1) {  // last b with prefix[b] * heads <= u (equal ones: empty requests before it)
        const int half = n >> 1;
        if ((long long)prefix[b + half] * c.heads <= u) b += half, n -= half;
        else n = half;
      }
    }
    const int tiles = prefix[b + 1] - prefix[b];
    const long long in_b = u - (long long)prefix[b] * c.heads;
    const int h = (int)(in_b / tiles), t0 = (int)(in_b % tiles);
    const int t1 = (int)(u1 - u < tiles - t0 ? t0 + (u1 - u) : tiles);
    const int len = a.lens[b];
    const int full = len & ~(P - 1);  // tokens in complete pages
    const int head0 = h * a.group + blockIdx.y * 8 * NT;
    const int heads = min(8 * NT, a.group - (int)blockIdx.y * 8 * NT);

    W w;
    w.begin(a.q + b * a.q_stride + (int64_t)head0 * D, heads, a.scale_log2);
    const int32_t* row = a.table + (int64_t)b * c.max_pages;

    auto tile_of = [&](int page, int tok, bool live) {
      TilePtr p;
      const bool ok = page >= 0 && page < c.num_pages;
      if (!ok && live && lane == 0) raise_status(c.status, kStatusBadIndex);
      const int64_t ph = ((int64_t)(ok ? page : 0) * c.heads + h) * 2;
      p.k = c.pages + (ph << c.page_shift) * D + (tok & (P - 1)) * D;
      const float2 s = *reinterpret_cast<const float2*>(c.scales + ph);
      p.ks = s.x;
      p.vs = s.y;
      if (!ok) p.k = nullptr;
      return p;
    };
    const int end = t1 * kUnit, page_end = min(end, full);
    int tok = t0 * kUnit + warp * 16 * kSub;
    if (tok < page_end) {
      uint4 kr[kSub][2][W::kChunks];
      uint32_t vr[kSub][4][W::kVw];
      TilePtr p[kSub];
      int next[kSub];
      // a group past the complete pages, or of a page out of range, takes no part
      auto page_at = [&](int tk) { return tk < page_end ? row[tk >> c.page_shift] : -1; };
      auto base_of = [&](const TilePtr& q) { return q.k ? q.k : c.pages; };
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        p[i] = tile_of(page_at(tok + 16 * i), tok + 16 * i, tok + 16 * i < page_end);
        w.load_k(base_of(p[i]), kr[i]);
        w.load_v(base_of(p[i]) + (size_t)P * D, vr[i]);
        next[i] = page_at(tok + kUnit + 16 * i);
      }
      for (;;) {
        const int then = tok + kUnit;
        const bool more = then < page_end;
        TilePtr pn[kSub];
        int after[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i) after[i] = page_at(then + kUnit + 16 * i);
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
          float s[NT][4];
          w.scores(kr[i], s);
          pn[i] = p[i];
          if (more) {
            pn[i] = tile_of(next[i], then + 16 * i, then + 16 * i < page_end);
            w.load_k(base_of(pn[i]), kr[i]);
          }
          if (p[i].k) {
            uint32_t pb[NT][2];
            w.weights(s, p[i].ks, p[i].ks, true, true, pb);
            w.values(vr[i], p[i].vs, pb);
          }
          if (more) w.load_v(base_of(pn[i]) + (size_t)P * D, vr[i]);
        }
        if (!more) break;
        tok = then;
#pragma unroll
        for (int i = 0; i < kSub; ++i) p[i] = pn[i], next[i] = after[i];
      }
    }
    const int tail_end = min(end, len);
    for (int tk = max(full, t0 * kUnit); tk < tail_end; tk += 16) {
      if (tk % kUnit / (16 * kSub) != warp) continue;
      const uint16_t* kt = c.tails + ((((int64_t)b * c.heads + h) * 2) << c.page_shift) * D + (tk - full) * D;
      w.tail_rows(kt, kt + (int64_t)P * D, min(16, len - tk));
    }

    // the four warps' sums
    __syncthreads();  // the last segment's readers are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = w.l[nt][i];
        x += __shfl_xor_sync(kFull, x, 4);
        x += __shfl_xor_sync(kFull, x, 8);
        x += __shfl_xor_sync(kFull, x, 16);
        const int hd = nt * 8 + 2 * t + i;
        if (g == 0) sml[warp][hd][0] = w.m[nt][i], sml[warp][hd][1] = x;
#pragma unroll
        for (int j = 0; j < W::kSteps; ++j) {
          so[warp][hd][g * (D / 8) + 2 * j] = w.o[nt][j][i];
          so[warp][hd][g * (D / 8) + 2 * j + 1] = w.o[nt][j][2 + i];
        }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    float* part = prm.part + ((((int64_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * prm.passes + blockIdx.y) * 8 * NT) * (D + 2);
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
      const int hd = i / D, ch = i % D;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sml[k][hd][0]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float o = 0.0f, l = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float f = exp2_fast(sml[k][hd][0] - ref);
        o = fmaf(f, so[k][hd][ch], o);
        l = fmaf(f, sml[k][hd][1], l);
      }
      if (whole) {
        const int64_t to = ((int64_t)b * a.q_heads + head0 + hd) * D + ch;
        const float r = o / l;
        if (a.out_f32) static_cast<float*>(a.out)[to] = r;
        else if (BF16) static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16(r);
        else static_cast<__half*>(a.out)[to] = __float2half(r);
      } else {
        part[hd * (D + 2) + ch] = o;
        if (ch == 0) part[hd * (D + 2) + D] = top, part[hd * (D + 2) + D + 1] = l;
      }
    }
    u += t1 - t0;
  }
}

// Merges the partial sums of each (request, query head) that several CTAs
// share, in the order of the CTAs; zeros for a request without tokens.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(D) paged_merge_kernel(const Params prm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedDecodeArgs& a = prm.a;
  const int b = blockIdx.x, hq = blockIdx.y, ch = threadIdx.x;
  const int h = hq / a.group, in_group = hq % a.group, pass = in_group / (8 * NT), hd = in_group % (8 * NT);
  const int p0 = prm.prefix[b], tiles = prm.prefix[b + 1] - p0;
  const int64_t to = ((int64_t)b * a.q_heads + hq) * D + ch;
  float r = 0.0f;
  if (tiles > 0) {
    const long long units = (long long)prm.prefix[a.requests] * prm.c.heads;
    const long long first = (long long)p0 * prm.c.heads + (long long)h * tiles, last = first + tiles - 1;
    // the CTA of unit u is the last c with floor(units c / ctas) <= u
    const int ctas = units < prm.ctas ? (int)units : prm.ctas;
    const int c0 = (int)(((first + 1) * ctas - 1) / units), c1 = (int)(((last + 1) * ctas - 1) / units);
    if (c0 == c1) return;  // finished by that CTA
    const int64_t step = (int64_t)2 * prm.passes * 8 * NT * (D + 2);
    const float* part = prm.part + (int64_t)c0 * step + ((int64_t)pass * 8 * NT + hd) * (D + 2);
    const int64_t second = step / 2;  // the row of a range's end; c0's is its start's
    float top = -INFINITY, o = 0.0f, l = 0.0f;
    constexpr int kBatch = 8;  // partial rows in flight
    for (int k0 = 0; k0 <= c1 - c0; k0 += kBatch) {
      float pm[kBatch], pl[kBatch], po[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool live = k0 + k <= c1 - c0;
        const float* row = part + (live ? k0 + k : 0) * step + (k0 + k == 0 || !live ? second : 0);
        pm[k] = live ? row[D] : -INFINITY;
        pl[k] = live ? row[D + 1] : 0.0f;
        po[k] = live ? row[ch] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float now = fmaxf(top, pm[k]);
        const float ref = now == -INFINITY ? 0.0f : now;
        const float fo = exp2_fast(top - ref), fn = exp2_fast(pm[k] - ref);
        o = o * fo + po[k] * fn;
        l = l * fo + pl[k] * fn;
        top = now;
      }
    }
    r = o / l;
  }
  if (a.out_f32) static_cast<float*>(a.out)[to] = r;
  else if (BF16) static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16(r);
  else static_cast<__half*>(a.out)[to] = __float2half(r);
}

template <int D, int CODE, bool BF16, int NT>
cudaError_t launch(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st) {
  Params p;
  p.c = c;
  p.a = a;
  p.ctas = a.sm_count * ctas_per_sm(NT);
  p.passes = (a.group + 8 * NT - 1) / (8 * NT);
  p.prefix = static_cast<int*>(a.ws);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + prefix_bytes(a.requests));
  static SmemAttr attr;
  const size_t smem = (size_t)(a.requests + 1) * 4;
  cudaError_t e = attr.ensure(paged_decode_kernel<D, CODE, BF16, NT>, (kMaxRequests + 1) * 4);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<D, CODE, BF16, NT><<<dim3(p.ctas, p.passes), kThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.requests, a.q_heads);
  cfg.blockDim = dim3(D);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, BF16, NT>, p);
}

template <int D, int CODE>
cudaError_t by_type(const PagedDev& c, const PagedDecodeArgs& a, cudaStream_t st) {
  if (nt_of(a.group) == 1)
    return c.dtype == KVQ_BF16 ? launch<D, CODE, true, 1>(c, a, st) : launch<D, CODE, false, 1>(c, a, st);
  return c.dtype == KVQ_BF16 ? launch<D, CODE, true, 2>(c, a, st) : launch<D, CODE, false, 2>(c, a, st);
}

}  // namespace pdec
}  // namespace kvq
