// Decode attention over the paged 8-bit cache (kvq_paged_decode_attention).
//
//   e_t = c <q, k_hat_t>,  o = sum_t softmax(e)_t v_hat_t,  x_hat = code * s(page, head)
//
// The step is bound by the bytes of codes it reads: 2 L H D per request,
// against 4 L H_q D operations. Per warp and 16 tokens,
//   S^T = K Q^T   A = K codes (16 tokens x 16 channels), B = Q (8 heads),
//   O^T += s_v V^T P^T   A = V codes (16 channels x 16 tokens), B = P^T,
// both m16n8k16 in fp16 with fp32 sums. Every code (int8 or e4m3) is an exact
// fp16 number, so only P is rounded (2^-11 of each weight). Tokens and
// channels may be summed in any order, so a lane reads 16 contiguous bytes
// and calls them the fragment's slots.
//
// The tiles (64 or 128 tokens of one request and kv-head, 16 KB of codes) of
// all requests form one line that is cut into equal ranges, one per CTA: the
// kernel makes the line from the device lengths itself, so the grid needs no
// host knowledge and ragged batches stay even. A (request, head) has kExtra
// more places on the line than tiles, for what its begin, tail and merge cost
// (4000 to 8000 clocks against 1300 to 1600 a tile): without them a CTA that
// got fourteen one-tile requests took three times as long as the others. A producer warp walks the
// range and keeps a ring of tiles in flight by TMA, on into the next request
// or head while the four consumer warps still merge the last one; these take
// 16 or 32 tokens of a tile each and keep their own running maximum and sums.
// A (request, head) that one CTA covers is finished there; the others leave
// partial sums, which a second kernel merges in the order of the CTAs.
//
// 16 requests of up to 131072 tokens, 8 kv-heads, 64 query heads (1.84 GB):
// 275 us, 0.98 of the copy rate. 64 ragged requests up to 8192 tokens (0.51
// GB): 91 us, 0.82 of it; what is left are the ends of requests (tail, merge,
// the next queries). 24 requests up to 2500 tokens, 32 heads of 64 channels
// (0.115 GB): 31 us, 0.54. One request of 777 tokens: 8.7 us, latency of two launches.
// Loads straight into the fragments' registers, without a ring, took 292, 101,
// 39 and 8.5 us.
#pragma once

#include "paged_internal.h"
#include "tensor_map.cuh"

namespace kvq {
namespace pdec {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;  // of the consumers; the producer is a fifth warp
constexpr unsigned kFull = 0xffffffffu;

// Groups of 16 tokens that a warp takes of a tile, and the tile's tokens.
__host__ __device__ constexpr int sub_of(int dim) { return 128 / dim; }
__host__ __device__ constexpr int unit_of(int dim) { return kWarps * 16 * sub_of(dim); }

// Places on the line before a (request, head)'s tiles.
constexpr int kExtra = 5;

// Heads of one pass over the codes: 8 NT (NT column tiles of the products).
// Two tiles a pass cost registers (two CTAs an SM and, with 128 channels, some
// spills, instead of three CTAs), but past 8 heads they save reading and
// converting the codes once more.
// us with one / with two, 64 ragged requests up to 8192 tokens, 8 kv-heads:
//   heads a kv-head     8         9        12        16        24        40
//   128 channels      95/129   173/131   177/137   182/145   267/261   435/388
//    64 channels      54/65     95/65     97/66     99/68    144/124   231/184
__host__ __device__ constexpr int nt_of(int group) { return group <= 8 ? 1 : 2; }
// CTAs per SM that the registers and the rings (kTileBytes each stage) allow.
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }
__host__ __device__ constexpr int stages_of(int nt) { return nt == 1 ? 3 : 4; }
constexpr int kTileBytes = 16384;  // keys, then values, of kWarps * 16 * sub_of(D) tokens

// Workspace: int prefix[requests + 1] of places (of one kv-head), then partial
// rows [ctas][2][passes][8 NT][D + 2]: o[D], m, l.
__host__ __device__ inline size_t prefix_bytes(int requests) { return ((size_t)(requests + 1) * 4 + 255) / 256 * 256; }

struct Params {
  CUtensorMap map;  // codes as [page, head, K or V][token][channel]
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

__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Exponent k with max |x| * 2^k in [2^14, 2^15), from the bits of max |x| in
// bf16: bf16 queries go to the fp16 products with the codes scaled by 2^k. That
// is exact but for elements below 2^-29 of the query's largest, whose rounding
// (2^-40 of it) is far below the fp32 sums' own. 126 keeps 2^k and 2^-k normal,
// and every bf16 number below 2^-111 times 2^126 is an exact fp16 one.
__device__ __forceinline__ int bf16_shift(uint32_t top_bits) {
  const int k = 14 - ((int)(top_bits >> 7) - 127);
  return k > 126 ? 126 : k;
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
  static constexpr float kLift = 7.0f;
  uint32_t qf[NT][kSteps][2];
  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2], qs[NT][2];  // heads 2 t4, 2 t4 + 1 of the column tile

  // Queries of `heads` heads, as they lie; begin() makes them ready.
  __device__ __forceinline__ void load_q(const uint16_t* q, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool live = nt * 8 + g < heads;
      const uint16_t* row = q + (int64_t)(live ? nt * 8 + g : 0) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + ((s >> 2) * 4 + t) * 16 + (s & 3) * 4);
        qf[nt][s][0] = live ? w.x : 0u;
        qf[nt][s][1] = live ? w.y : 0u;
      }
    }
  }

  // The loaded queries' factors 2^-k, and the empty running state.
  __device__ __forceinline__ void begin() {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f = 1.0f;
      if (BF16) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) top = abs_max2(abs_max2(top, qf[nt][s][0]), qf[nt][s][1]);
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
        f = exp2i(-k);
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

  // Scores s of 16 tokens (c0, c1: token g; c2, c3: token g + 8) to their
  // weights; q f0: the heads' factors. va, vb: whether the two tokens count.
  __device__ __forceinline__ void weights(float (&s)[NT][4], const float (&q)[NT][2], float f0, bool va, bool vb) {
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[nt][i] = va ? s[nt][i] * (q[nt][i] * f0) : -INFINITY;
        s[nt][2 + i] = vb ? s[nt][2 + i] * (q[nt][i] * f0) : -INFINITY;
        up |= fmaxf(s[nt][i], s[nt][2 + i]) - m[nt][i] > kLift + 8.0f;
      }
    }
    // The reference of the exponentials lies kLift below a score and moves only
    // when one passes that by 8: most tiles skip the reduction, weights stay
    // below 2^15, and those of 2^-21 of it and more above fp16's subnormal numbers
    // (below, many small weights beside a large one would be off to one side).
    if (__any_sync(kFull, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(s[nt][i], s[nt][2 + i]);
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
          const bool mine = x - m[nt][i] > kLift + 8.0f;  // each head by its own scores
          const float now = mine ? x - kLift : m[nt][i];
          const float f = mine ? exp2_fast(m[nt][i] - now) : 1.0f;
          m[nt][i] = now;
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
    }
  }
  // ... as the B operand of P^T in fp16.
  __device__ __forceinline__ void half_weights(const float (&s)[NT][4], uint32_t (&p)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
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

  // 16 tokens' codes from the swizzled tile (16-byte chunk index XOR address
  // bits 7 to 9); k, v: the group's first row, at a multiple of 1024 bytes.
  __device__ __forceinline__ void load_k(const uint8_t* k, uint4 (&kr)[2][kChunks]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        kr[r][c] = *reinterpret_cast<const uint4*>(k + swz<D>((g + 8 * r) * D + (c * 4 + t) * 16));
  }
  __device__ __forceinline__ void load_v(const uint8_t* v, uint32_t (&vr)[4][kVw]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* src = v + swz<D>((2 * t + (r & 1) + (r >> 1) * 8) * D + g * (D / 8));
      if (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        vr[r][0] = w.x, vr[r][1] = w.y, vr[r][2 % kVw] = w.z, vr[r][3 % kVw] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
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

  // 16 rows of the tail, `live` of them cached: the same products on the input
  // type's rows (qf: the queries as they lie). In bf16 a weight goes as the sum
  // of two bf16 numbers, 2^-16 of it off. k, v: the tail's rows at the first.
  __device__ __forceinline__ void tail_rows(const uint16_t* k, const uint16_t* v, int live, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float s[NT][4], q[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      q[nt][0] = q[nt][1] = scale_log2;
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nt][r] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      uint4 x[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4* src = reinterpret_cast<const uint4*>(k + (g + 8 * r) * D + (c * 4 + t) * 16);
        x[r][0] = g + 8 * r < live ? src[0] : zero;
        x[r][1] = g + 8 * r < live ? src[1] : zero;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 a = x[0][i >> 1], b = x[1][i >> 1];
        const uint32_t a0 = i & 1 ? a.z : a.x, a2 = i & 1 ? a.w : a.y, a1 = i & 1 ? b.z : b.x, a3 = i & 1 ? b.w : b.y;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = qf[nt][c * 4 + i][0], b1 = qf[nt][c * 4 + i][1];
          if (BF16) mma16816_bf16(s[nt], a0, a1, a2, a3, b0, b1);
          else mma16816(s[nt], a0, a1, a2, a3, b0, b1);
        }
      }
    }
    weights(s, q, 1.0f, g < live, g + 8 < live);
    uint32_t p[NT][2], pl[NT][2];
    if (BF16) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t hi = pack_bf2(s[nt][2 * r], s[nt][2 * r + 1]);
          p[nt][r] = movmatrix(hi);
          pl[nt][r] = movmatrix(pack_bf2(s[nt][2 * r] - __uint_as_float(hi << 16),
                                         s[nt][2 * r + 1] - __uint_as_float(hi & 0xffff0000u)));
        }
    } else {
      half_weights(s, p);
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 2 * t + (r & 1) + (r >> 1) * 8;
        x[r] = row < live ? reinterpret_cast<const uint4*>(v + row * D + g * (D / 8))[c] : zero;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // channels 2 j and 2 j + 1 of the lane's D / 8
        const int j = 4 * c + i;
        const uint32_t w0 = i == 0 ? x[0].x : i == 1 ? x[0].y : i == 2 ? x[0].z : x[0].w;
        const uint32_t w1 = i == 0 ? x[1].x : i == 1 ? x[1].y : i == 2 ? x[1].z : x[1].w;
        const uint32_t w2 = i == 0 ? x[2].x : i == 1 ? x[2].y : i == 2 ? x[2].z : x[2].w;
        const uint32_t w3 = i == 0 ? x[3].x : i == 1 ? x[3].y : i == 2 ? x[3].z : x[3].w;
        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (BF16) {
            mma16816_bf16(o[nt][j], a0, a1, a2, a3, p[nt][0], p[nt][1]);
            mma16816_bf16(o[nt][j], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          } else {
            mma16816(o[nt][j], a0, a1, a2, a3, p[nt][0], p[nt][1]);
          }
        }
      }
    }
  }
};

// A part of one (request, kv-head): its tiles [t0, t1), and the place on the
// line after the (request, head).
struct Part {
  int b, h, t0, t1, tiles;
  long long end;
  // the range's share of it
  __device__ __forceinline__ void cut(long long v0, long long v1) {
    const long long first = end - tiles;  // the place of tile 0
    t0 = v0 > first ? (int)(v0 - first) : 0;
    t1 = v1 < end ? (int)(v1 - first) : tiles;
  }
};

// n / d, in 32 bits where both fit (a 64-bit division takes half a microsecond).
__device__ __forceinline__ long long quotient(unsigned long long n, unsigned long long d) {
  return (n | d) >> 32 ? (long long)(n / d) : (long long)((uint32_t)n / (uint32_t)d);
}

// The first part of the range [v0, v1) of places; it may hold no tile
// (t1 <= t0: only places before tile 0, or beyond).
__device__ __forceinline__ Part first_part(const int* prefix, int requests, int heads, long long v0, long long v1) {
  Part x;
  x.b = 0;
  for (int n = requests; n > 1;) {  // last b with prefix[b] * heads <= v0 (equal ones: empty requests before it)
    const int half = n >> 1;
    if ((long long)prefix[x.b + half] * heads <= v0) x.b += half, n -= half;
    else n = half;
  }
  const int places = prefix[x.b + 1] - prefix[x.b];
  const long long at = v0 - (long long)prefix[x.b] * heads;
  x.h = (int)quotient(at, places);
  x.tiles = places - kExtra;
  x.end = (long long)prefix[x.b] * heads + (long long)(x.h + 1) * places;
  x.cut(v0, v1);
  return x;
}

// The next part, or false where the range ends before it has a tile.
__device__ __forceinline__ bool next_part(Part& x, const int* prefix, int requests, int heads, long long v0,
                                          long long v1) {
  do {
    if (x.end >= v1) return false;
    if (++x.h == heads) {
      x.h = 0;
      do ++x.b;
      while (prefix[x.b + 1] == prefix[x.b]);  // ends: there are places before v1
      x.tiles = prefix[x.b + 1] - prefix[x.b] - kExtra;
    }
    x.end += x.tiles + kExtra;
    x.cut(v0, v1);
  } while (x.t1 <= x.t0);
  return true;
}

template <int NT>
struct Ring {
  uint64_t full[stages_of(NT)], empty[stages_of(NT)];
  uint32_t live[stages_of(NT)];     // bit i: box i of the tile is there
  float2 scale[stages_of(NT)][8];   // its scales of keys and values
};

// Whole warp: false where the wait gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const bool done = mbar_wait_bounded(bar, parity);
  if (!done) raise_status(status, kStatusTimeout);
  return __all_sync(kFull, done);
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// The producer: per tile, boxes of min(P, 64) tokens of complete pages.
template <int D, int NT>
__device__ __forceinline__ void produce(const Params& prm, Ring<NT>& ring, unsigned char* tiles, const int* prefix,
                                        Part x, const long long v0, const long long v1) {
  constexpr int kStages = stages_of(NT), kUnit = unit_of(D);
  const PagedDev& c = prm.c;
  const int lane = threadIdx.x & 31, P = 1 << c.page_shift;
  const int box = P < 64 ? P : 64, boxes = kUnit / box;
  int i = 0;
  bool ok = true;
  do {
    const int full = prm.a.lens[x.b] & ~(P - 1);  // tokens in complete pages
    const int32_t* row = prm.a.table + (int64_t)x.b * c.max_pages;
    auto page_at = [&](int tile) {
      const int tk = tile * kUnit + lane * box;
      return lane < boxes && tk < full ? row[tk >> c.page_shift] : -1;
    };
    int page = page_at(x.t0);
    for (int tile = x.t0; tile < x.t1; ++tile, ++i) {
      const int st = i % kStages, tk = tile * kUnit + lane * box;
      const int next = tile + 1 < x.t1 ? page_at(tile + 1) : -1;
      const bool wanted = lane < boxes && tk < full, there = wanted && page >= 0 && page < c.num_pages;
      if (wanted && !there) raise_status(c.status, kStatusBadIndex);
      const uint32_t live = __ballot_sync(kFull, there);
      ok = wait(&ring.empty[st], ((i / kStages) & 1) ^ 1, c.status);
      if (!ok) break;
      if (lane == 0) {
        ring.live[st] = live;
        expect_tx(&ring.full[st], (uint32_t)__popc(live) * box * D * 2);
      }
      __syncwarp();
      if (there) {
        const int64_t ph = ((int64_t)page * c.heads + x.h) * 2;
        unsigned char* dst = tiles + st * kTileBytes + lane * box * D;
        tma_rows(dst, &prm.map, tk & (P - 1), (int)ph, &ring.full[st]);
        tma_rows(dst + kTileBytes / 2, &prm.map, tk & (P - 1), (int)ph + 1, &ring.full[st]);
        ring.scale[st][lane] = *reinterpret_cast<const float2*>(c.scales + ph);
      }
      __syncwarp();
      if (lane == 0) arrive(&ring.full[st]);
      page = next;
    }
  } while (ok && next_part(x, prefix, prm.a.requests, c.heads, v0, v1));
  // nothing is in flight into this CTA's shared memory when it ends
  for (int k = max(0, i - kStages); k < i; ++k) wait(&ring.full[k % kStages], (k / kStages) & 1, c.status);
}

template <int D, int CODE, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads + 32, ctas_per_sm(NT))
    paged_decode_kernel(const __grid_constant__ Params prm) {
  using W = Warp<D, CODE, BF16, NT>;
  constexpr int kSub = sub_of(D), kUnit = unit_of(D), kStages = stages_of(NT);
  const PagedDev& c = prm.c;
  const PagedDecodeArgs& a = prm.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  int* prefix = reinterpret_cast<int*>(tiles + kStages * kTileBytes);  // [requests + 1]
  __shared__ float so[kWarps][8 * NT][D + 1];
  __shared__ float sml[kWarps][8 * NT][2];
  __shared__ int wsum[kWarps];
  __shared__ Ring<NT> ring;
  __shared__ int failed;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int R = a.requests, P = 1 << c.page_shift;
  const int most = c.max_pages << c.page_shift;

  if (threadIdx.x == kThreads) {
    prefetch_map(&prm.map);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], kWarps);
    }
    mbar_fence_init();
    failed = 0;
  }
  // prefix sums of the requests' places
  auto places_of = [&](int n) { return n > 0 ? (n + kUnit - 1) / kUnit + kExtra : 0; };
  const int per = (R + kThreads - 1) / kThreads;
  int sum = 0, incl = 0;
  if (warp < kWarps) {
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      int n = b < R ? a.lens[b] : 0;
      if (n < 0 || n > most) bad = true, n = 0;
      sum += places_of(n);
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) raise_status(c.status, kStatusBadIndex);
    incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
  }
  __syncthreads();
  if (warp < kWarps) {
    int at = incl - sum;
    for (int i = 0; i < warp; ++i) at += wsum[i];
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b < R) {
        prefix[b] = at;
        int n = a.lens[b];
        if (n < 0 || n > most) n = 0;
        at += places_of(n);
        if (b == R - 1) prefix[R] = at;
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b <= R; b += kThreads + 32) prm.prefix[b] = prefix[b];

  const long long places = (long long)prefix[R] * c.heads;
  const int ctas = places < prm.ctas ? (int)places : prm.ctas;  // each of these has a place at least
  if ((int)blockIdx.x >= ctas) return;
  const long long v0 = quotient(places * blockIdx.x, ctas), v1 = quotient(places * (blockIdx.x + 1), ctas);
  Part cur = first_part(prefix, R, c.heads, v0, v1);
  if (cur.t1 <= cur.t0 && !next_part(cur, prefix, R, c.heads, v0, v1)) return;  // no tile: all of the CTA
  if (warp == kWarps) {
    produce<D, NT>(prm, ring, tiles, prefix, cur, v0, v1);
    return;
  }

  const int box_shift = c.page_shift < 6 ? c.page_shift : 6;
  const int pass0 = blockIdx.y * 8 * NT, heads = min(8 * NT, a.group - pass0);
  W w;
  auto load_q = [&](const Part& x) {
    w.load_q(a.q + x.b * a.q_stride + (int64_t)(x.h * a.group + pass0) * D, heads);
  };
  load_q(cur);
  bool ok = true;
  int len = a.lens[cur.b];
  for (int i = 0;;) {
    const int full = len & ~(P - 1);  // tokens in complete pages
    const uint16_t* tail = c.tails + ((((int64_t)cur.b * c.heads + cur.h) * 2) << c.page_shift) * D;
    const int tail0 = max(full, cur.t0 * kUnit), tail_end = min(cur.t1 * kUnit, len);
    for (int tk = tail0 + (threadIdx.x >> 1); tk < tail_end; tk += kThreads / 2) {  // half a row a thread, keys and values
      const uint16_t* at = tail + (tk - full) * D + (threadIdx.x & 1) * (D / 2);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at + (int64_t)P * D));
    }
    w.begin();
    for (int tile = cur.t0; tile < cur.t1; ++tile, ++i) {
      const int st = i % kStages;
      ok = ok && wait(&ring.full[st], (i / kStages) & 1, c.status);
      if (!ok) break;
      const unsigned char* k = tiles + st * kTileBytes + warp * 16 * kSub * D;
      uint4 kr[kSub][2][W::kChunks];
      uint32_t vr[kSub][4][W::kVw];
      float2 sc[kSub];
      const uint32_t live = ring.live[st];
      bool there[kSub];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const int box = (warp * 16 * kSub + 16 * j) >> box_shift;
        there[j] = (live >> box) & 1;
        sc[j] = ring.scale[st][box];
        w.load_k(k + 16 * j * D, kr[j]);
        w.load_v(k + kTileBytes / 2 + 16 * j * D, vr[j]);
      }
      __syncwarp();
      if (lane == 0) arrive(&ring.empty[st]);
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        if (!there[j]) continue;
        float s[NT][4];
        uint32_t pb[NT][2];
        w.scores(kr[j], s);
        // the page's and the softmax's scale first: 2^-k alone may be far off the scores' size
        w.weights(s, w.qs, sc[j].x * a.scale_log2, true, true);
        w.half_weights(s, pb);
        w.values(vr[j], sc[j].y, pb);
      }
    }
    if (BF16 && tail0 < tail_end) load_q(cur);  // the products with the codes had them scaled
    for (int tk = tail0; tk < tail_end; tk += 16)
      if (tk % kUnit / (16 * kSub) == warp)
        w.tail_rows(tail + (tk - full) * D, tail + (tk - full + P) * D, min(16, len - tk), a.scale_log2);

    // the four warps' sums; the next part's queries are on their way meanwhile
    const Part done = cur;
    if (!ok) failed = 1;
    const bool go_on = next_part(cur, prefix, R, c.heads, v0, v1);
    if (go_on) {
      len = a.lens[cur.b];
      load_q(cur);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        float x = w.l[nt][i2];
        x += __shfl_xor_sync(kFull, x, 4);
        x += __shfl_xor_sync(kFull, x, 8);
        x += __shfl_xor_sync(kFull, x, 16);
        const int hd = nt * 8 + 2 * t + i2;
        if (g == 0) sml[warp][hd][0] = w.m[nt][i2], sml[warp][hd][1] = x;
#pragma unroll
        for (int j = 0; j < W::kSteps; ++j) {
          so[warp][hd][g * (D / 8) + 2 * j] = w.o[nt][j][i2];
          so[warp][hd][g * (D / 8) + 2 * j + 1] = w.o[nt][j][2 + i2];
        }
      }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (failed) return;  // all four warps: a wait gave up
    const bool whole = done.t0 == 0 && done.t1 == done.tiles;
    const int head0 = done.h * a.group + pass0;
    float* part =
        prm.part + ((((int64_t)blockIdx.x * 2 + (done.t0 > 0 ? 0 : 1)) * prm.passes + blockIdx.y) * 8 * NT) * (D + 2);
    for (int k = threadIdx.x; k < heads * D; k += kThreads) {
      const int hd = k / D, ch = k % D;
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) top = fmaxf(top, sml[v][hd][0]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float o = 0.0f, l = 0.0f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float f = exp2_fast(sml[v][hd][0] - ref);
        o = fmaf(f, so[v][hd][ch], o);
        l = fmaf(f, sml[v][hd][1], l);
      }
      if (whole) {
        const int64_t to = ((int64_t)done.b * a.q_heads + head0 + hd) * D + ch;
        const float r = o / l;
        if (a.out_f32) static_cast<float*>(a.out)[to] = r;
        else if (BF16) static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16(r);
        else static_cast<__half*>(a.out)[to] = __float2half(r);
      } else {
        part[hd * (D + 2) + ch] = o;
        if (ch == 0) part[hd * (D + 2) + D] = top, part[hd * (D + 2) + D + 1] = l;
      }
    }
    if (!go_on) return;
    asm volatile("bar.sync 1, 128;" ::: "memory");  // so and sml may be written again
  }
}

// Merges the partial sums of each (request, query head) that several CTAs
// share, in the order of the CTAs; zeros for a request without tokens.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(D) paged_merge_kernel(const __grid_constant__ Params prm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedDecodeArgs& a = prm.a;
  const int b = blockIdx.x, hq = blockIdx.y, ch = threadIdx.x;
  const int h = hq / a.group, in_group = hq % a.group, pass = in_group / (8 * NT), hd = in_group % (8 * NT);
  const int p0 = prm.prefix[b], own = prm.prefix[b + 1] - p0;
  const int64_t to = ((int64_t)b * a.q_heads + hq) * D + ch;
  float r = 0.0f;
  if (own > 0) {
    const long long places = (long long)prm.prefix[a.requests] * prm.c.heads;
    const long long end = (long long)p0 * prm.c.heads + (long long)(h + 1) * own, first = end - (own - kExtra);
    // the CTA of a place v is the last c with floor(places c / ctas) <= v
    const int ctas = places < prm.ctas ? (int)places : prm.ctas;
    auto cta_of = [&](long long v) { return (int)quotient((v + 1) * ctas - 1, places); };
    const int c0 = cta_of(first), c1 = cta_of(end - 1);
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
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const int page = 1 << c.page_shift;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)c.num_pages * c.heads * 2};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * page};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)(page < 64 ? page : 64), 1u};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  if (fn(&p.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.pages, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
         D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static SmemAttr attr;
  const size_t ring = 1024 + stages_of(NT) * kTileBytes;
  cudaError_t e = attr.ensure(paged_decode_kernel<D, CODE, BF16, NT>, ring + (kMaxRequests + 1) * 4);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<D, CODE, BF16, NT>
      <<<dim3(p.ctas, p.passes), kThreads + 32, ring + (size_t)(a.requests + 1) * 4, st>>>(p);
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
