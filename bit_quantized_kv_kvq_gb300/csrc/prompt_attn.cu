// Causal attention over packed prompts on their own keys and values
// (kvq_prompt_attention).
//
//   o_i = sum_{t <= i} softmax(c <q_i, k_t>)_t v_t
//
// One pass over the keys per block of query rows, with the running maximum m
// and sum l of the exponentials. The 4 D L^2 / 2 operations per head bound it,
// so both products run on the 5th-generation tensor cores: S = Q K^T from
// shared memory into tensor memory, and O += P V with P in tensor memory (where
// S was) and V as TMA loaded it. P is rounded to the input type (half an eps
// of each weight, zero mean: that of an output element); m, l, S and O are fp32.
//
// A CTA holds two units of 128 query rows x one head: two heads of a group on
// the same rows (they share every key tile and its end), or, where the group
// is odd, two row blocks of one head. While the tensor cores work for one
// unit, the other's 128 threads (one row each) turn its scores into weights.
// Warps 0-3 and 4-7: softmax of the units; 8: TMA; 9: tensor core issue;
// 10, 11: the values of the tiles that the diagonal cuts (see check_values).
#include "paged_internal.h"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;  // query rows of a unit, keys of a tile
constexpr int kNever = 0x7fffffff;

template <int D>
struct Cfg {
  static constexpr int kTile = kRows * D * 2;        // bytes of a Q, K or V tile
  static constexpr int kStages = D == 128 ? 4 : 8;   // K and V tiles in flight
  static constexpr int kSmem = 1024 + (2 + kStages) * kTile;
};

struct Shared {
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2], drain;
  uint64_t v_full[2], v_checked[2];  // value tiles that the diagonal cuts (the last one or two): loaded, checked
  uint64_t kv_full[8], kv_empty[8];
  uint32_t tmem;
  int any_nonfinite;
  int first[3][128];  // first token of the cut tiles whose value is NaN, +inf, -inf, per channel
};

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

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  if (mbar_wait_bounded(bar, parity)) return true;
  raise_status(status, kStatusTimeout);
  return false;
}

// 0 * inf would carry a later token's infinity or NaN to an earlier row. In
// the tiles that the diagonal cuts, the tensor cores get 0 in their place; the
// rows from that token on get them at the end (Shared::first).
template <int D, bool BF16>
__device__ __forceinline__ void check_values(unsigned char* tile, int k0, Shared* sh) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u, kStep = BF16 ? 0x0080u : 0x0400u;
  const int tid = threadIdx.x - 320;
  for (int i = tid; i < kRows * D / 8; i += 64) {
    uint4* at = reinterpret_cast<uint4*>(tile) + i;
    uint4 x = *at;
    // an exponent of all ones carries into the sign bit's place
    const uint32_t hit = ((x.x & (kInf * 0x10001u)) + kStep * 0x10001u) | ((x.y & (kInf * 0x10001u)) + kStep * 0x10001u) |
                         ((x.z & (kInf * 0x10001u)) + kStep * 0x10001u) | ((x.w & (kInf * 0x10001u)) + kStep * 0x10001u);
    if ((hit & 0x80008000u) == 0) continue;
    // 16-byte chunk i of the tile: 64-channel half, token row, swizzled place
    const int row = (i >> 3) & 127, ch = (i >> 10) * 64 + (((i & 7) ^ (row & 7)) << 3);
    __align__(16) uint16_t e[8];
    *reinterpret_cast<uint4*>(e) = x;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((e[j] & kInf) == kInf) {
        const int kind = (e[j] & 0x7fffu) != kInf ? 0 : (e[j] >> 15) ? 2 : 1;
        atomicMin(&sh->first[kind][ch + j], k0 + row);
        sh->any_nonfinite = 1;
        e[j] = 0;
      }
    *at = *reinterpret_cast<uint4*>(e);
  }
}

// One unit's rows: scores to weights tile by tile, then the output.
template <int D, bool BF16>
__device__ __forceinline__ void softmax_unit(const PromptArgs& a, Shared* sh, unsigned char* stage, int unit, int row0,
                                             int tiles, int n, int c0, int hq, int check) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, r = warp * 32 + lane;
  const uint32_t lanes = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t tS = lanes + unit * 128, tP = tS, tO = lanes + 256 + unit * D;
  const float sc = a.scale_log2;
  float m = -INFINITY, l = 0.0f;
  bool ok = true;
  for (int j = 0; j < tiles && ok; ++j) {
    ok = __all_sync(0xffffffffu, wait(&sh->s_full[unit], j & 1, a.status));
    if (!ok) break;
    t5::fence_after();
    uint32_t s[128];
#pragma unroll
    for (int c = 0; c < 4; ++c) t5::ld32(tS + 32 * c, s + 32 * c);
#pragma unroll
    for (int c = 0; c < 4; ++c) t5::wait_ld32(s + 32 * c);
    if (j == tiles - 1) {  // the tile the diagonal cuts: keys of this block after the row
#pragma unroll
      for (int c = 0; c < 128; ++c)
        if (c > r) s[c] = 0xff800000u;
    }
    float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
    for (int c = 0; c < 128; c += 8) {
      t0 = fmaxf(fmaxf(t0, __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
      t1 = fmaxf(fmaxf(t1, __uint_as_float(s[c + 2])), __uint_as_float(s[c + 3]));
      t2 = fmaxf(fmaxf(t2, __uint_as_float(s[c + 4])), __uint_as_float(s[c + 5]));
      t3 = fmaxf(fmaxf(t3, __uint_as_float(s[c + 6])), __uint_as_float(s[c + 7]));
    }
    const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * sc;
    // The reference m moves only when a score passes it by 8 (weights stay
    // below 2^8), so that few tiles scale O. Each row goes by its own scores:
    // a row's bits do not depend on its neighbours. s_full came after the last PV.
    const bool up = top > m + 8.0f;
    if (__any_sync(0xffffffffu, up)) {
      const float f = up ? exp2_fast(m - top) : 1.0f;
      m = up ? top : m;
      l *= f;
      if (j > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          t5::ld32(tO + c, o);
          t5::wait_ld32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          t5::st32(tO + c, o);
        }
      }
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    const uint64_t sc2 = f2_pack(sc, sc), ref2 = f2_pack(-ref, -ref);
    uint64_t sum0 = f2_pack(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t p[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int c = half * 64 + 2 * i;
        float x, y;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, ref2), x, y);
        x = exp2_fast(x);
        y = exp2_fast(y);
        if (i & 1) sum1 = f2_add(sum1, f2_pack(x, y));
        else sum0 = f2_add(sum0, f2_pack(x, y));
        p[i] = pack2<BF16>(x, y);
      }
      t5::st32(tP + half * 32, p);
    }
    float x, y;
    f2_unpack(f2_add(sum0, sum1), x, y);
    l += x + y;
    t5::wait_st();
    t5::fence_before();
    arrive(&sh->p_full[unit]);
  }
  if (tiles == 0) return;  // all of the unit's threads
  if (ok) ok = __all_sync(0xffffffffu, wait(&sh->o_done[unit], 0, a.status) && wait(&sh->v_checked[check], 0, a.status));
  if (ok) {
    t5::fence_after();
    const float inv = 1.0f / l;
    const int row = row0 + r;
    const bool fix = sh->any_nonfinite != 0;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      t5::ld32(tO + c, o);
      t5::wait_ld32(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float x = __uint_as_float(o[i]) * inv;
        if (fix) {
          if (row >= sh->first[1][c + i]) x += INFINITY;
          if (row >= sh->first[2][c + i]) x -= INFINITY;
          if (row >= sh->first[0][c + i]) x = NAN;
        }
        o[i] = __float_as_uint(x);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack2<BF16>(__uint_as_float(o[8 * q + 2 * i]), __uint_as_float(o[8 * q + 2 * i + 1]));
        const int chunk = c / 8 + q;
        *reinterpret_cast<uint4*>(stage + r * (D * 2) + ((chunk ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  // through the unit's query tile (no longer read) to whole rows in order
  asm volatile("bar.sync %0, 128;" ::"r"(1 + unit) : "memory");
  if (!ok) return;
  for (int i = r; i < kRows * (D / 8); i += 128) {
    const int row = i / (D / 8), chunk = i % (D / 8);
    if (row0 + row < n)
      *reinterpret_cast<uint4*>(a.out + ((int64_t)(c0 + row0 + row) * a.q_heads + hq) * D + chunk * 8) =
          *reinterpret_cast<const uint4*>(stage + row * (D * 2) + ((chunk ^ (row & 7)) << 4));
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const PromptArgs a, const int pair) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sh;
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = pair ? kRows : 2 * kRows;  // query rows of the CTA
  const int lots = pair ? a.q_heads / 2 : a.q_heads;                          // heads or pairs of them
  const int lot = blockIdx.x % lots, w = (gridDim.x - 1 - blockIdx.x) / lots;  // the longest blocks first
  const int group = a.q_heads / a.kv_heads;
  const int* cu = a.cu;
  // row blocks of sequence s start at floor(cu[s] / span) + s: room for all of them
  const int s = warp_last_le(a.seqs, w, [&](int i) { return (int)((uint32_t)cu[i] / (uint32_t)span) + i; });
  const int c0 = cu[s], n = cu[s + 1] - c0;
  if (n <= 0) return;
  if (c0 < 0 || n > a.tokens - c0) {
    if (threadIdx.x == 0 && lot == 0) raise_status(a.status, kStatusBadIndex);
    return;
  }
  const int block = w - (c0 / span + s), q0 = block * span;
  if (block < 0 || q0 >= n) return;
  const int hq0 = pair ? 2 * lot : lot, h = hq0 / group;
  const int row1 = pair ? q0 : q0 + kRows;  // of unit 1
  const int tiles0 = q0 / kRows + 1, tiles1 = row1 < n ? row1 / kRows + 1 : 0;
  const int tiles = max(tiles0, tiles1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_checked[i], 64);
    }
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    mbar_fence_init();
    sh.any_nonfinite = 0;
  }
  for (int i = threadIdx.x; i < 3 * D; i += kThreads) sh.first[i / D][i % D] = kNever;
  if (warp == 9) t5::alloc(&sh.tmem, 512);
  t5::fence_before();
  __syncthreads();
  t5::fence_after();

  unsigned char* ring = smem + 2 * C::kTile;
  // Load i (2 j: keys of tile j, 2 j + 1: its values) and its barrier. The cut
  // tiles' values have one each, used once, so that the checking warps need
  // not follow the ring's phases.
  auto cut = [&](int i) { return (i & 1) && (i >> 1) >= tiles0 - 1; };
  auto full_of = [&](int i) { return cut(i) ? &sh.v_full[(i >> 1) - (tiles0 - 1)] : &sh.kv_full[i % C::kStages]; };
  auto phase_of = [&](int i) { return cut(i) ? 0u : (uint32_t)(i / C::kStages) & 1u; };
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int unit = warp >> 2;
    softmax_unit<D, BF16>(a, &sh, smem + unit * C::kTile, unit, unit ? row1 : q0, unit ? tiles1 : tiles0, n, c0,
                          unit && pair ? hq0 + 1 : hq0, unit && !pair ? 1 : 0);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 && lane == 0) {
      for (int u = 0; u < (tiles1 > 0 ? 2 : 1); ++u) {
        mbar_arrive_expect_tx(&sh.q_full[u], C::kTile);
        for (int b = 0; b < D / 64; ++b)
          tma_tile(smem_u32(smem + u * C::kTile + b * (kRows * 128)), &mq, b * 64, u && pair ? hq0 + 1 : hq0,
                   c0 + (u ? row1 : q0), &sh.q_full[u]);
      }
      int i = 0;
      for (; i < 2 * tiles; ++i) {
        const int st = i % C::kStages;
        if (i >= C::kStages && !wait(&sh.kv_empty[st], (i / C::kStages - 1) & 1, a.status)) break;
        uint64_t* bar = full_of(i);
        mbar_arrive_expect_tx(bar, C::kTile);
        for (int b = 0; b < D / 64; ++b)
          tma_tile(smem_u32(ring + st * C::kTile + b * (kRows * 128)), i & 1 ? &mv : &mk, b * 64, h,
                   c0 + (i >> 1) * kRows, bar);
      }
      // nothing is in flight into this CTA's shared memory when it ends
      for (int k = max(0, i - C::kStages); k < i; ++k) wait(full_of(k), phase_of(k), a.status);
      for (int u = 0; u < (tiles1 > 0 ? 2 : 1); ++u) wait(&sh.q_full[u], 0, a.status);
    } else if (warp == 9) {
      // The whole warp follows the schedule and one elected lane issues: with
      // uniform control flow the operands stay in uniform registers, and an
      // m128n128k16 issues every 64 clocks, the tensor cores' rate (in a
      // branch of one lane it took 90).
      constexpr uint32_t kQK = t5::instr_desc(128, 128, BF16, false), kPV = t5::instr_desc(128, D, BF16, true);
      const uint32_t tmem = sh.tmem;
      const uint64_t dq = t5::smem_desc(smem_u32(smem), 16), dk = t5::smem_desc(smem_u32(ring), 16);
      const uint64_t dv = t5::smem_desc(smem_u32(ring), kRows * 128);
      auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity, a.status)); };
      auto qk = [&](int u, int i) {
        const uint64_t q = dq + (uint32_t)(u * C::kTile >> 4), k = dk + (uint32_t)((i % C::kStages) * C::kTile >> 4);
        if (t5::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4;
            t5::mma_ss(tmem + u * 128, q + off, k + off, kQK, kk > 0);
          }
          t5::commit(&sh.s_full[u]);
        }
        __syncwarp();
      };
      auto pv = [&](int u, int i, bool first, bool last) {
        const uint64_t v = dv + (uint32_t)((i % C::kStages) * C::kTile >> 4);
        if (t5::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kRows / 16; ++kk)
            t5::mma_ts(tmem + 256 + u * D, tmem + u * 128 + kk * 8, v + kk * (2048 >> 4), kPV, !first || kk > 0);
          if (last) t5::commit(&sh.o_done[u]);
        }
        __syncwarp();
      };
      auto commit_one = [&](uint64_t* bar) {
        if (t5::elect_one()) t5::commit(bar);
        __syncwarp();
      };
      const int nt[2] = {tiles0, tiles1};
      bool ok = wait_all(full_of(0), 0);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (ok && nt[u] > 0) {
          ok = wait_all(&sh.q_full[u], 0);
          if (ok) qk(u, 0);
        }
      if (ok) commit_one(&sh.kv_empty[0]);
      for (int j = 0; j < tiles && ok; ++j) {
        const int vi = 2 * j + 1;
        ok = wait_all(full_of(vi), phase_of(vi));
        if (ok && cut(vi)) ok = wait_all(&sh.v_checked[j - (tiles0 - 1)], 0);
        if (ok && j + 1 < tiles) ok = wait_all(full_of(vi + 1), phase_of(vi + 1));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (ok && j < nt[u]) {
            ok = wait_all(&sh.p_full[u], j & 1);
            t5::fence_after();
            if (ok) pv(u, vi, j == 0, j == nt[u] - 1);
          }
          if (ok && j + 1 < nt[u]) qk(u, vi + 1);
        }
        if (ok) {
          commit_one(&sh.kv_empty[vi % C::kStages]);
          if (j + 1 < tiles) commit_one(&sh.kv_empty[(vi + 1) % C::kStages]);
        }
      }
      commit_one(&sh.drain);
      wait_all(&sh.drain, 0);
    } else if (warp >= 10) {
      for (int j = tiles0 - 1; j < tiles; ++j) {
        const int c = j - (tiles0 - 1);
        if (!__all_sync(0xffffffffu, wait(&sh.v_full[c], 0, a.status))) break;
        check_values<D, BF16>(ring + ((2 * j + 1) % C::kStages) * C::kTile, j * kRows, &sh);
        fence_proxy_async_smem();  // the tensor cores read what was written here
        arrive(&sh.v_checked[c]);
      }
    }
  }
  __syncwarp();
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  if (warp == 9) t5::dealloc(sh.tmem, 512);
}

cudaError_t encode(CUtensorMap* m, const void* base, int dim, int heads, int tokens, int64_t stride, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kRows};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool BF16>
cudaError_t launch(const PromptArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  cudaError_t e = encode(&mq, a.q, D, a.q_heads, a.tokens, a.q_stride, BF16);
  if (e == cudaSuccess) e = encode(&mk, a.k, D, a.kv_heads, a.tokens, a.k_stride, BF16);
  if (e == cudaSuccess) e = encode(&mv, a.v, D, a.kv_heads, a.tokens, a.v_stride, BF16);
  if (e != cudaSuccess) return e;
  static SmemAttr attr;
  e = attr.ensure(prompt_kernel<D, BF16>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int pair = (a.q_heads / a.kv_heads) % 2 == 0;
  const int span = pair ? kRows : 2 * kRows;
  const int64_t grid = (int64_t)(pair ? a.q_heads / 2 : a.q_heads) * (a.tokens / span + a.seqs);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  prompt_kernel<D, BF16><<<(unsigned)grid, kThreads, Cfg<D>::kSmem, st>>>(mq, mk, mv, a, pair);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t st) {
  if (a.dim == 64) return a.dtype == KVQ_BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return a.dtype == KVQ_BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace kvq
