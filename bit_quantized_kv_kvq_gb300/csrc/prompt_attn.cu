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
// A block is two units of 128 query rows x one head: two heads of a group on
// the same rows (they share every key tile and its end), or, where the group
// is odd, two row blocks of one head. While the tensor cores work for one
// unit, the other's 128 threads (one row each) turn its scores into weights.
// One persistent CTA per SM runs through blocks, and every role runs ahead of
// the slower ones as far as its buffers go, so that a block's loads and first
// scores overlap the end of the one before. Warps 0-3 and 4-7: softmax of the
// units; 8: TMA; 9: tensor core issue; 10: the gate, which follows the loads and
// checks the values of the tiles that the diagonal cuts (check_values); 11: the
// order of the blocks (Order).
//
// One prompt of 16384 tokens, 32/8 heads of 128: 1315 us, 1672 TFLOP/s, 0.88 of
// the measured bf16 rate. A key tile takes a pair of units 2700 to 3000 clocks,
// of which the products are 2060; a unit's own chain (scores, 1200 clocks of
// softmax, weights to the products, 500 of hand-overs) is as long. Eight
// prompts of 1024 tokens: 75 us (912 TFLOP/s): the ends of blocks, where both
// units write their rows, and half of every tile on the diagonal. With 64
// channels per head the softmax is the longer part: 8192 tokens 293 us (939).
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

// A block of query rows: token c0 + q0 of a sequence of n tokens on.
struct Block {
  int c0, n, q0, hq0;  // hq0 < 0: no more blocks
};

struct Shared {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2], drain;
  uint64_t kv_full[8], kv_empty[8];    // by ring stage
  uint64_t v_full[8];                  // by ring stage: values of a tile that the diagonal cuts
  uint64_t block_full[2], block_empty[2];
  uint64_t fix_ready[2], fix_free[2];  // by parity of the block: `first` written, read
  uint64_t* last_load[8];              // the barrier of the last load into each stage, and its phase
  uint32_t last_phase[8];
  Block block[2];
  uint32_t tmem;
  int any_nonfinite[2];
  int first[2][3][128];  // first token of the cut tiles whose value is NaN, +inf, -inf, per channel
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

// The order of the blocks and an empty unit wait for a whole block: 0.87 s in
// the longest prompt (2^26 tokens, 524288 tiles of 1.65 us for a pair). A poll
// that finds nothing takes 3.8 us, so these are four seconds.
constexpr int kPolls = 8 * kWaitLimit;

// Whole warp: false where the wait gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const bool done = mbar_wait_limited(bar, parity, kPolls, kWaitHintNs);
  if (!done) raise_status(status, kStatusTimeout);
  return __all_sync(0xffffffffu, done);
}

// What all warps follow: the block's units and their key tiles.
struct Units {
  int tiles[2], row0[2], hq[2], most;
  __device__ __forceinline__ Units(const Block& b, bool pair) {
    row0[0] = b.q0;
    row0[1] = pair ? b.q0 : b.q0 + kRows;
    hq[0] = b.hq0;
    hq[1] = pair ? b.hq0 + 1 : b.hq0;
    tiles[0] = row0[0] / kRows + 1;
    tiles[1] = row0[1] < b.n ? row0[1] / kRows + 1 : 0;
    most = max(tiles[0], tiles[1]);
  }
  // The diagonal cuts the last tile of each unit: its values are checked.
  __device__ __forceinline__ bool cut(int j) const { return j >= tiles[0] - 1; }
};

// The block of step `it`, for one warp; false at the end or on a timeout.
__device__ __forceinline__ bool take_block(Shared* sh, int it, uint32_t* status, Block& b) {
  const int slot = it & 1;
  if (!wait(&sh->block_full[slot], (it >> 1) & 1, status)) return false;
  b = sh->block[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(&sh->block_empty[slot]);
  return b.hq0 >= 0;
}

// Blocks in order of their number of key tiles, the longest first: level by
// level of the row block's index, in each level the sequences that reach it
// and their heads. CTA c of G takes blocks c, 2G - 1 - c, 2G + c, ...: the
// turns even out the CTAs' sums. nb: row blocks of each sequence.
struct Order {
  const int* nb;
  int seqs, lots, level;
  uint32_t base, count;  // blocks before this level, and of it (below 2^31, the launch sees to it)

  __device__ __forceinline__ Order(const int* nb_, int seqs_, int lots_) : nb(nb_), seqs(seqs_), lots(lots_) {
    level = 0;
    for (int s = threadIdx.x & 31; s < seqs; s += 32) level = max(level, nb[s]);
    level = __reduce_max_sync(0xffffffffu, level);
    base = count = 0;
  }
  __device__ __forceinline__ uint32_t reach(int s0) const {  // of 32 sequences, those with a row block `level`
    const int s = s0 + (threadIdx.x & 31);
    return __ballot_sync(0xffffffffu, s < seqs && nb[s] > level);
  }
  __device__ __forceinline__ Block get(const PromptArgs& a, int it, int span, bool pair) {
    const uint32_t want = it * gridDim.x + (it & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    while (level >= 0 && want >= base + count) {
      base += count;
      --level;
      int c = 0;
      for (int s0 = 0; level >= 0 && s0 < seqs; s0 += 32) c += __popc(reach(s0));
      count = (uint32_t)c * lots;
    }
    Block b;
    b.c0 = b.n = b.q0 = 0;
    b.hq0 = -1;
    if (level < 0) return b;
    int at = (int)((want - base) / (uint32_t)lots), s = 0;
    const int lot = (int)((want - base) % (uint32_t)lots);
    for (int s0 = 0; s0 < seqs; s0 += 32) {
      const uint32_t m = reach(s0);
      if (__popc(m) > at) {
        const int lane = threadIdx.x & 31;
        const bool mine = ((m >> lane) & 1) && __popc(m & ((1u << lane) - 1)) == at;
        s = s0 + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        break;
      }
      at -= __popc(m);
    }
    b.c0 = a.cu[s];
    b.n = a.cu[s + 1] - b.c0;
    b.q0 = level * span;
    b.hq0 = pair ? 2 * lot : lot;
    return b;
  }
};

// 0 * inf would carry a later token's infinity or NaN to an earlier row. In
// the tiles that the diagonal cuts, the tensor cores get 0 in their place; the
// rows from that token on get them at the end (Shared::first). One warp; a
// tile of finite values (0 * x summed is 0) costs one multiply-add a pair.
template <bool BF16>
__device__ __forceinline__ uint32_t fma_zero(uint32_t x, uint32_t acc) {
  if (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  return acc;
}
template <int D, bool BF16>
__device__ __forceinline__ void check_values(unsigned char* tile, int k0, int (*first)[128], int* any) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  constexpr int kBatch = 8;
  for (int i0 = threadIdx.x & 31; i0 < kRows * D / 8; i0 += 32 * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = reinterpret_cast<uint4*>(tile)[i0 + 32 * k];
    uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      acc[0] = fma_zero<BF16>(x[k].x, acc[0]);
      acc[1] = fma_zero<BF16>(x[k].y, acc[1]);
      acc[2] = fma_zero<BF16>(x[k].z, acc[2]);
      acc[3] = fma_zero<BF16>(x[k].w, acc[3]);
    }
    // +-0 where all were finite
    if ((((acc[0] | acc[1]) | (acc[2] | acc[3])) & 0x7fff7fffu) == 0) continue;
#pragma unroll 1
    for (int k = 0; k < kBatch; ++k) {
      // 16-byte chunk i of the tile: 64-channel half, token row, swizzled place
      const int i = i0 + 32 * k, row = (i >> 3) & 127, ch = (i >> 10) * 64 + (((i & 7) ^ (row & 7)) << 3);
      uint16_t* e = reinterpret_cast<uint16_t*>(tile) + i * 8;
#pragma unroll 1
      for (int j = 0; j < 8; ++j)
        if ((e[j] & kInf) == kInf) {
          const int kind = (e[j] & 0x7fffu) != kInf ? 0 : (e[j] >> 15) ? 2 : 1;
          atomicMin(&first[kind][ch + j], k0 + row);
          *any = 1;
          e[j] = 0;
        }
    }
  }
}

// 2 N scores of a row to weights: p = 2^(s sc - off), packed, and their sum.
template <bool BF16, int N>
__device__ __forceinline__ uint64_t to_weights(const uint32_t* s, uint64_t sc2, float off, uint32_t* p) {
  const uint64_t off2 = f2_pack(-off, -off);
  uint64_t sum0 = f2_pack(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x, y;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, off2), x, y);
    x = exp2_fast(x);
    y = exp2_fast(y);
    if (i & 1) sum1 = f2_add(sum1, f2_pack(x, y));
    else sum0 = f2_add(sum0, f2_pack(x, y));
    p[i] = pack2<BF16>(x, y);
  }
  return f2_add(sum0, sum1);
}

// N scores of a row to the exponents of their weights, s sc - off.
template <int N>
__device__ __forceinline__ void scaled(uint32_t* s, uint64_t sc2, float off) {
  const uint64_t off2 = f2_pack(-off, -off);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float x, y;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sc2, off2), x, y);
    s[i] = __float_as_uint(x);
    s[i + 1] = __float_as_uint(y);
  }
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

// The reference of a row's exponentials moves only when a score passes it by 8
// in units of log 2, so that few tiles scale O (o: it has a value). Each row goes
// by its own scores: its bits do not depend on its neighbours.
//
// A weight is 2^(s sc - m), one multiply-add, with m = raw sc - lift rounded.
// In fp16 the lift of 7 puts weights below 2^15 and 2^-21 of the reference's
// above the type's subnormal numbers (below those, many small weights beside a
// large one would all be off to the same side); bf16 needs none. m's rounding is
// a factor that all weights of the row share, but among scores past 2^20 it
// grows without limit: such a row subtracts `raw` from its scores first (`sub`),
// which is exact near the largest ones. `far`: a row of the warp does.
template <int D, bool BF16>
struct Reference {
  static constexpr float kLift = BF16 ? 0.0f : 7.0f;
  float sc, raw, m, sub, off;  // off: what to_weights takes off the scaled scores
  bool far;

  __device__ __forceinline__ void reset(float sc_) {
    sc = sc_;
    raw = m = -INFINITY;
    sub = off = 0.0f;
    far = false;
  }
  // what m's rounding added, of a row that does not subtract
  __device__ __forceinline__ float rounding() const { return fabsf(m) <= 0x1p20f ? fmaf(raw, sc, -m) - kLift : 0.0f; }

  // s: N scores of the row to subtract from. (Where sc is 0 no score raises
  // the reference, as inf * 0 compares false: every weight is 2^0.)
  template <int N>
  __device__ __forceinline__ void raise(float top, float& l, uint32_t tO, bool o, uint32_t* s) {
    const bool up = (top - raw) * sc > 8.0f;
    if (!__any_sync(0xffffffffu, up || sub != 0.0f)) return;
    raise_rows(up, top, l, tO, o);
    if (N > 0) subtract<N>(s);
  }
  __device__ __forceinline__ void raise_rows(bool up, float top, float& l, uint32_t tO, bool o) {
    if (!__any_sync(0xffffffffu, up)) return;
    float f = 1.0f;
    if (up) {
      f = (raw - top) * sc - rounding();
      raw = top;
      m = fmaf(raw, sc, -kLift);
      f = exp2_fast(f + rounding());
      const bool own = !(fabsf(m) <= 0x1p20f);
      sub = own ? raw : 0.0f;
      off = own ? -kLift : m;
    }
    far = __any_sync(0xffffffffu, sub != 0.0f);
    l *= f;
    if (!o) return;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t x[32];
      t5::ld32(tO + c, x);
      t5::wait_ld32(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
      t5::st32(tO + c, x);
    }
  }
  template <int N>
  __device__ __forceinline__ void subtract(uint32_t* s) const {
    if (!far) return;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) - sub);
  }
};

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

// One unit's warps: scores to weights tile by tile, then the output rows.
template <int D, bool BF16>
__device__ __forceinline__ void softmax_role(const PromptArgs& a, Shared* sh, const int unit, const bool pair) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, r = warp * 32 + lane;
  const uint32_t lanes = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t tS = lanes + unit * 128, tP = tS, tO = lanes + 256 + unit * D;
  const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
  Reference<D, BF16> ref;
  const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  uint32_t tile_phase = 0, out_phase = 0;
  Block b;
  for (int it = 0; take_block(sh, it, a.status, b); ++it) {
    const Units un(b, pair);
    const int tiles = unit ? un.tiles[1] : un.tiles[0], row = (unit ? un.row0[1] : un.row0[0]) + r;
    ref.reset(a.scale_log2);
    float l = 0.0f;
    for (int j = 0; j < tiles; ++j, tile_phase ^= 1) {
      if (!wait(&sh->s_full[unit], tile_phase, a.status)) return;
      t5::fence_after();
      uint64_t sum;
      if (j < tiles - 1) {
        uint32_t s[128], p[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) t5::ld32(tS + 32 * c, s + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) t5::wait_ld32(s + 32 * c);
        ref.template raise<128>(max_of<128>(s), l, tO, j > 0, s);  // s_full came after the last PV
        sum = to_weights<BF16, 32>(s, sc2, ref.off, p);
        t5::st32(tP, p);
        sum = f2_add(sum, to_weights<BF16, 32>(s + 64, sc2, ref.off, p));
        t5::st32(tP + 32, p);
      } else {
        // The tile the diagonal cuts, by groups of 32 keys: the warp's rows see
        // all of the first `warp` groups, up to the row's own key of the next,
        // and nothing after. (P of a group lies where scores already read were.)
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c <= warp; ++c) {
          uint32_t s[32];
          t5::ld32(tS + 32 * c, s);
          t5::wait_ld32(s);
          if (c == warp) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i > lane) s[i] = 0xff800000u;
          }
          top = fmaxf(top, max_of<32>(s));
        }
        ref.template raise<0>(top, l, tO, j > 0, nullptr);
        sum = f2_pack(0.0f, 0.0f);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32], p[16];
          if (c <= warp) {
            t5::ld32(tS + 32 * c, s);
            t5::wait_ld32(s);
            ref.template subtract<32>(s);
            scaled<32>(s, sc2, ref.off);
            if (c == warp) {  // after the scale: -inf * 0 is NaN
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i > lane) s[i] = 0xff800000u;
            }
            sum = f2_add(sum, to_weights<BF16, 16>(s, f2_pack(1.0f, 1.0f), 0.0f, p));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = 0u;
          }
          t5::st16(tP + 16 * c, p);
        }
      }
      t5::wait_st();
      t5::fence_before();
      arrive(&sh->p_full[unit]);
      float x, y;
      f2_unpack(sum, x, y);
      l += x + y;
    }
    const int par = it & 1;
    // an empty unit waits too: its arrival on fix_free counts for this block
    if (!wait(&sh->fix_ready[par], (it >> 1) & 1, a.status)) return;
    if (tiles > 0) {
      if (!wait(&sh->o_done[unit], out_phase, a.status)) return;
      out_phase ^= 1;
      t5::fence_after();
      const float inv = 1.0f / l;
      const bool fix = sh->any_nonfinite[par] != 0;
      uint16_t* out = a.out + ((int64_t)(b.c0 + row) * a.q_heads + (unit ? un.hq[1] : un.hq[0])) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32], w[16];
        t5::ld32(tO + c, o);
        t5::wait_ld32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
        if (fix) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x = __uint_as_float(o[i]);
            if (row >= sh->first[par][1][c + i]) x += INFINITY;
            if (row >= sh->first[par][2][c + i]) x -= INFINITY;
            if (row >= sh->first[par][0][c + i]) x = NAN;
            o[i] = __float_as_uint(x);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<BF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
        if (row < b.n) store_row(out + c, w, wide);
      }
      t5::fence_before();  // O has been read: ordered before the next block's first weights
    }
    __syncwarp();
    if (lane == 0) arrive(&sh->fix_free[par]);
  }
}

template <int D>
__device__ __forceinline__ void load_role(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                          const PromptArgs& a, Shared* sh, unsigned char* smem, bool pair) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, group = a.q_heads / a.kv_heads;
  unsigned char* ring = smem + 2 * C::kTile;
  uint32_t q_phase[2] = {0, 0}, full_phase = 0, cut_phase = 0;
  int i = 0;  // loads into the ring so far
  bool ok = true;
  Block b;
  for (int it = 0; ok && take_block(sh, it, a.status, b); ++it) {
    const Units un(b, pair);
    const int h = b.hq0 / group;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!ok || un.tiles[u] == 0) continue;
      // the first wait is for the phase before the first and passes at once
      ok = wait(&sh->q_empty[u], q_phase[u] ^ 1, a.status);
      if (!ok) break;
      q_phase[u] ^= 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh->q_full[u], C::kTile);
        for (int x = 0; x < D / 64; ++x)
          tma_tile(smem_u32(smem + u * C::kTile + x * (kRows * 128)), &mq, x * 64, un.hq[u], b.c0 + un.row0[u],
                   &sh->q_full[u]);
      }
    }
    for (int k = 0; ok && k < 2 * un.most; ++k, ++i) {  // keys, values, keys, ...
      const int st = i % C::kStages;
      ok = wait(&sh->kv_empty[st], ((i / C::kStages) & 1) ^ 1, a.status);
      if (!ok) break;
      const bool cut = (k & 1) && un.cut(k >> 1);
      uint64_t* bar = cut ? &sh->v_full[st] : &sh->kv_full[st];
      const uint32_t phase = ((cut ? cut_phase : full_phase) >> st) & 1;
      if (cut) cut_phase ^= 1u << st;
      else full_phase ^= 1u << st;
      if (lane == 0) {
        sh->last_load[st] = bar;
        sh->last_phase[st] = phase;
        mbar_arrive_expect_tx(bar, C::kTile);
        for (int x = 0; x < D / 64; ++x)
          tma_tile(smem_u32(ring + st * C::kTile + x * (kRows * 128)), k & 1 ? &mv : &mk, x * 64, h,
                   b.c0 + (k >> 1) * kRows, bar);
      }
    }
  }
  __syncwarp();
  // nothing is in flight into this CTA's shared memory when it ends
  for (int st = 0; st < min(i, C::kStages); ++st) wait(sh->last_load[st], sh->last_phase[st], a.status);
  for (int u = 0; u < 2; ++u) wait(&sh->q_full[u], q_phase[u] ^ 1, a.status);
}

// The whole warp follows the schedule and one elected lane issues: with
// uniform control flow the operands stay in uniform registers, and an
// m128n128k16 issues every 64 clocks, the tensor cores' rate (in a branch of
// one lane it took 90). One warp serves both units, first one, then the other:
// that keeps their softmaxes out of step (with a warp for each unit they ran
// side by side, and the tensor cores idled: 1620 us instead of 1390 for a
// prompt of 16384).
template <int D, bool BF16>
__device__ __forceinline__ void mma_role(const PromptArgs& a, Shared* sh, unsigned char* smem, bool pair) {
  using C = Cfg<D>;
  constexpr uint32_t kQK = t5::instr_desc(128, 128, BF16, false), kPV = t5::instr_desc(128, D, BF16, true);
  const uint32_t tmem = sh->tmem;
  const unsigned char* ring = smem + 2 * C::kTile;
  const uint64_t dq = t5::smem_desc(smem_u32(smem), 16), dk = t5::smem_desc(smem_u32(ring), 16);
  const uint64_t dv = t5::smem_desc(smem_u32(ring), kRows * 128);
  uint32_t q_phase = 0, p_phase[2] = {0, 0}, full_phase = 0;
  // S of unit u from the key tile in stage st
  auto scores = [&](int u, int st) {
    const uint64_t q = dq + (uint32_t)(u * C::kTile >> 4), k = dk + (uint32_t)(st * C::kTile >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4;
      t5::mma_ss(tmem + u * 128, q + off, k + off, kQK, kk > 0);
    }
    t5::commit(&sh->s_full[u]);
  };
  int i = 0;
  bool ok = true;
  Block b;
  for (int it = 0; ok && take_block(sh, it, a.status, b); ++it) {
    const Units un(b, pair);
    {
      const int st = i % C::kStages;
      ok = wait(&sh->kv_full[st], (full_phase >> st) & 1, a.status);
      full_phase ^= 1u << st;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (ok && un.tiles[u] > 0) {
          ok = wait(&sh->q_full[u], (q_phase >> u) & 1, a.status);
          q_phase ^= 1u << u;
          if (ok && t5::elect_one()) {
            scores(u, st);
            if (un.tiles[u] == 1) t5::commit(&sh->q_empty[u]);
          }
          __syncwarp();
        }
      if (ok && t5::elect_one()) t5::commit(&sh->kv_empty[st]);
      __syncwarp();
    }
    for (int j = 0; j < un.most && ok; ++j) {
      const int sv = (i + 2 * j + 1) % C::kStages, sk = (i + 2 * j + 2) % C::kStages;
      const bool more = j + 1 < un.most;
      // p_full also says that this tile's values and the next one's keys are
      // there (gate_role): their waits would cost the products' queue
      if (!un.cut(j)) full_phase ^= 1u << sv;
      if (more) full_phase ^= 1u << sk;
      const uint64_t v = dv + (uint32_t)(sv * C::kTile >> 4);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool mine = j < un.tiles[u], next = j + 1 < un.tiles[u];
        if (ok && mine) {
          ok = wait(&sh->p_full[u], p_phase[u], a.status);
          p_phase[u] ^= 1;
          t5::fence_after();
        }
        if (ok && t5::elect_one()) {
          if (mine) {
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)
              t5::mma_ts(tmem + 256 + u * D, tmem + u * 128 + kk * 8, v + kk * (2048 >> 4), kPV, j > 0 || kk > 0);
            if (!next) t5::commit(&sh->o_done[u]);
          }
          if (u) t5::commit(&sh->kv_empty[sv]);
          if (next) {
            scores(u, sk);
            if (j + 1 == un.tiles[u] - 1) t5::commit(&sh->q_empty[u]);
          }
          if (u && more) t5::commit(&sh->kv_empty[sk]);
        }
        __syncwarp();
      }
    }
    i += 2 * un.most;
  }
  __syncwarp();
  if (t5::elect_one()) t5::commit(&sh->drain);
  __syncwarp();
  wait(&sh->drain, 0, a.status);
}

// Hands out the blocks.
__device__ __forceinline__ void order_role(const PromptArgs& a, Shared* sh, Order order, int span, bool pair) {
  for (int it = 0;; ++it) {
    const Block b = order.get(a, it, span, pair);
    const int slot = it & 1;
    if (it >= 2 && !wait(&sh->block_empty[slot], ((it >> 1) - 1) & 1, a.status)) return;
    if ((threadIdx.x & 31) == 0) {
      sh->block[slot] = b;
      arrive(&sh->block_full[slot]);
    }
    __syncwarp();
    if (b.hq0 < 0) return;
  }
}

// Follows the loads and lets the products of each tile go on: its values and
// the next tile's keys are there, and checked where the diagonal cuts the tile.
template <int D, bool BF16>
__device__ __forceinline__ void gate_role(const PromptArgs& a, Shared* sh, unsigned char* ring, bool pair) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t full_phase = 0, cut_phase = 0, p_phase[2] = {0, 0}, opened[2] = {0, 0};
  int i = 0;
  Block b;
  for (int it = 0; take_block(sh, it, a.status, b); ++it) {
    const Units un(b, pair);
    const int par = it & 1;
    // the rows of the block before the last have read what this one overwrites
    if (!wait(&sh->fix_free[par], ((it >> 1) & 1) ^ 1, a.status)) return;
    if (it < 2 || sh->any_nonfinite[par]) {
      for (int k = lane; k < 3 * 128; k += 32) sh->first[par][k / 128][k % 128] = kNever;
      __syncwarp();
      if (lane == 0) sh->any_nonfinite[par] = 0;
    }
    __syncwarp();
    // Every load is waited for in order, and its stage given back here too: the
    // ring cannot run two phases ahead, which a parity would not tell apart.
    const int s0 = i % C::kStages;
    if (!wait(&sh->kv_full[s0], (full_phase >> s0) & 1, a.status)) return;
    full_phase ^= 1u << s0;
    if (lane == 0) arrive(&sh->kv_empty[s0]);
    for (int j = 0; j < un.most; ++j) {
      const int sv = (i + 2 * j + 1) % C::kStages, sk = (i + 2 * j + 2) % C::kStages;
      const bool cut = un.cut(j), more = j + 1 < un.most;
      if (more) {
        if (!wait(&sh->kv_full[sk], (full_phase >> sk) & 1, a.status)) return;
        full_phase ^= 1u << sk;
        if (lane == 0) arrive(&sh->kv_empty[sk]);
      }
      if (cut) {
        if (!wait(&sh->v_full[sv], (cut_phase >> sv) & 1, a.status)) return;
        cut_phase ^= 1u << sv;
        check_values<D, BF16>(ring + sv * C::kTile, j * kRows, sh->first[par], &sh->any_nonfinite[par]);
        fence_proxy_async_smem();  // the tensor cores read what was written here
      } else {
        if (!wait(&sh->kv_full[sv], (full_phase >> sv) & 1, a.status)) return;
        full_phase ^= 1u << sv;
      }
      __syncwarp();
      if (lane == 0) arrive(&sh->kv_empty[sv]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (j >= un.tiles[u]) continue;
        // one arrival a phase: the one before is complete
        if (opened[u] && !wait(&sh->p_full[u], p_phase[u] ^ 1, a.status)) return;
        opened[u] = 1;
        p_phase[u] ^= 1;
        if (lane == 0) arrive(&sh->p_full[u]);
      }
    }
    arrive(&sh->fix_ready[par]);
    i += 2 * un.most;
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
  int* nb = reinterpret_cast<int*>(smem + (2 + C::kStages) * C::kTile);  // [seqs]
  const int warp = threadIdx.x >> 5;
  const int span = pair ? kRows : 2 * kRows;           // query rows of a block
  const int lots = pair ? a.q_heads / 2 : a.q_heads;   // heads or pairs of them

  if (threadIdx.x == 32) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 129);  // the unit's threads, and the gate
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.block_full[i], 1);
      mbar_init(&sh.block_empty[i], 11);  // every warp but the one that fills it
      mbar_init(&sh.fix_ready[i], 32);
      mbar_init(&sh.fix_free[i], 8);
    }
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 2);  // the products have read it, the gate has seen it
      mbar_init(&sh.v_full[i], 1);
    }
    mbar_fence_init();
  }
  for (int s = threadIdx.x; s < a.seqs; s += kThreads) {
    const int c0 = a.cu[s], n = a.cu[s + 1] - c0;
    const bool bad = n > 0 && (c0 < 0 || n > a.tokens - c0);
    if (bad && blockIdx.x == 0) raise_status(a.status, kStatusBadIndex);
    nb[s] = n > 0 && !bad ? (n + span - 1) / span : 0;
  }
  if (warp == 9) t5::alloc(&sh.tmem, 512);
  t5::fence_before();
  __syncthreads();
  t5::fence_after();

  if (warp < 8) {
    // 256 threads x 208 + 128 x 88 registers = 384 x 168, what the launch holds
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_role<D, BF16>(a, &sh, warp >> 2, pair);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) load_role<D>(mq, mk, mv, a, &sh, smem, pair);
    else if (warp == 9) mma_role<D, BF16>(a, &sh, smem, pair);
    else if (warp == 10) gate_role<D, BF16>(a, &sh, smem + 2 * C::kTile, pair);
    else order_role(a, &sh, Order(nb, a.seqs, lots), span, pair);
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
  const size_t smem = Cfg<D>::kSmem + (size_t)a.seqs * 4;
  e = attr.ensure(prompt_kernel<D, BF16>, Cfg<D>::kSmem + kMaxRequests * 4);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int pair = (a.q_heads / a.kv_heads) % 2 == 0;
  const int span = pair ? kRows : 2 * kRows;
  const int64_t most = (int64_t)(pair ? a.q_heads / 2 : a.q_heads) * (a.tokens / span + a.seqs);  // blocks at most
  if (most > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  prompt_kernel<D, BF16><<<(unsigned)(most < sms ? most : sms), kThreads, smem, st>>>(mq, mk, mv, a, pair);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t st) {
  if (a.dim == 64) return a.dtype == KVQ_BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return a.dtype == KVQ_BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace kvq
