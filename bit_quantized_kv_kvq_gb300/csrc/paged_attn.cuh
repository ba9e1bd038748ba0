// Attention of several new tokens per request over the paged 8-bit cache
// (kvq_paged_attention).
//
//   e_t = c <q_i, k_hat_t>,  o_i = sum_{t <= p_i} softmax(e)_t v_hat_t,  x_hat = code * s(page, head)
//
// For long chunks the 4 D operations per (row, key) bound it, for a few tokens the
// 2 D bytes of codes per key. Both products run on the 5th-generation tensor
// cores as in the prompt attention: S = Q K^T into tensor memory, P where S was,
// O += P V. A unit is 128 rows: every query head of one kv-head on 128 / group
// consecutive tokens, so that the group shares each key tile and the diagonal cuts few.
//
// Codes are exact numbers of the input type (fp16 or bf16, int8 or e4m3; values and
// weights are fp16 in both where they can, see Scales), so the operands are the codes
// themselves, copied to shared memory and converted there by eight warps, and the
// scales stay out of them: a score's factor is c s_k of its page; a value's scale s_v =
// f 2^e goes half into the weight (2^(s - m + log2 f), f in [1, 2)) and half into the
// operand (code 2^e, exact), so that weights stay in their range whatever the scales; the sum
// of weights takes 1 / f off again. Scales below fp16's numbers round the operand, not the
// weight (scales_to). All of this is per group of 16 keys, so pages of any size cost the same.
//
// A block is two units: consecutive tokens of a request on the same key tiles, or,
// where the tokens left fit one unit, the same rows on every other tile (their sums
// are joined at the end), so that a few rows still keep two chains of scores,
// softmax and products going. The blocks' tiles form a line that is cut into
// equal ranges, one per CTA, as in the decode: the grid needs no lengths, ragged
// steps stay even, and one long request fills the GPU. A block that a range's end
// cuts leaves partial sums, which a second kernel merges in the order of the CTAs.
//
// Warps 0-3 and 4-7: softmax of the units; 8: the range's blocks and their
// queries; 9: tensor core issue; 10: tiles (page ids, scales, copies of their codes);
// 11: the gate, which follows the operands (gate_role); 12-19: codes and open rows to operands.
//
// 2048 tokens at 65536, 32/8 heads of 128, int8, fp16: 1933 us, 1120 TFLOP/s, 0.59 of the
// measured bf16 rate (1725 us with a sum of unrounded weights, see to_weights). A pair of
// units takes 4500 clocks a key tile, of which the products are
// 2048: what bounds it is a unit's chain (scores, 2000 clocks of softmax beside the
// conversion on the same schedulers, products at 80 to 90 clocks each for 64, as operands,
// copies and conversion share the bandwidth of shared memory). 4 requests of 8 draft tokens on
// up to 110000, 64/8 heads, bf16: 204 us, 2870 GB/s, 0.43 of the copy rate: about 3300 clocks a
// tile, of which conversion of its two operands takes 1800 and the products 1024. What a tile waits
// for besides has not been measured (no unit of the SM is busy more than 0.6 of the time). Eight
// requests of 1 to 5 tokens on 1000: 29 us, latency of the first tile of cold code, the ends and the merge.
// Tried: codes loaded straight into registers (their latency shows at every fence: 2.4 ms
// for the first case), keys and values in rings of their own with two groups of four
// converting warps (2.17 ms), pieces of half an operand (1.92 ms), one issue loop for
// both orders of the units (1.87 ms), no gate (1.87 ms).
#pragma once

#include "attn_common.cuh"
#include "paged_internal.h"

namespace kvq {
namespace patt {

constexpr int kThreads = 640;
constexpr int kRows = 128;  // rows of a unit, keys of a tile
constexpr int kGroups = kRows / 16;
constexpr int kInfo = 8;    // tiles looked up ahead
constexpr int kParts = 4;   // parts handed out ahead
constexpr int kNever = 0x7fffffff;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kFar = 0x1p20f;

// Places on the line, about 700 clocks each: of a tile of two units' rows, of one that a
// unit takes alone, and of a block for its queries, ends and merge. (Measured with 128
// channels. With 64, where operands are half as large, they are taken over and not tuned.)
constexpr int kBoth = 6, kAlone = 5, kExtra = 18;

template <int D>
struct Cfg {
  static constexpr int kTile = kRows * D * 2;       // bytes of a Q, K or V operand
  static constexpr int kStages = D == 128 ? 3 : 6;  // K and V operands
  static constexpr int kRaw = kRows * D;            // bytes of an operand's codes
  static constexpr int kRaws = D == 128 ? 3 : 6;    // codes in flight
  static constexpr int kSmem = 1024 + (2 + kStages) * kTile + kRaws * kRaw;
};

struct Params {
  CUtensorMap mq;
  PagedDev c;
  PagedAttnArgs a;
  int ctas;
  // heads of a unit, chunks of 128 heads of a larger group, tokens of a unit, (kv-head, chunk) pairs
  int unit_heads, chunks, unit_tokens, lots;
  int4* pos;     // [ctas + 1] where each CTA's range starts: request, lot, block, tile
  float* part_o; // [ctas][2][256][D]
  float* part_ml;
};

__host__ __device__ inline size_t pos_bytes(int ctas) { return ((size_t)(ctas + 1) * 16 + 255) / 256 * 256; }

// --------------------------------------------------------------------------
// The line
// --------------------------------------------------------------------------
struct Req {
  int c0, m, n;  // first packed token, new tokens, length with them
};

__device__ __forceinline__ Req load_req(const Params& p, int b, bool& bad) {
  Req r;
  r.c0 = p.a.cu[b];
  const long long m = (long long)p.a.cu[b + 1] - r.c0;
  r.n = p.a.lens[b];
  r.m = 0;
  if (m <= 0) return r;
  if (r.c0 < 0 || m > p.a.tokens - r.c0 || r.n < m || r.n > (long long)p.c.max_pages << p.c.page_shift) {
    bad = true;
    return r;
  }
  r.m = (int)m;
  return r;
}

// The blocks of a request for one lot, and the places before block i (whole
// blocks: their tiles by the sum of their ends).
struct Blocks {
  long long old, whole, rest;
  int bt, ut, n;
  __device__ __forceinline__ Blocks(const Params& p, const Req& r) {
    ut = p.unit_tokens;
    bt = 2 * ut;
    n = r.n;
    old = r.n - r.m;
    whole = r.m / bt;
    rest = r.m % bt;
  }
  __device__ __forceinline__ long long count() const { return whole + (rest > 0); }
  __device__ __forceinline__ int last_weight() const { return rest <= ut ? kAlone : kBoth; }
  __device__ __forceinline__ long long before(long long i) const {
    const long long ends = i * old + bt * (i * (i + 1) / 2);
    return i * kExtra + (ends >> 7) * kBoth + (((ends & 127) * kBoth) >> 7);
  }
  __device__ __forceinline__ long long all() const {
    return before(whole) + (rest > 0 ? kExtra + (long long)last_weight() * ((n + kRows - 1) / kRows) : 0);
  }
  __device__ __forceinline__ int tiles(long long i) const {
    const long long end = i < whole ? old + (i + 1) * bt : n;
    return (int)((end + kRows - 1) / kRows);
  }
};

struct Pos {
  int b, lot, i, t;
};

// n / d, in 32 bits where both fit (a 64-bit division takes half a microsecond).
__device__ __forceinline__ long long quotient(unsigned long long n, unsigned long long d) {
  return (n | d) >> 32 ? (long long)(n / d) : (long long)((uint32_t)n / (uint32_t)d);
}

// The place v of a request's line.
__device__ __forceinline__ Pos locate(const Params& p, int b, const Req& r, long long v) {
  const Blocks k(p, r);
  const long long all = k.all();
  Pos x;
  x.b = b;
  x.lot = (int)quotient(v, all);
  const long long w = v - x.lot * all;
  long long i = k.whole, lo = k.before(k.whole), hi = all;
  if (w < lo) {
    i = 0;
    for (long long n = k.whole; n > 1;) {
      const long long half = n >> 1;
      if (k.before(i + half) <= w) i += half, n -= half;
      else n = half;
    }
    lo = k.before(i);
    hi = k.before(i + 1);
  }
  const int tiles = k.tiles(i);
  long long t = quotient((w - lo) * tiles, hi - lo);
  // no slivers: a cut near an end is none
  const int least = tiles >= 16 ? 2 : 1;
  if (t < least) t = 0;
  if (tiles - t < least) t = 0, ++i;
  x.i = (int)i;
  x.t = (int)t;
  if (i == k.count()) x.i = 0, ++x.lot;
  return x;
}

// --------------------------------------------------------------------------
// Shared memory
// --------------------------------------------------------------------------
struct alignas(16) Info {  // per 16 keys
  float2 a[kGroups], lg[kGroups];  // score factor, log2 f, twice each: operands of pairs
  float inv[kGroups];              // 1 / f
  uint32_t up[kGroups];                          // 2^e, a pair of the values' operand type
  uint32_t low[kGroups];                         // what is left of 2^e where fp16 does not hold it, else 1
  int page[2][kGroups];                          // of keys, of values; -1: open rows or none, -2: zeros
  int coded;                                     // all of them pages, with low 1
  int half;                                      // values and weights in fp16
};

struct Part {
  int b, h, hq0, heads;  // kv-head, first query head and how many of the chunk
  int c0, tokens, pos0;  // first packed token, how many, position of the first
  int n, t0, t1, tiles, slot;  // slot: -1 the whole block, else where its partial sums go
  bool both;             // two units of rows; else one, on every other tile
  __device__ __forceinline__ bool has(int unit) const { return unit == 0 || both || t1 - t0 > 1; }
  __device__ __forceinline__ bool mine(int unit, int t) const { return both || ((t - t0) & 1) == unit; }
};

struct Shared {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2], drain;
  uint64_t kv_full[8], kv_empty[8];  // by operand stage
  uint64_t raw_full[6], raw_empty[6];  // by stage of codes
  uint64_t info_full[kInfo], info_empty[kInfo];
  uint64_t part_full[kParts], part_empty[kParts];
  uint64_t fix_ready[2], fix_free[2];  // by parity of the part: `first` written, read
  uint64_t join_ready, join_done;
  Info info[kInfo];
  Part part[kParts];
  int half[8];  // by operand stage: its values are fp16
  uint32_t tmem;
  // By parity of the part: the number of the last part with a value in the open page that is
  // not finite (from 1 on), and the first position of a NaN, +inf, -inf per channel, under the part it is of (first_key).
  int any_nonfinite[2];
  unsigned long long first[2][3][128];
  float join[2][kRows][3];  // of a unit's row: reference, sum, factor of its O
  long long scan[kThreads / 32];
  Pos from, to;
};

// Waits last as long as a few tiles, but those of the warp that hands out the parts as
// long as a block (four and 32 seconds, a poll that finds nothing taking 3.8 us).
constexpr int kPolls = 8 * kWaitLimit, kLongPolls = 64 * kWaitLimit;

// Whole warp: false where the wait gave up. (A rolled loop: unrolled, the many
// waits of the roles were three quarters of the kernel's code, and its fetches
// what the warps waited for.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status, int polls = kPolls) {
  bool done = false;
#pragma unroll 1
  for (int k = 0; k < polls && !done; ++k) done = mbar_try_wait_hint(bar, parity, kWaitHintNs);
  if (!done) raise_status(status, kStatusTimeout);
  return __all_sync(kFull, done);
}

// The part of step `it`, for one warp, which gives it back when done with it;
// null at the end or on a timeout.
__device__ __forceinline__ const Part* take_part(Shared* sh, int it, uint32_t* status) {
  const int slot = it % kParts;
  if (!wait(&sh->part_full[slot], (it / kParts) & 1, status)) return nullptr;
  return sh->part[slot].b >= 0 ? &sh->part[slot] : nullptr;
}
__device__ __forceinline__ void give_part(Shared* sh, int it) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(&sh->part_empty[it % kParts]);
}

// The operands of a part's tiles, numbered in the order in which the products take
// them: K0 V0 K1 V1 ..., or, where units and tiles alternate, K0 K1 V0 K2 V1 ... . Stages
// of codes and operands go round in this order, and whoever waits for one waits for all
// of them, one after the other: of phases seen only now and then a parity would not tell which one it is.
struct Order {
  uint32_t base;  // operands before this part
  int n;          // tiles
  bool both;
  // operand k of the part: whether it is values, and of which tile
  __device__ __forceinline__ int which(int k) const { return both ? k & 1 : k == 2 * n - 1 || (k > 0 && (k & 1) == 0); }
  __device__ __forceinline__ int tile(int k) const { return both || k == 2 * n - 1 || k == 0 ? k >> 1 : k & 1 ? (k + 1) >> 1 : (k >> 1) - 1; }
};

// --------------------------------------------------------------------------
// Blocks and their queries
// --------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void part_role(const Params& p, Shared* sh, unsigned char* smem) {
  const int lane = threadIdx.x & 31;
  uint32_t* status = p.c.status;
  uint32_t q_phase[2] = {0, 0};
  Pos x = sh->from;
  const Pos to = sh->to;
  bool ok = true, bad = false;
  Req r = {0, 0, 0};
  if (x.b < p.a.requests) r = load_req(p, x.b, bad);
  for (int it = 0; ok; ++it) {
    // the next request with a place
    while (x.b < p.a.requests && (x.lot == p.lots || r.m == 0)) {
      x.lot = x.i = x.t = 0;
      if (++x.b < p.a.requests) r = load_req(p, x.b, bad);
    }
    const bool before = x.b < to.b || (x.b == to.b && (x.lot < to.lot || (x.lot == to.lot && x.i < to.i)));
    const bool here = x.b == to.b && x.lot == to.lot && x.i == to.i;
    Part y;
    y.b = -1;
    if (x.b < p.a.requests && (before || (here && x.t < to.t))) {
      const Blocks k(p, r);
      const int chunk = x.lot % p.chunks;
      y.b = x.b;
      y.h = x.lot / p.chunks;
      y.hq0 = y.h * p.a.group + chunk * kRows;
      y.heads = min(p.unit_heads, p.a.group - chunk * kRows);
      const long long first = (long long)x.i * k.bt;
      y.c0 = r.c0 + (int)first;
      y.tokens = (int)min((long long)k.bt, r.m - first);
      y.pos0 = (int)(k.old + first);
      y.n = r.n;
      y.tiles = k.tiles(x.i);
      y.t0 = x.t;
      y.t1 = here ? to.t : y.tiles;
      y.slot = y.t0 > 0 ? 0 : y.t1 < y.tiles ? 1 : -1;
      y.both = y.tokens > k.ut;
      x.t = 0;
      if (++x.i == k.count()) x.i = 0, ++x.lot;
    }
    const int slot = it % kParts;
    if (it >= kParts && !wait(&sh->part_empty[slot], (it / kParts - 1) & 1, status, kLongPolls)) break;
    if (lane == 0) {
      sh->part[slot] = y;
      arrive(&sh->part_full[slot]);
    }
    __syncwarp();
    if (y.b < 0) break;
    const uint32_t bytes = (uint32_t)p.unit_heads * p.unit_tokens * D * 2;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!ok || !y.has(u)) continue;
      // the first wait is for the phase before the first and passes at once
      ok = wait(&sh->q_empty[u], q_phase[u] ^ 1, status, kLongPolls);
      if (!ok) break;
      q_phase[u] ^= 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh->q_full[u], bytes);
        for (int half = 0; half < D / 64; ++half)
          tma_tile(smem_u32(smem + u * Cfg<D>::kTile + half * (kRows * 128)), &p.mq, half * 64, y.hq0,
                   y.c0 + (y.both ? u * p.unit_tokens : 0), &sh->q_full[u]);
      }
    }
  }
  __syncwarp();
  // nothing is in flight into this CTA's shared memory when it ends
  for (int u = 0; u < 2; ++u) wait(&sh->q_full[u], q_phase[u] ^ 1, status);
}

// --------------------------------------------------------------------------
// Tiles: pages, scales, prefetch
// --------------------------------------------------------------------------
struct Scales {
  float a, lg, inv;  // of Info
  int e;
  bool zero, half;  // values' operand is zeros; code 2^e is an exact fp16 number
};

// The least e with an exact fp16 product code 2^e (e4m3: multiples of 2^-9), and the least 2^e of fp16.
template <int CODE>
constexpr int kExactHalf = CODE == KVQ_PAGE_INT8 ? -24 : -15;
constexpr int kLeastHalf = -24;

// 2^e stays a number of the operand's type, with products code 2^e exact. An fp16 cache may
// have smaller scales (e4m3: values below 2^-6.2, int8: below 2^-17): there f is taken from
// [1/2, 1) and the product is rounded, once, to fp16's subnormal numbers: f times at most 2^-25, half
// of the output's smallest step. (A smaller f would take the tokens' weights below fp16's numbers, and
// with them their share of the sum.) A bf16 weight holds the f of scales below 2^-126.
template <int CODE, bool BF16>
__device__ __forceinline__ Scales scales_to(float sk, float sv, float scale_log2) {
  constexpr int kMaxHalf = CODE == KVQ_PAGE_INT8 ? 8 : 7;
  const bool finite = fabsf(sv) <= 3.0e38f;
  const uint32_t bits = __float_as_uint(sv);
  Scales r;
  r.e = (int)((bits >> 23) & 255) - 127;
  float f = __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);
  if (BF16) {
    if (r.e < -126) r.e = -126, f = sv * 0x1p126f;  // exact
  } else if (r.e < kExactHalf<CODE>) {
    ++r.e, f *= 0.5f;
  }
  r.zero = !finite || sv == 0.0f;
  if (r.zero) r.e = 0, f = finite ? 1.0f : NAN;
  r.half = !BF16 || (r.e >= kExactHalf<CODE> && r.e <= kMaxHalf);
  r.a = fabsf(sk) <= 3.0e38f ? sk * scale_log2 : NAN;
  r.lg = log2f(f);
  r.inv = f == f ? 1.0f / f : 1.0f;  // a masked weight's share stays 0
  return r;
}

// The pair 2^e (0 below the type's numbers).
__device__ __forceinline__ uint32_t power_pair(int e, bool half) {
  const uint32_t w = !half              ? (uint32_t)(e + 127) << 7
                     : e >= -14         ? (uint32_t)(e + 15) << 10
                     : e >= kLeastHalf  ? 1u << (e - kLeastHalf)
                                        : 0u;
  return w | (w << 16);
}

// Four tiles at a time, a lane for each of their groups of 16 keys. The next
// four's pages are looked up, and their codes called into L2, before these four go out.
template <int D, int CODE, bool BF16>
__device__ __forceinline__ void tile_role(const Params& p, Shared* sh, unsigned char* raw) {
  using C = Cfg<D>;
  const PagedDev& c = p.c;
  const int lane = threadIdx.x & 31, g = lane & 7, ahead = lane >> 3, P = 1 << c.page_shift;
  int i = 0;       // tiles so far
  uint32_t x = 0;  // operands so far
  bool ok = true;
  for (int it = 0; ok; ++it) {
    const Part* at = take_part(sh, it, c.status);
    if (!at) break;
    const int n = at->n, full = n & ~(P - 1), t0 = at->t0, t1 = at->t1, head = at->h;
    const bool both = at->both;
    const int32_t* row = p.a.table + (int64_t)at->b * c.max_pages;
    give_part(sh, it);
    // -1: no page, -2: a bad one
    auto page_of = [&](int t) {
      if (t + ahead >= t1) return -1;
      const int pos = (t + ahead) * kRows + 16 * g;
      if (pos >= full) return -1;
      const int page = row[pos >> c.page_shift];
      return page >= 0 && page < c.num_pages ? page : -2;
    };
    auto scales_of = [&](int page) {
      float2 s = make_float2(0.0f, 0.0f);
      if (page >= 0) {
        const int64_t ph = ((int64_t)page * c.heads + head) * 2;
        if ((16 * g & (P - 1)) == 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(c.pages + (ph << c.page_shift) * D),
                       "r"(2 * P * D)
                       : "memory");
        s = *reinterpret_cast<const float2*>(c.scales + ph);
      }
      return s;
    };
    // copies the codes of tile `tile`'s keys or values
    auto call = [&](int tile, int which) {
      const int id = sh->info[tile % kInfo].page[which][g], st = x % C::kRaws;
      const bool copy = lane < 8 && id >= 0 && (16 * g & (P - 1)) == 0;
      const uint32_t copies = __popc(__ballot_sync(kFull, copy));
      if (!wait(&sh->raw_empty[st], ((x / C::kRaws) & 1) ^ 1, c.status)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&sh->raw_full[st], copies * P * D);
      __syncwarp();
      if (copy)
        bulk_g2s(raw + st * C::kRaw + 16 * g * D, c.pages + ((((int64_t)id * c.heads + head) * 2 + which) << c.page_shift) * D,
                 P * D, &sh->raw_full[st]);
      ++x;
      return true;
    };
    int page = page_of(t0);
    float2 s = scales_of(page);
    for (int t = t0; ok && t < t1; t += 4) {
      Scales f = {p.a.scale_log2, 0.0f, 1.0f, 0, true, true};
      if (page >= 0) f = scales_to<CODE, BF16>(s.x, s.y, p.a.scale_log2);
      if (page == -2) {
        raise_status(c.status, kStatusBadIndex);
        f.a = 0.0f, f.lg = -INFINITY;
      }
      const int page_v = page >= 0 && f.zero ? -2 : page;
      const uint32_t own = 255u << (lane & 24);  // the lanes of the tile
      const bool down = !BF16 && f.e < kLeastHalf;  // 2^e in two factors, the first with exact products
      const bool coded = (__ballot_sync(kFull, page >= 0 && page_v >= 0 && !down) & own) == own;
      // The values' products take fp16 in either type, where they can: weights of 11 bits.
      // (A page of zeros or NaN, one out of range and what lies past the request's end are
      // zeros as operands, and no reason against it: their neighbours' rows keep their bits.)
      const bool open = page == -1 && (t + ahead) * kRows + 16 * g < n;
      const bool half = (__ballot_sync(kFull, !BF16 || (!open && f.half)) & own) == own;
      const int live = min(4, t1 - t), now = page;
      page = page_of(t + 4);
#pragma unroll 1
      for (int k = 0; ok && k < live; ++k, ++i) {
        const int slot = i % kInfo;
        ok = wait(&sh->info_empty[slot], ((i / kInfo) & 1) ^ 1, c.status);
        if (!ok) break;
        if (ahead == k) {
          Info& o = sh->info[slot];
          o.a[g] = make_float2(f.a, f.a);
          o.lg[g] = make_float2(f.lg, f.lg);
          o.inv[g] = f.inv;
          o.up[g] = power_pair(down ? kExactHalf<CODE> : f.e, half);
          o.low[g] = power_pair(down ? f.e - kExactHalf<CODE> : 0, true);
          o.page[0][g] = now;
          o.page[1][g] = page_v;
          if (g == 0) o.coded = coded, o.half = half;
        }
        __syncwarp();
        if (lane == 0) arrive(&sh->info_full[slot]);
        ok = call(i, 0);
        if (ok && both) ok = call(i, 1);
        if (ok && !both && t + k > t0) ok = call(i - 1, 1);
        if (k == 0) s = scales_of(page);
      }
    }
    if (ok && !both) ok = call(i - 1, 1);
  }
  __syncwarp();
  // nothing is in flight into this CTA's shared memory when it ends
  for (uint32_t y = x > C::kRaws ? x - C::kRaws : 0; y < x; ++y) wait(&sh->raw_full[y % C::kRaws], (y / C::kRaws) & 1, c.status);
}

// --------------------------------------------------------------------------
// Codes to operands
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The four codes of a word as numbers of the input type, times the pair `up` (values).
template <int CODE, bool BF16, bool VALUES>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t up, uint32_t& lo, uint32_t& hi) {
  if (CODE == KVQ_PAGE_INT8 && !BF16) {
    // 0x6400 | u is 1024 + u in fp16; u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else if (CODE == KVQ_PAGE_INT8) {
    // 0x4300 | u is 128 + u in bf16 for u < 128: the low seven bits, less 128, and 128 more where the sign is set
    const uint32_t u = w & 0x7f7f7f7fu, s = w & 0x80808080u;
    lo = bsub2(__byte_perm(u, 0x43434343u, 0x4140), __byte_perm(s, 0x43434343u, 0x4140));
    hi = bsub2(__byte_perm(u, 0x43434343u, 0x4342), __byte_perm(s, 0x43434343u, 0x4342));
  } else if (!BF16) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // the code's bits as those of a bf16 number 2^-120 of it
    const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
    lo = mul2<true>((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), 0x7b807b80u);
    hi = mul2<true>((b & 0x80008000u) | ((b >> 4) & 0x07f007f0u), 0x7b807b80u);
  }
  if (VALUES) lo = mul2<BF16>(lo, up), hi = mul2<BF16>(hi, up);
}

// A thread's eight channels of a row: eight threads side by side read 64 bytes of
// codes and write the eight 16-byte chunks of a 128-byte row of the operand tile,
// which the swizzle puts into different banks.
template <int D>
struct Place {
  int row, channel;
  uint32_t at;  // bytes of its chunk in the tile
  __device__ __forceinline__ Place(int tid) {
    const int chunk = tid % (D / 8);
    row = tid / (D / 8);
    channel = chunk * 8;
    at = (chunk >> 3) * (kRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  }
};

// Codes of the thread's channels in the row `down` further down (a multiple of 8). LOW: times the
// pair `low` too.
template <int D, int CODE, bool BF16, bool VALUES, bool LOW = false>
__device__ __forceinline__ void put_codes(unsigned char* tile, const Place<D>& at, int down, const uint2& x, uint32_t up,
                                          uint32_t low = 0) {
  uint4 a;
  widen4<CODE, BF16, VALUES>(x.x, up, a.x, a.y);
  widen4<CODE, BF16, VALUES>(x.y, up, a.z, a.w);
  if (LOW) a.x = mul2<BF16>(a.x, low), a.y = mul2<BF16>(a.y, low), a.z = mul2<BF16>(a.z, low), a.w = mul2<BF16>(a.w, low);
  *reinterpret_cast<uint4*>(tile + at.at + down * 128) = a;
}

// Position `pos` of part `it`. A later part's keys are below all of an earlier one, so that the
// smallest key is the last part's first position, whatever an earlier part left there: nothing is put
// back between parts, and no warp has to know how far the others are.
__device__ __forceinline__ unsigned long long first_key(int it, int pos) {
  return ((unsigned long long)(uint32_t)~it << 32) | (uint32_t)pos;
}

// Infinities and NaN of 8 values of an open row: 0 in their place, and where
// they were, in sh->first (0 * inf would carry them to rows that do not see them).
template <bool BF16>
__device__ __forceinline__ void finite8(uint4& x, int pos, int ch, int it, unsigned long long (*first)[128], int* any) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t acc = fma_zero<BF16>(x.w, fma_zero<BF16>(x.z, fma_zero<BF16>(x.y, fma_zero<BF16>(x.x, 0u))));
  if ((acc & 0x7fff7fffu) == 0) return;
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t v = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu;
    if ((v & kInf) == kInf) {
      const int kind = (v & 0x7fffu) != kInf ? 0 : (v >> 15) ? 2 : 1;
      atomicMin(&first[kind][ch + j], first_key(it, pos));
      *any = it + 1;
      w[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
    }
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of pass after pass of an operand that is all pages.
template <int D, int CODE, bool BF16, bool VALUES>
__device__ __forceinline__ void convert_codes(unsigned char* to, const Place<D>& at, const uint2* from, const Info& info) {
  constexpr int kPasses = D / 16, kStep = 2048 / D;
#pragma unroll
  for (int k0 = 0; k0 < kPasses; k0 += 4) {
    uint2 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = from[(k0 + k) * 256];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      put_codes<D, CODE, BF16, VALUES>(to, at, (k0 + k) * kStep, x[k], VALUES ? info.up[((k0 + k) * kStep + at.row) >> 4] : 0u);
  }
}

// Eight warps take every operand together, in the order of the products.
template <int D, int CODE, bool BF16>
__device__ __forceinline__ void convert_role(const Params& p, Shared* sh, unsigned char* ring, const unsigned char* raw) {
  using C = Cfg<D>;
  constexpr int kPasses = D / 16, kStep = 2048 / D;  // passes over a tile, rows of one
  const PagedDev& c = p.c;
  const int tid = threadIdx.x & 255, lane = threadIdx.x & 31, P = 1 << c.page_shift;
  const Place<D> at(tid);
  int tiles = 0;  // before this part
  for (int it = 0;; ++it) {
    const Part* part = take_part(sh, it, c.status);
    if (!part) return;
    const int par = it & 1;
    const Order order = {2u * tiles, part->t1 - part->t0, part->both};
    // the rows of the part before the last have read what this one may overwrite
    if (!wait(&sh->fix_free[par], ((it >> 1) & 1) ^ 1, c.status)) return;
#pragma unroll 1
    for (int o = 0; o < 2 * order.n; ++o) {
      const int which = order.which(o), j = order.tile(o), tile = tiles + j;
      const uint32_t i = order.base + o, slot = tile % kInfo, st = i % C::kStages, rs = i % C::kRaws;
      const Info& info = sh->info[slot];
      unsigned char* to = ring + st * C::kTile;
      const uint2* from = reinterpret_cast<const uint2*>(raw + rs * C::kRaw) + tid;  // of pass k: 256 k further on
      if (which == 0 && !wait(&sh->info_full[slot], (tile / kInfo) & 1, c.status)) return;
      if (!wait(&sh->raw_full[rs], (i / C::kRaws) & 1, c.status)) return;
      if (!wait(&sh->kv_empty[st], ((i / C::kStages) & 1) ^ 1, c.status)) return;
      const bool coded = info.coded != 0, half = info.half != 0;
      if (BF16 && which && lane == 0) sh->half[st] = half;  // all warps the same
      if (coded) {
        if (which == 0) convert_codes<D, CODE, BF16, false>(to, at, from, info);
        else if (!BF16 || half) convert_codes<D, CODE, false, true>(to, at, from, info);
        else convert_codes<D, CODE, BF16, true>(to, at, from, info);
      } else {
        const int n = part->n, full = n & ~(P - 1), t = part->t0 + j;
        const uint16_t* tail =
            c.tails + (((((int64_t)part->b * c.heads + part->h) * 2 + which) << c.page_shift)) * D + at.channel;
#pragma unroll 1
        for (int k0 = 0; k0 < kPasses; k0 += 4) {
          uint4 a[4];
          int page[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = (k0 + k) * kStep + at.row, pos = t * kRows + row;
            page[k] = info.page[which][row >> 4];
            a[k] = make_uint4(0u, 0u, 0u, 0u);
            if (page[k] == -1 && pos < n) a[k] = *reinterpret_cast<const uint4*>(tail + (int64_t)(pos - full) * D);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int down = (k0 + k) * kStep, row = down + at.row, pos = t * kRows + row;
            if (page[k] >= 0) {
              const uint32_t one = BF16 ? 0x3f803f80u : 0x3c003c00u;  // keys: times 1
              if (BF16 && which && half) put_codes<D, CODE, false, true>(to, at, down, from[(k0 + k) * 256], info.up[row >> 4]);
              else put_codes<D, CODE, BF16, true, !BF16>(to, at, down, from[(k0 + k) * 256],
                                                         which ? info.up[row >> 4] : one, which ? info.low[row >> 4] : one);
            } else {
              if (which) finite8<BF16>(a[k], pos, at.channel, it, sh->first[par], &sh->any_nonfinite[par]);
              *reinterpret_cast<uint4*>(to + at.at + down * 128) = a[k];
            }
          }
        }
      }
      fence_proxy_async_smem();  // the tensor cores read what was written here
      __syncwarp();
      if (lane == 0) {
        arrive(&sh->kv_full[st]);
        arrive(&sh->raw_empty[rs]);
        if (which) arrive(&sh->info_empty[slot]);
      }
    }
    tiles += order.n;
    __syncwarp();
    if (lane == 0) arrive(&sh->fix_ready[par]);
    give_part(sh, it);
  }
}

// --------------------------------------------------------------------------
// Products
// --------------------------------------------------------------------------
// Tells the compiler that a value is the whole warp's: what the products' operands
// are made of stays in uniform registers then.
template <typename T>
__device__ __forceinline__ T uniform(T x) {
  return (T)__shfl_sync(kFull, x, 0);
}

// Operand descriptors differ in the lower word only (address, and in bits 16 up the
// stride); the upper one says 1024 bytes between groups of eight rows and the 128-byte swizzle.
__device__ __forceinline__ uint64_t operand(uint32_t lower) {
  return (uint64_t)lower | ((uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32);
}

// The issue of the products is as long as the products themselves where it takes
// more than 64 clocks each, so the two orders are written out, a unit being a constant
// in each step.
template <int D, bool BF16>
__device__ __forceinline__ void mma_role(const Params& p, Shared* sh, unsigned char* smem) {
  using C = Cfg<D>;
  constexpr uint32_t kQK = t5::instr_desc(128, 128, BF16, false), kPV = t5::instr_desc(128, D, BF16, true);
  constexpr uint32_t kHalfPV = t5::instr_desc(128, D, false, true);
  const uint32_t tmem = uniform(sh->tmem);
  uint32_t* status = p.c.status;
  const uint32_t base = smem_u32(smem) >> 4;
  uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
  uint32_t st = 0, st_phase = 0;  // the next operand's stage
  bool ok = true;
  auto next = [&]() {  // the next operand's stage
    const uint32_t at = st;
    if (++st == C::kStages) st = 0, st_phase ^= 1;
    return at;
  };
  auto next_ready = [&]() {  // ... once it is there
    ok = ok && wait(&sh->kv_full[st], st_phase, status);
    return next();
  };
  // S of unit u from the keys in stage at
  auto scores = [&](const int u, uint32_t at) {
    uint32_t b = base;
    asm volatile("" : "+r"(b));  // made here each time: sixteen operands kept over the loop spill
    const uint32_t q = b + (1u << 16) + u * (C::kTile >> 4), k = b + (1u << 16) + (2 + at) * (C::kTile >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4;
      t5::mma_ss(tmem + u * 128, operand(q + off), operand(k + off), kQK, kk > 0);
    }
    t5::commit(&sh->s_full[u]);
  };
  auto values = [&](const int u, uint32_t at, bool first, uint32_t kind) {
    uint32_t b = base;
    asm volatile("" : "+r"(b));
    const uint32_t v = b + ((kRows * 128 >> 4) << 16) + (2 + at) * (C::kTile >> 4);
#pragma unroll
    for (int kk = 0; kk < kRows / 16; ++kk)
      t5::mma_ts(tmem + 256 + u * D, tmem + u * 128 + 64 + kk * 8, operand(v + kk * (2048 >> 4)), kind, kk > 0 || !first);
  };
  auto query = [&](const int u) {
    ok = ok && wait(&sh->q_full[u], q_phase[u], status);
    q_phase[u] ^= 1;
  };
  auto weights = [&](const int u) {
    ok = ok && wait(&sh->p_full[u], p_phase[u], status);
    p_phase[u] ^= 1;
    t5::fence_after();
  };
  for (int it = 0; ok; ++it) {
    const Part* part = take_part(sh, it, status);
    if (!part) break;
    const int n = uniform(part->t1 - part->t0);
    const bool both = uniform(part->both);
    give_part(sh, it);
    if (both) {
      uint32_t k = next_ready();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        query(u);
        t5::fence_after();
        if (ok && t5::elect_one()) {
          scores(u, k);
          if (n == 1) t5::commit(&sh->q_empty[u]);
          if (u) t5::commit(&sh->kv_empty[k]);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        const uint32_t v = next();
        k = more ? next() : 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          weights(u);  // says that these operands are there, too (gate_role)
          const uint32_t kind = BF16 && uniform(sh->half[v]) ? kHalfPV : kPV;
          if (ok && t5::elect_one()) {
            values(u, v, j == 0, kind);
            if (u) t5::commit(&sh->kv_empty[v]);
            if (more) {
              scores(u, k);
              if (u) t5::commit(&sh->kv_empty[k]);
              if (j + 2 == n) t5::commit(&sh->q_empty[u]);
            } else {
              t5::commit(&sh->o_done[u]);
            }
          }
          __syncwarp();
        }
      }
    } else {  // tile j is unit j & 1's
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u >= n) continue;
        query(u);
        const uint32_t k = next_ready();
        t5::fence_after();
        if (ok && t5::elect_one()) {
          scores(u, k);
          t5::commit(&sh->kv_empty[k]);
          if (u + 2 >= n) t5::commit(&sh->q_empty[u]);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j0 = 0; j0 < n && ok; j0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = j0 + u;
          if (j >= n) continue;
          const bool more = j + 2 < n;
          const uint32_t v = next(), k = more ? next() : 0;
          weights(u);
          const uint32_t kind = BF16 && uniform(sh->half[v]) ? kHalfPV : kPV;
          if (ok && t5::elect_one()) {
            values(u, v, j0 == 0, kind);
            t5::commit(&sh->kv_empty[v]);
            if (more) {
              scores(u, k);
              t5::commit(&sh->kv_empty[k]);
              if (j + 4 >= n) t5::commit(&sh->q_empty[u]);
            } else {
              t5::commit(&sh->o_done[u]);
            }
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  if (t5::elect_one()) t5::commit(&sh->drain);
  __syncwarp();
  wait(&sh->drain, 0, status);
}

// Follows the operands and lets each step's products go on: its values and the
// unit's next keys are there. (Waited for by the issuing warp they cost the products' queue.)
template <int D>
__device__ __forceinline__ void gate_role(const Params& p, Shared* sh) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t* status = p.c.status;
  uint32_t st = 0, st_phase = 0, p_phase = 0, opened = 0;  // by unit: parity of its last arrival, whether there was one
  auto next = [&]() {
    if (!wait(&sh->kv_full[st], st_phase, status)) return false;
    if (lane == 0) arrive(&sh->kv_empty[st]);  // seen: the ring cannot run two phases ahead
    __syncwarp();
    if (++st == C::kStages) st = 0, st_phase ^= 1;
    return true;
  };
  auto open = [&](int u) {  // one arrival a phase: the one before is complete
    if ((opened >> u) & 1)
      if (!wait(&sh->p_full[u], ((p_phase >> u) & 1) ^ 1, status)) return false;
    opened |= 1u << u;
    p_phase ^= 1u << u;
    if (lane == 0) arrive(&sh->p_full[u]);
    __syncwarp();
    return true;
  };
  for (int it = 0;; ++it) {
    const Part* part = take_part(sh, it, status);
    if (!part) return;
    const int n = part->t1 - part->t0;
    const bool both = part->both;
    give_part(sh, it);
    if (!next()) return;
    if (!both && n > 1 && !next()) return;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      if (!next()) return;
      if (j + (both ? 1 : 2) < n && !next()) return;
      if (both ? !(open(0) && open(1)) : !open(j & 1)) return;
    }
  }
}

// --------------------------------------------------------------------------
// Softmax
// --------------------------------------------------------------------------
// lo + hi of the pair w, added to two sums.
template <bool BF16>
__device__ __forceinline__ void add_pair(uint32_t w, float& lo, float& hi) {
  if (BF16)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.f32.bf16 %0, a, %0;\n\tadd.f32.bf16 %1, b, %1;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.f32.f16 %0, a, %0;\n\tadd.f32.f16 %1, b, %1;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "r"(w));
}

// 16 scores to weights: p = 2^(s a + off), packed; their sum, as rounded: what a
// large weight's rounding adds to the output it then takes off again (outputs are 1.2 to
// 1.35 times a rounding away from 64 bits, 1.4 to 1.5 with a sum of unrounded
// weights). a2, off2: each twice.
template <bool BF16>
__device__ __forceinline__ float to_weights(const uint32_t* s, uint64_t a2, uint64_t off2, uint32_t* p) {
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x, y;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), a2, off2), x, y);
    p[i] = pack2<BF16>(exp2_fast(x), exp2_fast(y));
    add_pair<BF16>(p[i], lo, hi);
  }
  return lo + hi;
}

// The reference of a row's exponentials: it moves only when a score (by its
// page's factor, in units of log 2) passes it by 8, so that few tiles scale O.
// Each row goes by its own scores. A weight is 2^(s a + log2 f - m), one multiply-add.
// m lies 6 below the score that set it: weights with f stay below 2^15, and in fp16
// those 2^-20 of it (2^-19 where f is below 1) above the type's subnormal numbers. Past 2^20 m's own
// rounding would be a factor without limit: such a row (`far`) rounds its scaled scores and
// subtracts the score itself, which is exact near the largest ones.
template <int D>
struct Reference {
  static constexpr float kLift = 6.0f;
  float m;       // far: the score, else what is subtracted
  bool far, any_far;

  __device__ __forceinline__ void reset() { m = -INFINITY, far = any_far = false; }
  __device__ __forceinline__ float lift() const { return far ? kLift : 0.0f; }
  // true where a row of the warp moved
  __device__ __forceinline__ bool raise(float top, float& l, uint32_t tO, bool o) {
    const bool up = top - m > 8.0f + (far ? 0.0f : kLift);
    if (!__any_sync(kFull, up)) return false;
    float f = 1.0f;
    if (up) {
      const float was = m, was_lift = lift();
      far = !(fabsf(top) <= kFar);
      m = far ? top : top - kLift;
      f = exp2_fast((was - m) - (was_lift - lift()));
    }
    any_far = __any_sync(kFull, far);
    l *= f;
    if (!o) return true;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t x[32];
      t5::ld32(tO + c, x);
      t5::wait_ld32(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
      t5::st32(tO + c, x);
    }
    return true;
  }
  // what is added to the scaled scores of a group, but for its log2 f
  __device__ __forceinline__ float off() const { return far ? kLift : m == -INFINITY ? 0.0f : -m; }
  // 16 scores of a far row: scaled, less the reference. Factor: what is left for to_weights.
  __device__ __forceinline__ void settle(uint32_t* s, float a) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = far ? __float_as_uint(__fmul_rn(__uint_as_float(s[i]), a) - m) : s[i];
  }
};

// The factors of 32 keys, in pairs, read here and not earlier (the compiler would
// keep all groups' in registers, and the scores out of them).
struct Factors {
  uint64_t a[2], lg[2];
  float inv[2];
  __device__ __forceinline__ Factors(const Info& info, int c) {
    two(&info.a[2 * c], a);
    two(&info.lg[2 * c], lg);
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(inv[0]), "=f"(inv[1]) : "r"(smem_u32(&info.inv[2 * c])));
  }
  static __device__ __forceinline__ void two(const float2* from, uint64_t (&to)[2]) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(to[0]), "=l"(to[1]) : "r"(smem_u32(from)));
  }
};

// What row r of a unit is: its token of the block, its head of the unit.
struct RowOf {
  int token, head;
  bool live;
  __device__ __forceinline__ RowOf(const Params& p, const Part& y, int unit, int r) {
    asm volatile("" : "+r"(r));
    const int tok = r / p.unit_heads;
    head = r - tok * p.unit_heads;
    token = (y.both ? unit * p.unit_tokens : 0) + tok;
    live = tok < p.unit_tokens && head < y.heads && token < y.tokens;
  }
};

template <int D, bool BF16>
__device__ __forceinline__ void softmax_role(const Params& p, Shared* sh, const int unit) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, r = warp * 32 + lane;
  uint32_t* status = p.c.status;
  const uint32_t lanes = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t tS = lanes + unit * 128, tP = tS + 64, tO = lanes + 256 + unit * D, tO_other = lanes + 256 + (1 - unit) * D;
  Reference<D> ref;
  uint32_t phase = 0;  // bits 0: scores, 1, 2: the units' outputs, 3: joins
  int tile = 0;
  for (int it = 0;; ++it) {
    const Part* part = take_part(sh, it, status);
    if (!part) return;
    const Part& y = *part;
    // Keys that the row attends, or none where it is no (token, head) of the
    // block. (What else the row is gets worked out at the end: registers are short here.)
    const RowOf row(p, y, unit, r);
    const int limit = row.live ? y.pos0 + row.token + 1 : kNever;
    const bool warp_live = __any_sync(kFull, limit != kNever);
    ref.reset();
    float l = 0.0f;
    bool any = false;  // a tile of this unit came before
    for (int t = y.t0; t < y.t1; ++t, ++tile) {
      const int slot = tile % kInfo;
      if (!wait(&sh->info_full[slot], (tile / kInfo) & 1, status)) return;
      if (y.mine(unit, t)) {
        if (!wait(&sh->s_full[unit], phase & 1, status)) return;
        phase ^= 1;
        t5::fence_after();
        const Info& info = sh->info[slot];
        const int seen = limit - t * kRows;  // keys of the tile that the row attends
        if (!warp_live) {
          // nothing reads these rows' weights
        } else {
          uint64_t off2;
          // 32 scores to weights. P takes the upper half of the scores' place: of the
          // keys in descending order, a group's weights lie where scores already read were.
          // (In bf16 weights, of 8 bits, only those of a tile whose values fp16 does not
          // hold: open rows, scales out of its range.)
          const bool half = !BF16 || info.half != 0;
          auto weights32 = [&](uint32_t* x, int c, Factors& f) {
            uint32_t w[16];
#pragma unroll
            for (int g = 0; g < 2; ++g)
              l = fmaf(to_weights<false>(x + 16 * g, f.a[g], f2_add(off2, f.lg[g]), w + 8 * g), f.inv[g], l);
            if (c > 0) f = Factors(info, c - 1);  // the next group's, on their way meanwhile
            t5::st16(tP + 16 * c, w);
          };
          // The same for rows that do not see all keys, far ones, and bf16 weights; keys
          // from `none` on no row attends.
          auto slow = [&](uint32_t* x, int none) {
            const float off = ref.off();
#pragma unroll 1
            for (int c = 3; c >= 0; --c) {
              uint32_t w[16];
              if (32 * c >= none) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0u;
                t5::st16(tP + 16 * c, w);
                continue;
              }
              t5::ld32(tS + 32 * c, x);
              t5::wait_ld32(x);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const int k = 2 * c + g;
                if (ref.any_far) ref.settle(x + 16 * g, info.a[k].x);
                const float a = ref.far ? 1.0f : info.a[k].x, lg = info.lg[k].x;
#pragma unroll
                for (int i = 0; i < 16; ++i)  // masked after the factor: -inf * 0 is NaN
                  x[16 * g + i] = 32 * c + 16 * g + i >= seen ? 0xff800000u
                                                              : __float_as_uint(fmaf(__uint_as_float(x[16 * g + i]), a, off + lg));
                const uint64_t one = f2_pack(1.0f, 1.0f), zero = f2_pack(0.0f, 0.0f);
                const float part = half ? to_weights<false>(x + 16 * g, one, zero, w + 8 * g)
                                        : to_weights<BF16>(x + 16 * g, one, zero, w + 8 * g);
                l = fmaf(part, info.inv[k], l);
              }
              t5::st16(tP + 16 * c, w);
            }
          };
          auto reference = [&]() {
            const float off = ref.off();
            off2 = f2_pack(off, off);
          };
          if (__all_sync(kFull, seen >= kRows)) {
            // The lower half of the scores is read twice: for the maximum, and again
            // once the upper half's registers are free.
            uint32_t s[64];
            float top;
            {
              uint32_t lo[64];
              t5::ld32(tS, lo);
              t5::ld32(tS + 32, lo + 32);
              t5::ld32(tS + 64, s);
              t5::wait_ld32(lo);
              t5::wait_ld32(lo + 32);
              t5::wait_ld32(s);
              top = fmaxf(max_of<16>(lo) * info.a[0].x, max_of<16>(lo + 16) * info.a[1].x);
              t5::ld32(tS + 96, s + 32);
              top = fmaxf(top, fmaxf(max_of<16>(lo + 32) * info.a[2].x, max_of<16>(lo + 48) * info.a[3].x));
            }
            top = fmaxf(top, fmaxf(max_of<16>(s) * info.a[4].x, max_of<16>(s + 16) * info.a[5].x));
            t5::wait_ld32(s + 32);
            top = fmaxf(top, fmaxf(max_of<16>(s + 32) * info.a[6].x, max_of<16>(s + 48) * info.a[7].x));
            // (s_full came after the unit's last PV.) Read again after a rescale of
            // O: held over it, the scores' registers would push others out of every tile.
            if (ref.raise(limit != kNever ? top : -INFINITY, l, tO, any)) {
              t5::ld32(tS + 64, s);
              t5::ld32(tS + 96, s + 32);
              t5::wait_ld32(s);
              t5::wait_ld32(s + 32);
            }
            reference();
            if (!ref.any_far && half) {
              uint32_t a[32];
              Factors f(info, 3);
              weights32(s + 32, 3, f);
              t5::ld32(tS + 32, a);
              weights32(s, 2, f);
              t5::wait_ld32(a);
              t5::ld32(tS, s);
              weights32(a, 1, f);
              t5::wait_ld32(s);
              weights32(s, 0, f);
            } else {
              slow(s, kRows);
            }
          } else {
            // a tile that ends past some row's own key; keys from `none` on no row attends
            const int none = __reduce_max_sync(kFull, limit != kNever ? seen : 0);
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4 && 32 * c < none; ++c) {
              uint32_t s[32];
              t5::ld32(tS + 32 * c, s);
              t5::wait_ld32(s);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= seen) s[i] = 0xff800000u;
#pragma unroll
              for (int g = 0; g < 2; ++g) top = fmaxf(top, max_of<16>(s + 16 * g) * info.a[2 * c + g].x);
            }
            ref.raise(limit != kNever ? top : -INFINITY, l, tO, any);
            uint32_t s[32];
            slow(s, none);
          }
        }
        t5::wait_st();
        t5::fence_before();
        __syncwarp();
        if (lane == 0) arrive(&sh->p_full[unit]);
        any = true;
      }
      __syncwarp();
      if (lane == 0) arrive(&sh->info_empty[slot]);
    }

    const RowOf end(p, y, unit, r);
    const bool live = end.live;
    const int head = end.head, my_token = end.token, pos = y.pos0 + my_token;
    const int par = it & 1;
    if (!wait(&sh->fix_ready[par], (it >> 1) & 1, status)) return;
    const bool fix = sh->any_nonfinite[par] == it + 1;
    // sums by the reference itself
    float top = ref.m;
    l *= ref.far ? exp2_fast(-ref.kLift) : 1.0f;
    float mine = ref.far ? exp2_fast(-ref.kLift) : 1.0f, other = 0.0f;
    if (!y.both) {  // join the units' sums: each thread half of the row's channels
      sh->join[unit][r][0] = top;
      sh->join[unit][r][1] = l;
      sh->join[unit][r][2] = mine;
      // (a unit without a tile has m = -inf and l = 0)
      if (!wait(&sh->o_done[0], (phase >> 1) & 1, status)) return;
      if (y.has(1) && !wait(&sh->o_done[1], (phase >> 2) & 1, status)) return;
      t5::fence_after();
      __syncwarp();
      if (lane == 0) arrive(&sh->join_ready);
      if (!wait(&sh->join_ready, (phase >> 3) & 1, status)) return;
      const float top2 = sh->join[1 - unit][r][0], l2 = sh->join[1 - unit][r][1];
      const float best = fmaxf(top, top2), base = best == -INFINITY ? 0.0f : best;
      const float f1 = exp2_fast(top - base), f2 = exp2_fast(top2 - base);
      l = l * f1 + l2 * f2;
      mine *= f1;
      other = f2 * sh->join[1 - unit][r][2];
      top = best;
    } else if (y.has(unit)) {
      if (!wait(&sh->o_done[unit], (phase >> (1 + unit)) & 1, status)) return;
      t5::fence_after();
    }
    phase ^= y.has(1) ? 6 : 2;

    const bool wide = (reinterpret_cast<uintptr_t>(p.a.out) & 31) == 0;
    const bool wide_part = (reinterpret_cast<uintptr_t>(p.part_o) & 31) == 0;
    const int c0 = y.both ? 0 : unit * (D / 2), c1 = y.both ? D : c0 + D / 2;
    const bool own = y.both || y.has(unit), both_o = !y.both && y.has(1);
    const float scale = y.slot < 0 ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
    const int part_row = y.slot < 0 ? 0 : ((blockIdx.x * 2 + y.slot) * 2 + (y.both ? unit : 0)) * kRows + r;
    if (warp_live) {
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t o[32];
        if (own) {
          t5::ld32(tO + c, o);
          t5::wait_ld32(o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = own ? __float_as_uint(__uint_as_float(o[i]) * mine) : 0u;
        if (!y.both && (unit == 1 || both_o)) {
          uint32_t o2[32];
          t5::ld32(tO_other + c, o2);
          t5::wait_ld32(o2);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(fmaf(__uint_as_float(o2[i]), other, __uint_as_float(o[i])));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale);
        if (fix) {
          const unsigned long long key = first_key(it, pos);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x = __uint_as_float(o[i]);
            if (key >= sh->first[par][1][c + i]) x += INFINITY;
            if (key >= sh->first[par][2][c + i]) x -= INFINITY;
            if (key >= sh->first[par][0][c + i]) x = NAN;
            o[i] = __float_as_uint(x);
          }
        }
        if (live && y.slot < 0) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack2<BF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          store_row(p.a.out + ((int64_t)(y.c0 + my_token) * p.a.q_heads + y.hq0 + head) * D + c, w, wide);
        } else if (live) {
          uint16_t* to = reinterpret_cast<uint16_t*>(p.part_o + (int64_t)part_row * D + c);
          store_row(to, o, wide_part);
          store_row(to + 32, o + 16, wide_part);
        }
      }
      if (live && y.slot >= 0 && (y.both || unit == 0))
        *reinterpret_cast<float2*>(p.part_ml + (int64_t)part_row * 2) = make_float2(top, l);
    }
    if (!y.both) {
      t5::fence_before();
      __syncwarp();
      if (lane == 0) arrive(&sh->join_done);
      if (!wait(&sh->join_done, (phase >> 3) & 1, status)) return;
      phase ^= 8;
    }
    t5::fence_before();  // O has been read: ordered before the next part's first weights
    __syncwarp();
    if (lane == 0) arrive(&sh->fix_free[par]);
    give_part(sh, it);
  }
}

// --------------------------------------------------------------------------
// The kernel
// --------------------------------------------------------------------------
// Where the CTA's range starts and ends: sums of the requests' places over the block.
__device__ __forceinline__ void find_range(const Params& p, Shared* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = p.a.requests;
  const int per = (R + kThreads - 1) / kThreads;
  long long sum = 0;
  bool bad = false;
  for (int k = 0; k < per; ++k) {
    const int b = threadIdx.x * per + k;
    if (b >= R) break;
    const Req r = load_req(p, b, bad);
    if (r.m > 0) sum += Blocks(p, r).all() * p.lots;
  }
  if (bad && blockIdx.x == 0) raise_status(p.c.status, kStatusBadIndex);
  long long in = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(kFull, in, d);
    if (lane >= d) in += u;
  }
  if (lane == 31) sh->scan[warp] = in;
  if (threadIdx.x == 0) {
    const Pos end = {R, 0, 0, 0};
    sh->from = sh->to = end;
  }
  __syncthreads();
  long long at = in - sum, places = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += sh->scan[w];
    places += sh->scan[w];
  }
  const int ctas = places < p.ctas ? (int)places : p.ctas;
  if ((int)blockIdx.x >= ctas) return;
  const long long share = quotient(places, ctas), rest = places - share * ctas;  // rest < ctas
  const long long v[2] = {share * blockIdx.x + (uint32_t)rest * blockIdx.x / (uint32_t)ctas,
                          share * (blockIdx.x + 1) + (uint32_t)rest * (blockIdx.x + 1) / (uint32_t)ctas};
  for (int e = 0; e < 2; ++e) {
    if (v[e] < at || v[e] >= at + sum) continue;
    long long a = at;
    for (int k = 0; k < per; ++k) {
      const int b = threadIdx.x * per + k;
      if (b >= R) break;
      const Req r = load_req(p, b, bad);
      const long long size = r.m > 0 ? Blocks(p, r).all() * p.lots : 0;
      if (v[e] < a + size) {
        (e ? sh->to : sh->from) = locate(p, b, r, v[e] - a);
        break;
      }
      a += size;
    }
  }
}

template <int D, int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sh;
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    prefetch_map(&p.mq);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 5);  // the unit's warps, and the gate
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.fix_ready[i], 8);
      mbar_init(&sh.fix_free[i], 8);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sh.part_full[i], 1);
      mbar_init(&sh.part_empty[i], 19);  // every warp but the one that fills it
    }
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.join_ready, 8);
    mbar_init(&sh.join_done, 8);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.kv_full[i], 8);
      mbar_init(&sh.kv_empty[i], 2);  // the products have read it, the gate has seen it
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 8);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&sh.info_full[i], 1);
      mbar_init(&sh.info_empty[i], 16);
    }
    mbar_fence_init();
    sh.any_nonfinite[0] = sh.any_nonfinite[1] = 0;
  }
  for (int k = threadIdx.x; k < 2 * 3 * 128; k += kThreads) (&sh.first[0][0][0])[k] = ~0ull;
  find_range(p, &sh);
  if (warp == 9) t5::alloc(&sh.tmem, 512);
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  if (threadIdx.x == 0) {
    p.pos[blockIdx.x] = make_int4(sh.from.b, sh.from.lot, sh.from.i, sh.from.t);
    if (blockIdx.x == gridDim.x - 1) p.pos[gridDim.x] = make_int4(p.a.requests, 0, 0, 0);
  }

  // 256 threads x 152 + 128 x 48 + 256 x 64 registers = 640 x 96, what the launch holds
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    softmax_role<D, BF16>(p, &sh, warp >> 2);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 8) part_role<D>(p, &sh, smem);
    else if (warp == 9) mma_role<D, BF16>(p, &sh, smem);
    else if (warp == 10) tile_role<D, CODE, BF16>(p, &sh, smem + (2 + C::kStages) * C::kTile);
    else gate_role<D>(p, &sh);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    unsigned char* ring = smem + 2 * C::kTile;
    convert_role<D, CODE, BF16>(p, &sh, ring, ring + C::kStages * C::kTile);
  }
  __syncwarp();
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  if (warp == 9) t5::dealloc(sh.tmem, 512);
}

// Merges the partial sums of the blocks that a range's end cuts, in the order of
// the CTAs. CTA x: the block that range x + 1 starts inside, if no earlier range
// does; y: which of its units' rows. A warp takes four rows side by side.
constexpr int kMergeThreads = 1024;

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) paged_attn_merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = D / 32, kSide = kRows / 32;
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, unit = blockIdx.y;
  // where ranges c - 1 + lane start: these first, all at once
  const int4 none = make_int4(p.a.requests, 0, 0, 0);
  int4 mine = c - 1 + lane <= p.ctas ? p.pos[c - 1 + lane] : none;
  auto pos_of = [&](int k) {
    return make_int4(__shfl_sync(kFull, mine.x, k), __shfl_sync(kFull, mine.y, k), __shfl_sync(kFull, mine.z, k),
                     __shfl_sync(kFull, mine.w, k));
  };
  const int4 prev = pos_of(0), at = pos_of(1);
  if (at.w == 0) return;
  auto same = [&](const int4& x) { return x.x == at.x && x.y == at.y && x.z == at.z; };
  if (same(prev) && prev.w > 0) return;
  bool bad = false;
  const Req r = load_req(p, at.x, bad);
  const Blocks k(p, r);
  const int chunk = at.y % p.chunks, hq0 = at.y / p.chunks * p.a.group + chunk * kRows;
  const int heads = min(p.unit_heads, p.a.group - chunk * kRows);
  const long long first = (long long)at.z * k.bt;
  const int tokens = (int)min((long long)k.bt, r.m - first);
  int token[kSide], head[kSide];
  bool live[kSide], any = false;
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    const int in = warp + 32 * i, tok = in / p.unit_heads;
    head[i] = in - tok * p.unit_heads;
    token[i] = unit * p.unit_tokens + tok;
    live[i] = tok < p.unit_tokens && head[i] < heads && token[i] < tokens;
    any |= live[i];
  }
  if (!any) return;
  float top[kSide], l[kSide], o[kSide][kPer];
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    top[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[i][e] = 0.0f;
  }
  int4 from = prev;
  int base = c - 1;  // the CTA of mine in lane 0
  int x = c - 1;
  uint32_t gone = 0;  // by row: the last part's factor is 0
  for (; x < p.ctas; ++x) {
    if (x + 1 - base == 32) {
      base += 31;
      mine = base + lane <= p.ctas ? p.pos[base + lane] : none;
    }
    const int4 to = pos_of(x + 1 - base);
    const bool inside = same(to) && to.w > 0;  // the block goes on in the next range
    const bool empty = x >= c && inside && to.w == from.w;
    from = to;
    gone = 0;
    if (!empty) {
      float2 ml[kSide];
      float v[kSide][kPer];
#pragma unroll
      for (int i = 0; i < kSide; ++i) {
        const int64_t pr = ((int64_t)(x * 2 + (x >= c ? 0 : 1)) * 2 + unit) * kRows + warp + 32 * i;
        const float* src = p.part_o + pr * D + lane * kPer;
        ml[i] = live[i] ? *reinterpret_cast<const float2*>(p.part_ml + pr * 2) : make_float2(-INFINITY, 0.0f);
        if (D == 128) {
          const float4 w = live[i] ? *reinterpret_cast<const float4*>(src) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          v[i][0] = w.x, v[i][1] = w.y, v[i][2 % kPer] = w.z, v[i][3 % kPer] = w.w;
        } else {
          const float2 w = live[i] ? *reinterpret_cast<const float2*>(src) : make_float2(0.0f, 0.0f);
          v[i][0] = w.x, v[i][1] = w.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kSide; ++i) {
        const float now = fmaxf(top[i], ml[i].x), ref = now == -INFINITY ? 0.0f : now;
        const float fo = exp2_fast(top[i] - ref), fn = exp2_fast(ml[i].x - ref);
        gone |= (fn == 0.0f ? 1u : 0u) << i;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[i][e] = o[i][e] * fo + v[i][e] * fn;
        l[i] = l[i] * fo + ml[i].y * fn;
        top[i] = now;
      }
    }
    if (!inside) break;
  }
  // A factor of 0 is too small for a number, but not for the open page's infinities, which are in the last part.
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    if (!live[i] || !((gone >> i) & 1)) continue;
    const float* src = p.part_o + (((int64_t)(x * 2 + (x >= c ? 0 : 1)) * 2 + unit) * kRows + warp + 32 * i) * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float v = src[e];
      if (!(fabsf(v) < INFINITY)) o[i][e] = v;
    }
  }
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    if (!live[i]) continue;
    const float inv = l[i] == 0.0f ? 1.0f : 1.0f / l[i];  // no weight at all: o is 0, or the open page's
    uint16_t* out = p.a.out + ((int64_t)(r.c0 + first + token[i]) * p.a.q_heads + hq0 + head[i]) * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
      *reinterpret_cast<uint32_t*>(out + e) = pack2<BF16>(o[i][e] * inv, o[i][e + 1] * inv);
  }
}

template <int D, int CODE, bool BF16>
cudaError_t launch(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  Params p;
  p.c = c;
  p.a = a;
  p.ctas = a.sm_count;
  p.unit_heads = a.group < kRows ? a.group : kRows;
  p.chunks = (a.group + kRows - 1) / kRows;
  p.unit_tokens = kRows / p.unit_heads;
  p.lots = c.heads * p.chunks;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  p.pos = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + pos_bytes(p.ctas));
  p.part_o = p.part_ml + (size_t)p.ctas * 4 * kRows * 2;
  cudaError_t e = encode_heads(&p.mq, a.q, D, a.q_heads, a.tokens, a.q_stride, BF16, p.unit_heads, p.unit_tokens);
  if (e != cudaSuccess) return e;
  static SmemAttr attr;
  e = attr.ensure(paged_attn_kernel<D, CODE, BF16>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, CODE, BF16><<<p.ctas, kThreads, Cfg<D>::kSmem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.ctas < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas - 1, 2);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_merge_kernel<D, BF16>, p);
}

template <int D, int CODE>
cudaError_t by_type(const PagedDev& c, const PagedAttnArgs& a, cudaStream_t st) {
  return c.dtype == KVQ_BF16 ? launch<D, CODE, true>(c, a, st) : launch<D, CODE, false>(c, a, st);
}

}  // namespace patt
}  // namespace kvq
