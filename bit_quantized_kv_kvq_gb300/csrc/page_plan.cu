// Planning of a paged step on the GPU: block tables, slot maps and positions
// from request lengths (kvq_paged_reserve), and the return of pages
// (kvq_paged_release).
//
// Request b holds n tokens in ceil(n / P) pages and takes m more: it grows by
// ceil((n + m) / P) - ceil(n / P) pages. Two exclusive prefix sums over the
// requests, of m and of the growth, give every packed token its request and
// position and every new page its place on the free stack, so everything after
// the sums is independent per token and per page.
//
// A decode step reads and writes a few hundred bytes: latency, 4.9 us for
// 16 requests (thirty in a graph). Many packed tokens go over the GPU (8 bytes written a
// token, searched for four at a time): 262144 tokens of 1024 requests 8.1 us,
// 1 us of it to look over the pages first; one cluster of eight CTAs took 20.5 us.
#include "paged_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = kMaxRequests / kThreads;  // requests per thread
// Packed tokens that one CTA plans alone. us alone / in two launches over the
// GPU, 256 requests: 1024 tokens 6.0/6.0, 4096 6.6/6.6, 6144 7.9/6.8, 16384
// 11.6/6.9; 16 requests: 1024 5.1/5.4, 4096 5.7/5.9, 6144 6.7/6.0.
constexpr int kOneLaunch = 4096;

// Exclusive prefix sums of (x, y) over the block; totals in *tx, *ty.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long* tx, long long* ty) {
  __shared__ long long wx[32], wy[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, ix, d), uy = __shfl_up_sync(0xffffffffu, iy, d);
    if (lane >= d) ix += ux, iy += uy;
  }
  if (lane == 31) wx[warp] = ix, wy[warp] = iy;
  __syncthreads();
  if (warp == 0) {
    long long a = wx[lane], b = wy[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long ua = __shfl_up_sync(0xffffffffu, a, d), ub = __shfl_up_sync(0xffffffffu, b, d);
      if (lane >= d) a += ua, b += ub;
    }
    wx[lane] = a, wy[lane] = b;
  }
  __syncthreads();
  x = ix - x + (warp ? wx[warp - 1] : 0);
  y = iy - y + (warp ? wy[warp - 1] : 0);
  *tx = wx[31];
  *ty = wy[31];
}

// The last index b in [0, n) with key[b] <= x (keys ascending, key[0] <= x).
__device__ __forceinline__ int last_le(const int* key, int n, int x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (key[lo + half] <= x) lo += half, n -= half;
    else n = half;
  }
  return lo;
}

// What a reserve kernel does: the new table entries, slots and positions
// (kPlan), the state after the step (kState), or both. Every CTA makes the
// sums for itself (a few thousand lengths at most) and takes its share of the
// tokens and pages. lens_out and free_count_out may be the input arrays: one
// CTA writes them once it has read those; with several, a second launch does,
// after all of the first have ended.
constexpr int kPlan = 1, kState = 2;

template <int WHAT>
__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveArgs a) {
  extern __shared__ int sm[];
  const int R = a.requests;
  int* cu = sm;                // [R + 1] packed token where the request starts
  int* first = sm + R + 1;     // [R + 1] pages taken before the request's
  int* old = sm + 2 * (R + 1); // [R] length before
  __shared__ int bad_s;
  // the second launch makes its own sums meanwhile, and waits before it writes
  if (WHAT == kPlan) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int P = 1 << a.page_shift;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();

  const int free_count = *a.free_count;
  const bool over = free_count < 0 || free_count > a.num_pages;
  // the k-th page from the stack's top, where the stack has one
  auto popped = [&](int k) { return a.free_pages[free_count - 1 - k]; };
  auto in_cache = [&](int page) { return page >= 0 && page < a.num_pages; };
  int n[kPer], m[kPer], g[kPer];
  long long add = 0, grow = 0;
  bool bad = false, full = false, torn = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    n[i] = b < R ? a.lens[b] : 0;
    m[i] = b < R ? a.add[b] : 0;
    bad |= n[i] < 0 || m[i] < 0;
    const long long have = ((long long)n[i] + P - 1) >> a.page_shift;
    const long long need = ((long long)n[i] + m[i] + P - 1) >> a.page_shift;
    full |= need > a.max_pages;
    g[i] = (int)(need - have);
    add += m[i];
    grow += g[i];
    // new tokens go into the open page first
    if (m[i] > 0 && n[i] > 0 && (n[i] & (P - 1)) && have <= a.max_pages)
      torn |= !in_cache(a.table[(int64_t)b * a.max_pages + have - 1]);
  }
  const int flags = (bad || over ? 1 : 0) | (full ? 2 : 0);
  if (flags) atomicOr(&bad_s, flags);
  long long total, pages;
  block_scan2(add, grow, &total, &pages);  // its barriers publish bad_s too
  // The pages that the step takes off the stack are looked over before anything
  // is planned with them: every CTA does so, and all come to the same answer.
  const bool room = bad_s == 0 && total <= a.max_tokens && pages <= free_count;
  if (room) {
    const int count = (int)pages, *lowest = a.free_pages + (free_count - count);
    const int head = min(count, (int)(-reinterpret_cast<uintptr_t>(lowest) & 15) >> 2);  // up to a 16-byte border
    const int wide = (count - head) >> 2, rest = head + 4 * wide;
    const int at = threadIdx.x;
    if (at < head) torn |= !in_cache(lowest[at]);
    if (at < count - rest) torn |= !in_cache(lowest[rest + at]);
#pragma unroll 4
    for (int i = at; i < wide; i += kThreads) {
      const int4 x = reinterpret_cast<const int4*>(lowest + head)[i];
      torn |= !(in_cache(x.x) && in_cache(x.y) && in_cache(x.z) && in_cache(x.w));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = threadIdx.x * kPer + i;
      if (b < R) cu[b] = (int)add, first[b] = (int)grow, old[b] = n[i];
      add += m[i];
      grow += g[i];
      if (b == R - 1) cu[R] = (int)add, first[R] = (int)grow;
    }
  }
  const bool bad_page = __syncthreads_or(torn);
  const bool fits = room && !bad_page;
  if (WHAT == kState) asm volatile("griddepcontrol.wait;" ::: "memory");

  const int at0 = blockIdx.x * kThreads + threadIdx.x, stride = gridDim.x * kThreads;
  if (!fits) {
    for (int64_t i = at0; (WHAT & kPlan) && i < a.max_tokens; i += stride) a.slots[i] = -1, a.positions[i] = -1;
    if (WHAT & kState) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = threadIdx.x * kPer + i;
        if (b < R) a.lens_out[b] = n[i];
      }
      for (int b = threadIdx.x; b <= R; b += kThreads) a.cu[b] = 0;
      if (threadIdx.x == 0) {
        *a.free_count_out = free_count;
        raise_status(a.status, (bad_s & 1) || bad_page ? kStatusBadIndex : kStatusNoRoom);
      }
    }
    return;
  }
  if (WHAT & kState) {
    for (int b = threadIdx.x; b <= R; b += kThreads) {
      a.cu[b] = cu[b];
      if (b < R) a.lens_out[b] = old[b] + (cu[b + 1] - cu[b]);
    }
    if (threadIdx.x == 0) *a.free_count_out = free_count - (int)pages;
  }
  if (!(WHAT & kPlan)) return;
  for (int k = at0; k < (int)pages; k += stride) {
    const int b = last_le(first, R + 1, k);
    const int j = ((old[b] + P - 1) >> a.page_shift) + (k - first[b]);
    a.table[(int64_t)b * a.max_pages + j] = popped(k);
  }
  // four packed tokens a step: one search, then on from request to request
  const bool vec = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  for (int64_t at = 4 * at0; at < a.max_tokens; at += 4 * stride) {
    const int i0 = (int)at;
    int slot[4], pos[4];
    int b = i0 < (int)total ? last_le(cu, R + 1, i0) : R;
    int page = 0, page_index = -1;  // of request b, the last one looked up
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      slot[k] = pos[k] = -1;
      if (at + k >= total) continue;
      const int i = i0 + k;
      while (cu[b + 1] <= i) ++b, page_index = -1;
      const int p = old[b] + (i - cu[b]), j = p >> a.page_shift;
      if (j != page_index) {
        const int have = (old[b] + P - 1) >> a.page_shift;
        page = j < have ? a.table[(int64_t)b * a.max_pages + j] : popped(first[b] + j - have);
        page_index = j;
      }
      pos[k] = p;
      slot[k] = (page << a.page_shift) + (p & (P - 1));
    }
    if (vec && at + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int k = 0; k < 4 && at + k < a.max_tokens; ++k) a.slots[i0 + k] = slot[k], a.positions[i0 + k] = pos[k];
    }
  }
}

// One CTA: requests end a few at a time. 797 pages take 3 us, and where many
// requests end at once its rounds of dependent loads show: 196615 pages 143 us.
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
  __shared__ int first[kMaxRequests + 1];
  const int R = a.requests;
  const int P = 1 << a.page_shift;
  int count = *a.free_count;
  long long mine = 0, unused = 0;
  int g[kPer];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    g[i] = 0;
    if (b < R && a.done[b] != 0) {
      const int n = a.lens[b];
      const long long pages = ((long long)n + P - 1) >> a.page_shift;
      if (n < 0 || pages > a.max_pages) bad = true;
      else g[i] = (int)pages;
    }
    mine += g[i];
  }
  if (count < 0 || count > a.num_pages) bad = true;
  long long total;
  block_scan2(mine, unused, &total, &unused);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    if (b < R) first[b] = (int)(mine < INT32_MAX ? mine : INT32_MAX);
    mine += g[i];
    if (b == R - 1) first[R] = (int)(mine < INT32_MAX ? mine : INT32_MAX);
  }
  if (bad) raise_status(a.status, kStatusBadIndex);
  __syncthreads();
  if (count < 0 || count > a.num_pages) return;  // the stack is not touched
  const long long room = a.num_pages - count;
  if (total > room) {
    if (threadIdx.x == 0) raise_status(a.status, kStatusBadIndex);
    total = room;
  }
  for (int k = threadIdx.x; k < (int)total; k += kThreads) {
    const int b = last_le(first, R + 1, k);
    const int page = a.table[(int64_t)b * a.max_pages + (k - first[b])];
    // an entry out of range keeps its place on the stack, where reserve refuses it
    if (page < 0 || page >= a.num_pages) raise_status(a.status, kStatusBadIndex);
    a.free_pages[count + k] = page;
  }
  for (int b = threadIdx.x; b < R; b += kThreads)
    if (a.done[b] != 0) a.lens[b] = 0;
  if (threadIdx.x == 0) *a.free_count = count + (int)total;
}

}  // namespace

int reserve_launches(int max_tokens) { return max_tokens <= kOneLaunch ? 1 : 2; }

cudaError_t launch_reserve(const ReserveArgs& a, cudaStream_t st) {
  static SmemAttr one, plan, state;
  const size_t smem = (size_t)(3 * a.requests + 2) * 4, most = (3 * kMaxRequests + 2) * 4;
  if (a.max_tokens <= kOneLaunch) {
    const cudaError_t e = one.ensure(reserve_kernel<kPlan | kState>, most);
    if (e != cudaSuccess) return e;
    reserve_kernel<kPlan | kState><<<1, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  cudaError_t e = plan.ensure(reserve_kernel<kPlan>, most);
  if (e == cudaSuccess) e = state.ensure(reserve_kernel<kState>, most);
  if (e != cudaSuccess) return e;
  const int64_t ctas = ((int64_t)a.max_tokens + 4 * kThreads - 1) / (4 * kThreads);
  reserve_kernel<kPlan><<<(unsigned)(ctas < 128 ? ctas : 128), kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reserve_kernel<kState>, a);
}

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t st) {
  release_kernel<<<1, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
