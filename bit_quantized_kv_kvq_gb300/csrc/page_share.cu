// Requests that share pages: forks (kvq_paged_fork) and the release of pages
// that others may hold (kvq_paged_release_shared).
//
// shared[p] counts the holders of page p beyond the first, so pages on the stack and
// of single requests are 0 and planning knows nothing of it. A complete page
// never changes and can be named by several rows; the open page's rows are in the
// request's tail, so a fork copies those rows and takes a page of its own.
//
// 60 forks in 8 layers of 8 heads of 128 (116 MB read and written): 22 us, 0.8 of the copy rate. Release
// of 184000 entries 52 us (sixteen CTAs, eight entries a thread side by side; eight CTAs, one
// by one, 134 us): scattered counts from sixteen SMs. Release of 464 entries 4 us, latency.
#include <cooperative_groups.h>

#include <atomic>

#include "paged_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kPer = kMaxRequests / kThreads;  // requests or pairs per thread

// Exclusive prefix sum over the block; the total in *all.
__device__ __forceinline__ long long block_scan(long long x, long long* all) {
  __shared__ long long w[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long in = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, in, d);
    if (lane >= d) in += u;
  }
  if (lane == 31) w[warp] = in;
  __syncthreads();
  if (warp == 0) {
    long long a = w[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, a, d);
      if (lane >= d) a += u;
    }
    w[lane] = a;
  }
  __syncthreads();
  const long long r = in - x + (warp ? w[warp - 1] : 0);
  *all = w[31];
  __syncthreads();  // w may be written again
  return r;
}

// --------------------------------------------------------------------------
// Fork
// --------------------------------------------------------------------------
// A fork's kernels do its copies (kCopy), the state after it (kState), or
// both. As in the planning, every CTA looks all pairs over for itself and comes to
// the same answer, and the state, which that reads, is written by the one CTA
// that is alone, or by a second launch after the first has ended.
constexpr int kCopy = 1, kState = 2;
constexpr int kEntries = 256;      // table entries of a unit of work
constexpr int kTailBytes = 4096;   // bytes of a tail slab of a unit of work
// Room of the pairs' tails, in bytes, up to which one CTA copies alone. us alone / by two launches:
// 16 KB 4.5/5.4, 64 KB 5.1/6.3, 128 KB 6.8/7.6, 256 KB 9.1/7.6, 1 MB 22/7.6.
constexpr int64_t kOneLaunchBytes = 128 << 10;

template <int WHAT>
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a) {
  extern __shared__ int sm[];
  const int N = a.pairs, P = 1 << a.page_shift;
  int* len = sm;      // [N] tokens of pair i's source, -1: no pair
  int* pop = sm + N;  // [N] pages that the pairs before take
  __shared__ uint32_t seen[kMaxRequests / 32];
  if (WHAT == kCopy) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < kMaxRequests / 32; i += kThreads) seen[i] = 0;
  __syncthreads();
  const int free_count = *a.free_count;
  bool bad = free_count < 0 || free_count > a.num_pages;
  int n[kPer];
  long long pops = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x * kPer + k;
    n[k] = -1;
    if (i >= N) continue;
    const int s = a.src[i], d = a.dst[i];
    if (s < 0) continue;
    if (s >= a.requests || d < 0 || d >= a.requests || s == d) {
      bad = true;
      continue;
    }
    n[k] = a.lens[s];
    bad |= n[k] < 0 || n[k] > (int64_t)a.max_pages << a.page_shift || a.lens[d] != 0;
    bad |= (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1;
    pops += (n[k] & (P - 1)) != 0;
  }
  long long total;
  const long long before = block_scan(pops, &total);
  const bool refused = __syncthreads_or(bad);
  const bool room = total <= free_count;
  long long at = before;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x * kPer + k;
    if (i >= N) continue;
    len[i] = n[k];
    pop[i] = (int)at;
    at += n[k] >= 0 && (n[k] & (P - 1)) != 0;
  }
  bool torn = false;
  if (!refused && room)
    for (int k = threadIdx.x; k < (int)total; k += kThreads) {
      const int page = a.free_pages[free_count - 1 - k];
      torn |= page < 0 || page >= a.num_pages;
    }
  const bool bad_page = __syncthreads_or(torn);  // also: len and pop are there
  const bool go = !refused && room && !bad_page;

  if ((WHAT & kCopy) && go) {
    const int warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kThreads / 32);
    const int lane = threadIdx.x & 31;
    // table rows
    const int row_units = (a.max_pages + kEntries - 1) / kEntries;
    const int64_t table_units = (int64_t)N * row_units;
    for (int64_t u = warp; u < table_units; u += warps) {
      const int i = (int)(u / row_units), j0 = (int)(u % row_units) * kEntries;
      const int full = len[i] >> a.page_shift;  // -1 >> s is -1
      const bool open = len[i] >= 0 && (len[i] & (P - 1)) != 0;
      if (j0 >= full + open) continue;
      const int32_t* from = a.table + (int64_t)a.src[i] * a.max_pages;
      int32_t* to = a.table + (int64_t)a.dst[i] * a.max_pages;
      int page[kEntries / 32];
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) {
        const int j = j0 + 32 * k + lane;
        page[k] = j < full ? from[j] : 0;
      }
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) {
        const int j = j0 + 32 * k + lane;
        if (j < full) {
          to[j] = page[k];
          if (page[k] >= 0 && page[k] < a.num_pages) atomicAdd(a.shared + page[k], 1);
          else raise_status(a.status, kStatusBadIndex);
        } else if (j == full && open) {
          to[j] = a.free_pages[free_count - 1 - pop[i]];
        }
      }
    }
    // open rows, layer by layer
    const int slab = a.row_bytes << a.page_shift;
    const int chunks = (slab + kTailBytes - 1) / kTailBytes;
    const int64_t per_pair = (int64_t)a.layers * a.slabs * chunks, tail_units = N * per_pair;
    for (int64_t u = warp; u < tail_units; u += warps) {
      const int i = (int)(u / per_pair);
      const int bytes = len[i] < 0 ? 0 : (len[i] & (P - 1)) * a.row_bytes;
      int64_t rest = u % per_pair;
      const int c0 = (int)(rest % chunks) * kTailBytes;
      if (c0 >= bytes) continue;
      rest /= chunks;
      unsigned char* layer = a.tails + (rest / a.slabs) * a.layer_bytes;
      const int which = (int)(rest % a.slabs);
      const unsigned char* from = layer + ((int64_t)a.src[i] * a.slabs + which) * slab + c0;
      unsigned char* to = layer + ((int64_t)a.dst[i] * a.slabs + which) * slab + c0;
      const int m = min(bytes - c0, kTailBytes) / 16;
      uint4 x[kTailBytes / 512];
#pragma unroll
      for (int k = 0; k < kTailBytes / 512; ++k)
        if (32 * k + lane < m) x[k] = reinterpret_cast<const uint4*>(from)[32 * k + lane];
#pragma unroll
      for (int k = 0; k < kTailBytes / 512; ++k)
        if (32 * k + lane < m) reinterpret_cast<uint4*>(to)[32 * k + lane] = x[k];
    }
  }
  if (!(WHAT & kState)) return;
  if (WHAT == kState) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!go) {
    if (threadIdx.x == 0) raise_status(a.status, refused || bad_page ? kStatusBadIndex : kStatusNoRoom);
    return;
  }
  for (int i = threadIdx.x; i < N; i += kThreads)
    if (len[i] >= 0) a.lens[a.dst[i]] = len[i];
  if (threadIdx.x == 0) *a.free_count = free_count - (int)total;
}

// --------------------------------------------------------------------------
// Release
// --------------------------------------------------------------------------
constexpr int kCluster = 16;  // CTAs of the large form
constexpr int kRun = 8;       // and consecutive entries of its threads
// Table entries (of all rows) up to which one CTA releases alone. us alone / by the cluster:
// 456 entries 4.0/8.2, 2048 8.0/9.2, 4032 15.6/10.1, 8000 28/10.1, 32000 111/14.
constexpr int64_t kAlone = 2048;

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

// The released entries, numbered in order of request and position, are cut into a
// run for each CTA of a cluster; three passes over them with a barrier between: every
// entry takes one off its page's count; of the entries whose page's count went below
// zero, the last one leaves its number there (smaller numbers than any count); and
// that entry puts the page on the stack, at the place that a prefix sum over such
// entries gives. A thread takes RUN entries side by side, so that their loads
// and counts are on their way together, and keeps the pages of its first ones.
template <int CTAS, int RUN>
__global__ void __launch_bounds__(kThreads) release_shared_kernel(const ReleaseSharedArgs args) {
  const ReleaseArgs& a = args.r;
  __shared__ int first[kMaxRequests + 1];
  __shared__ int pushes, base_s;
  const int R = a.requests, P = 1 << a.page_shift, rank = blockIdx.x;
  auto sync = [&]() {
    if (CTAS > 1) cg::this_cluster().sync();
    else __syncthreads();
  };
  const int count = *a.free_count;
  int g[kPer];
  bool bad = count < 0 || count > a.num_pages;
  const bool no_stack = bad;
  long long mine = 0, total;
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
  long long at = block_scan(mine, &total);
  const bool refused = no_stack || total >= 1 << 30;
  if (bad || refused) raise_status(a.status, kStatusBadIndex);
  if (refused) return;  // the whole cluster: all its CTAs see the same
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    if (b < R) first[b] = (int)at;
    at += g[i];
    if (b == R - 1) first[R] = (int)at;
  }
  __syncthreads();
  // runs of whole groups of RUN entries
  const int groups = ((int)total + RUN - 1) / RUN, per = (groups + CTAS - 1) / CTAS;
  const int g0 = min(rank * per, groups), g1 = min(g0 + per, groups);
  // the pages of group q, -1 where there is none or no such page
  auto look_up = [&](int q, int (&page)[RUN], bool raise) {
    int b = q < g1 ? last_le(first, R + 1, q * RUN) : R;
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      page[k] = -1;
      const int e = q * RUN + k;
      if (q >= g1 || e >= (int)total) continue;
      while (first[b + 1] <= e) ++b;
      page[k] = a.table[(int64_t)b * a.max_pages + (e - first[b])];
    }
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      if (q >= g1 || q * RUN + k >= (int)total) continue;
      if (page[k] < 0 || page[k] >= a.num_pages) {
        page[k] = -1;
        if (raise) raise_status(a.status, kStatusBadIndex);
      }
    }
  };
  int kept[RUN];  // of the thread's first group
  look_up(g0 + threadIdx.x, kept, true);
  auto pages_of = [&](int q, int (&page)[RUN], bool raise) {
    if (q != g0 + (int)threadIdx.x) return look_up(q, page, raise);
#pragma unroll
    for (int k = 0; k < RUN; ++k) page[k] = kept[k];
  };
  auto number = [](int k) { return INT32_MIN + ((1 << 30) - k); };  // later entries: lower, all below any count
  for (int q = g0 + threadIdx.x; q < g1; q += kThreads) {
    int page[RUN];
    pages_of(q, page, true);
#pragma unroll
    for (int k = 0; k < RUN; ++k)
      if (page[k] >= 0) atomicAdd(args.shared + page[k], -1);
  }
  sync();
  for (int q = g0 + threadIdx.x; q < g1; q += kThreads) {
    int page[RUN], held[RUN];
    pages_of(q, page, false);
#pragma unroll
    for (int k = 0; k < RUN; ++k) held[k] = page[k] >= 0 ? __ldcg(args.shared + page[k]) : 0;
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      if (held[k] >= 0) continue;
      // released more often than held (who comes first sees it: others may see a number)
      if (held[k] < -1 && held[k] > INT32_MIN + (1 << 30)) raise_status(a.status, kStatusBadIndex);
      atomicMin(args.shared + page[k], number(q * RUN + k));
    }
  }
  sync();
  // which of group q's entries are their page's last: bits, and the pages
  auto last_of = [&](int q, int (&page)[RUN]) {
    pages_of(q, page, false);
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < RUN; ++k)
      if (page[k] >= 0 && __ldcg(args.shared + page[k]) == number(q * RUN + k)) bits |= 1u << k;
    return bits;
  };
  if (threadIdx.x == 0) pushes = 0;
  __syncthreads();
  int here = 0;
  for (int q = g0 + threadIdx.x; q < g1; q += kThreads) {
    int page[RUN];
    here += __popc(last_of(q, page));
  }
  here = __reduce_add_sync(0xffffffffu, here);
  if ((threadIdx.x & 31) == 0) atomicAdd(&pushes, here);
  sync();
  if (threadIdx.x == 0) {
    int before = 0, all = 0;
    for (int r = 0; r < CTAS; ++r) {
      const int p = CTAS > 1 ? *cg::this_cluster().map_shared_rank(&pushes, r) : pushes;
      before += r < rank ? p : 0;
      all += p;
    }
    base_s = before;
    if (rank == 0) {
      if (all > a.num_pages - count) raise_status(a.status, kStatusBadIndex);  // pages past the stack's room are dropped
      *a.free_count = min(count + all, a.num_pages);
    }
  }
  sync();
  long long base = (long long)count + base_s;
  for (int q0 = g0; q0 < g1; q0 += kThreads) {
    int page[RUN];
    const uint32_t bits = last_of(q0 + threadIdx.x, page);
    long long pushed;
    long long place = base + block_scan(__popc(bits), &pushed);
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      if (!((bits >> k) & 1)) continue;
      if (place < a.num_pages) a.free_pages[place] = page[k];
      args.shared[page[k]] = 0;
      ++place;
    }
    base += pushed;
  }
  if (rank == 0)
    for (int b = threadIdx.x; b < R; b += kThreads)
      if (a.done[b] != 0) a.lens[b] = 0;
}

int64_t tail_bytes(const ForkArgs& a) {
  return ((int64_t)a.pairs * a.layers * a.slabs * a.row_bytes) << a.page_shift;
}

}  // namespace

int fork_launches(const ForkArgs& a) { return tail_bytes(a) <= kOneLaunchBytes ? 1 : 2; }

cudaError_t launch_fork(const ForkArgs& a, int sm_count, cudaStream_t st) {
  const size_t smem = (size_t)a.pairs * 8;  // 32 KB at most
  if (fork_launches(a) == 1) {
    fork_kernel<kCopy | kState><<<1, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  const int64_t ctas = (tail_bytes(a) / kTailBytes + kThreads / 32 - 1) / (kThreads / 32);
  fork_kernel<kCopy><<<(unsigned)(ctas < sm_count ? ctas : sm_count), kThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
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
  return cudaLaunchKernelEx(&cfg, fork_kernel<kState>, a);
}

cudaError_t launch_release_shared(const ReleaseSharedArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  bool cluster = (int64_t)a.r.requests * a.r.max_pages > kAlone;
  if (cluster) {
    // 16 CTAs a cluster are more than every device must take, and more than a part of one may hold:
    // asked for once a device; where there is no room for one, a CTA releases alone, whatever the size
    static std::atomic<unsigned long long> asked{0}, has{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (asked.load(std::memory_order_acquire) & bit) {
      cluster = has.load(std::memory_order_relaxed) & bit;
    } else {
      int clusters = 0;
      e = cudaFuncSetAttribute(release_shared_kernel<kCluster, kRun>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, release_shared_kernel<kCluster, kRun>, &cfg);
      if (e != cudaSuccess) cudaGetLastError();  // no such clusters either
      cluster = e == cudaSuccess && clusters > 0;
      if (cluster) has.fetch_or(bit, std::memory_order_relaxed);
      asked.fetch_or(bit, std::memory_order_release);
    }
  }
  if (!cluster) {
    release_shared_kernel<1, 1><<<1, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  return cudaLaunchKernelEx(&cfg, release_shared_kernel<kCluster, kRun>, a);
}

}  // namespace kvq
