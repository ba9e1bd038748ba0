// Host side of the paged cache and of prompt attention (include/kvq.h):
// argument checks, the layout inside the caller's buffer and the launches.
#include <cstdarg>
#include <cstdio>
#include <new>

#include "paged_internal.h"

namespace {

kvq_status fail(kvq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kvq_status fail(kvq_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    kvq::set_error_message(buf);
  } catch (...) {  // no memory for the text: the status still says what failed
  }
  return s;
}

kvq_status cuda_fail(cudaError_t e, const char* what) {
  return fail(KVQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

kvq_status check_config(const kvq_paged_config* c) {
  if (!c) return fail(KVQ_ERR_INVALID_ARG, "config is NULL");
  if (c->num_layers < 1 || c->num_layers > 4096)
    return fail(KVQ_ERR_INVALID_ARG, "num_layers %d must be in [1, 4096]", c->num_layers);
  if (c->max_requests < 1 || c->max_requests > kvq::kMaxRequests)
    return fail(KVQ_ERR_INVALID_ARG, "max_requests %d must be in [1, %d]", c->max_requests, kvq::kMaxRequests);
  if (c->num_kv_heads < 1 || c->num_kv_heads > 1024)
    return fail(KVQ_ERR_INVALID_ARG, "num_kv_heads %d must be in [1, 1024]", c->num_kv_heads);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(KVQ_ERR_UNSUPPORTED, "head_dim %d must be 64 or 128", c->head_dim);
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return fail(KVQ_ERR_UNSUPPORTED, "page_tokens %d must be 16, 32, 64 or 128", c->page_tokens);
  if (c->num_pages < 1 || (int64_t)c->num_pages * c->page_tokens > INT32_MAX)
    return fail(KVQ_ERR_INVALID_ARG, "num_pages %d must be >= 1 and num_pages * page_tokens below 2^31", c->num_pages);
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_tokens > INT32_MAX - 255)  // tile ends stay 32-bit
    return fail(KVQ_ERR_INVALID_ARG, "max_pages %d must be >= 1 and max_pages * page_tokens at most 2^31 - 256",
                c->max_pages);
  if ((int64_t)c->max_requests * (((int64_t)c->max_pages * c->page_tokens + 63) / 64 + 5) > INT32_MAX)
    return fail(KVQ_ERR_UNSUPPORTED, "max_requests %d times max_pages %d is too large to plan a decode", c->max_requests,
                c->max_pages);
  if ((int64_t)c->num_pages * c->num_kv_heads * 2 > INT32_MAX)  // the code tiles' index
    return fail(KVQ_ERR_UNSUPPORTED, "num_pages %d times num_kv_heads %d must be below 2^30", c->num_pages,
                c->num_kv_heads);
  if (c->code != KVQ_PAGE_INT8 && c->code != KVQ_PAGE_E4M3)
    return fail(KVQ_ERR_INVALID_ARG, "code %d must be KVQ_PAGE_INT8 or KVQ_PAGE_E4M3", c->code);
  if (c->dtype != KVQ_F16 && c->dtype != KVQ_BF16)
    return fail(KVQ_ERR_INVALID_ARG, "dtype %d must be KVQ_F16 or KVQ_BF16", c->dtype);
  return KVQ_OK;
}

struct PagedPlan {
  int64_t pages_bytes, scales_bytes, tails_bytes;  // of one layer
  int64_t scales_off, tails_off, layer_bytes, total;
};

constexpr int64_t kHeader = 256;

PagedPlan make_plan(const kvq_paged_config& c) {
  PagedPlan p;
  const int64_t tile = 2ll * c.page_tokens * c.head_dim;
  p.pages_bytes = (int64_t)c.num_pages * c.num_kv_heads * tile;
  p.scales_bytes = (int64_t)c.num_pages * c.num_kv_heads * 2 * 4;
  p.tails_bytes = (int64_t)c.max_requests * c.num_kv_heads * tile * 2;
  p.scales_off = round_up(p.pages_bytes, 256);
  p.tails_off = p.scales_off + round_up(p.scales_bytes, 256);
  p.layer_bytes = p.tails_off + round_up(p.tails_bytes, 256);
  p.total = kHeader + p.layer_bytes * c.num_layers;
  return p;
}

}  // namespace

struct kvq_paged_cache {
  kvq_paged_config cfg;
  PagedPlan plan;
  unsigned char* base;
  int sm_count;
  int device;
};

namespace {

kvq_status check_handle(const kvq_paged_cache* h) {
  if (!h) return fail(KVQ_ERR_INVALID_ARG, "cache handle is NULL");
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != h->device)
    return fail(KVQ_ERR_INVALID_ARG, "the current device is %d but the cache lives on device %d", dev, h->device);
  return KVQ_OK;
}

kvq_status check_layer(const kvq_paged_cache* h, int layer) {
  if (!h) return fail(KVQ_ERR_INVALID_ARG, "cache handle is NULL");
  if (layer < 0 || layer >= h->cfg.num_layers)
    return fail(KVQ_ERR_INVALID_ARG, "layer %d out of range [0, %d)", layer, h->cfg.num_layers);
  return KVQ_OK;
}

kvq_status check_requests(const kvq_paged_cache* h, int requests) {
  if (requests < 1 || requests > h->cfg.max_requests)
    return fail(KVQ_ERR_INVALID_ARG, "requests %d must be in [1, %d]", requests, h->cfg.max_requests);
  return KVQ_OK;
}

kvq_status check_row(const char* what, const void* p, int64_t stride, int64_t row) {
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "%s must not be NULL", what);
  if (!aligned(p, 16)) return fail(KVQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  if (stride < row || stride % 8 != 0 || stride > (int64_t)1 << 31)
    return fail(KVQ_ERR_INVALID_ARG, "the token stride %lld of %s must be a multiple of 8 elements and in [%lld, 2^31]",
                (long long)stride, what, (long long)row);
  return KVQ_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

kvq::PagedDev layer_dev(const kvq_paged_cache* h, int layer) {
  unsigned char* lb = h->base + kHeader + h->plan.layer_bytes * layer;
  kvq::PagedDev c;
  c.pages = lb;
  c.scales = reinterpret_cast<float*>(lb + h->plan.scales_off);
  c.tails = reinterpret_cast<uint16_t*>(lb + h->plan.tails_off);
  c.heads = h->cfg.num_kv_heads;
  c.dim = h->cfg.head_dim;
  c.page_shift = log2_of(h->cfg.page_tokens);
  c.num_pages = h->cfg.num_pages;
  c.max_pages = h->cfg.max_pages;
  c.code = h->cfg.code;
  c.dtype = h->cfg.dtype;
  c.status = reinterpret_cast<uint32_t*>(h->base);
  return c;
}

kvq_status done(cudaError_t e, int launches, const char* what) {
  if (e != cudaSuccess) return cuda_fail(e, what);
  kvq::count_launches(launches);
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_paged_cache_bytes(const kvq_paged_config* cfg, size_t* bytes) {
  if (!bytes) return fail(KVQ_ERR_INVALID_ARG, "bytes is NULL");
  const kvq_status s = check_config(cfg);
  if (s != KVQ_OK) return s;
  *bytes = (size_t)make_plan(*cfg).total;
  return KVQ_OK;
}

kvq_status kvq_paged_cache_create(const kvq_paged_config* cfg, void* dev_buf, size_t bytes, void* stream,
                                  kvq_paged_cache** out) {
  if (!out) return fail(KVQ_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  const kvq_status s = check_config(cfg);
  if (s != KVQ_OK) return s;
  if (!dev_buf) return fail(KVQ_ERR_INVALID_ARG, "dev_buf is NULL");
  if (!aligned(dev_buf, 256)) return fail(KVQ_ERR_INVALID_ARG, "dev_buf must be 256-byte aligned");
  const PagedPlan p = make_plan(*cfg);
  if (bytes < (size_t)p.total)
    return fail(KVQ_ERR_BUFFER_TOO_SMALL, "cache buffer has %zu bytes, needs %lld", bytes, (long long)p.total);
  cudaPointerAttributes attr;
  cudaError_t e = cudaPointerGetAttributes(&attr, dev_buf);
  if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
  if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
    return fail(KVQ_ERR_INVALID_ARG, "dev_buf is not device memory");
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, attr.device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  e = cudaMemsetAsync(dev_buf, 0, (size_t)p.total, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  kvq_paged_cache* h = new (std::nothrow) kvq_paged_cache;
  if (!h) return fail(KVQ_ERR_INVALID_ARG, "no host memory for the handle");
  h->cfg = *cfg;
  h->plan = p;
  h->base = static_cast<unsigned char*>(dev_buf);
  h->sm_count = sms > 0 ? sms : 1;
  h->device = attr.device;
  *out = h;
  return KVQ_OK;
}

kvq_status kvq_paged_cache_destroy(kvq_paged_cache* cache) {
  delete cache;
  return KVQ_OK;
}

kvq_status kvq_paged_cache_get_layout(const kvq_paged_cache* h, int32_t layer, kvq_paged_layout* out) {
  const kvq_status s = check_layer(h, layer);
  if (s != KVQ_OK) return s;
  if (!out) return fail(KVQ_ERR_INVALID_ARG, "out is NULL");
  const kvq::PagedDev c = layer_dev(h, layer);
  out->pages_bytes = h->plan.pages_bytes;
  out->scales_bytes = h->plan.scales_bytes;
  out->tails_bytes = h->plan.tails_bytes;
  out->pages = c.pages;
  out->scales = c.scales;
  out->tails = c.tails;
  return KVQ_OK;
}

kvq_status kvq_paged_cache_status(kvq_paged_cache* h, void* stream, uint32_t* word) {
  const kvq_status s = check_handle(h);
  if (s != KVQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t w = 0;
  cudaError_t e = cudaMemcpyAsync(&w, h->base, sizeof w, cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync status");
  e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  if (w != 0) {
    e = cudaMemsetAsync(h->base, 0, sizeof w, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync status");
  }
  if (word) *word = w;
  if (w & kvq::kStatusTimeout) return fail(KVQ_ERR_TIMEOUT, "a bounded device wait gave up (status 0x%x)", w);
  if (w & ~kvq::kStatusNoRoom) return fail(KVQ_ERR_DEVICE_STATUS, "device status word 0x%x", w);
  if (w) return fail(KVQ_ERR_CAPACITY, "a reserve did not fit (status 0x%x)", w);
  return KVQ_OK;
}

kvq_status kvq_paged_reserve(kvq_paged_cache* h, int32_t requests, const int32_t* lens, const int32_t* new_tokens,
                             int32_t* table, const int32_t* free_pages, const int32_t* free_count,
                             int32_t max_tokens, int32_t* cu_tokens, int32_t* slots, int32_t* positions,
                             int32_t* lens_out, int32_t* free_count_out, void* stream) {
  kvq_status s = check_handle(h);
  if (s == KVQ_OK) s = check_requests(h, requests);
  if (s != KVQ_OK) return s;
  if (max_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "max_tokens must be >= 0");
  if (!lens || !new_tokens || !table || !free_pages || !free_count || !cu_tokens || !lens_out || !free_count_out ||
      (max_tokens > 0 && (!slots || !positions)))
    return fail(KVQ_ERR_INVALID_ARG, "the arrays must not be NULL");
  for (const void* p : {(const void*)lens, (const void*)new_tokens, (const void*)table, (const void*)free_pages,
                        (const void*)free_count, (const void*)cu_tokens, (const void*)slots, (const void*)positions,
                        (const void*)lens_out, (const void*)free_count_out})
    if (!aligned(p, 4)) return fail(KVQ_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  kvq::ReserveArgs a;
  a.requests = requests;
  a.page_shift = log2_of(h->cfg.page_tokens);
  a.num_pages = h->cfg.num_pages;
  a.max_pages = h->cfg.max_pages;
  a.max_tokens = max_tokens;
  a.lens = lens;
  a.add = new_tokens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.table = table;
  a.cu = cu_tokens;
  a.slots = slots;
  a.positions = positions;
  a.lens_out = lens_out;
  a.free_count_out = free_count_out;
  a.status = reinterpret_cast<uint32_t*>(h->base);
  return done(kvq::launch_reserve(a, static_cast<cudaStream_t>(stream)), kvq::reserve_launches(max_tokens),
              "reserve launch");
}

kvq_status kvq_paged_release(kvq_paged_cache* h, int32_t requests, const int32_t* done_flags, int32_t* lens,
                             const int32_t* table, int32_t* free_pages, int32_t* free_count, void* stream) {
  kvq_status s = check_handle(h);
  if (s == KVQ_OK) s = check_requests(h, requests);
  if (s != KVQ_OK) return s;
  if (!done_flags || !lens || !table || !free_pages || !free_count)
    return fail(KVQ_ERR_INVALID_ARG, "the arrays must not be NULL");
  for (const void* p : {(const void*)done_flags, (const void*)lens, (const void*)table, (const void*)free_pages,
                        (const void*)free_count})
    if (!aligned(p, 4)) return fail(KVQ_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  kvq::ReleaseArgs a;
  a.requests = requests;
  a.page_shift = log2_of(h->cfg.page_tokens);
  a.num_pages = h->cfg.num_pages;
  a.max_pages = h->cfg.max_pages;
  a.done = done_flags;
  a.table = table;
  a.lens = lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.status = reinterpret_cast<uint32_t*>(h->base);
  return done(kvq::launch_release(a, static_cast<cudaStream_t>(stream)), 1, "release launch");
}

kvq_status kvq_paged_write(kvq_paged_cache* h, int32_t layer, int32_t requests, const void* k, const void* v,
                           int64_t k_stride, int64_t v_stride, int32_t max_tokens, const int32_t* cu_tokens,
                           const int32_t* slots, const int32_t* lens, void* stream) {
  kvq_status s = check_layer(h, layer);
  if (s == KVQ_OK) s = check_handle(h);
  if (s == KVQ_OK) s = check_requests(h, requests);
  if (s != KVQ_OK) return s;
  if (max_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "max_tokens must be >= 0");
  if (max_tokens == 0) return KVQ_OK;
  const int64_t row = (int64_t)h->cfg.num_kv_heads * h->cfg.head_dim;
  s = check_row("k", k, k_stride, row);
  if (s == KVQ_OK) s = check_row("v", v, v_stride, row);
  if (s != KVQ_OK) return s;
  if (!cu_tokens || !slots || !lens) return fail(KVQ_ERR_INVALID_ARG, "the arrays must not be NULL");
  if (!aligned(cu_tokens, 4) || !aligned(slots, 4) || !aligned(lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  kvq::PagedWriteArgs a;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.max_tokens = max_tokens;
  a.requests = requests;
  a.cu = cu_tokens;
  a.slots = slots;
  a.lens = lens;
  return done(kvq::launch_paged_write(layer_dev(h, layer), a, static_cast<cudaStream_t>(stream)), 1,
              "paged write launch");
}

kvq_status kvq_paged_decode_workspace_bytes(const kvq_paged_cache* h, int32_t num_q_heads, size_t* bytes) {
  if (!h) return fail(KVQ_ERR_INVALID_ARG, "cache handle is NULL");
  if (!bytes) return fail(KVQ_ERR_INVALID_ARG, "bytes is NULL");
  const int hkv = h->cfg.num_kv_heads;
  if (num_q_heads < hkv || num_q_heads % hkv != 0 || num_q_heads > 65535)
    return fail(KVQ_ERR_INVALID_ARG, "num_q_heads %d must be a multiple of num_kv_heads %d and at most 65535",
                num_q_heads, hkv);
  *bytes = kvq::paged_decode_workspace(h->cfg.head_dim, num_q_heads / hkv, h->cfg.max_requests, h->sm_count);
  return KVQ_OK;
}

kvq_status kvq_paged_decode_attention(kvq_paged_cache* h, int32_t layer, int32_t requests, const void* q,
                                      int64_t q_stride, int32_t num_q_heads, const int32_t* table,
                                      const int32_t* lens, float softmax_scale, void* out, int32_t out_dtype,
                                      void* workspace, size_t ws_bytes, void* stream) {
  kvq_status s = check_layer(h, layer);
  if (s == KVQ_OK) s = check_handle(h);
  if (s == KVQ_OK) s = check_requests(h, requests);
  size_t need = 0;
  if (s == KVQ_OK) s = kvq_paged_decode_workspace_bytes(h, num_q_heads, &need);
  if (s == KVQ_OK) s = check_row("q", q, q_stride, (int64_t)num_q_heads * h->cfg.head_dim);
  if (s != KVQ_OK) return s;
  if (!table || !lens || !out || !workspace)
    return fail(KVQ_ERR_INVALID_ARG, "table, lens, out and workspace must not be NULL");
  if (!aligned(table, 4) || !aligned(lens, 4)) return fail(KVQ_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  if (!aligned(out, 16) || !aligned(workspace, 16))
    return fail(KVQ_ERR_INVALID_ARG, "out and workspace must be 16-byte aligned");
  if (out_dtype != KVQ_F32 && out_dtype != h->cfg.dtype)
    return fail(KVQ_ERR_INVALID_ARG, "out_dtype must be KVQ_F32 or the cache's dtype");
  if (!(softmax_scale > -2.0e38f && softmax_scale < 2.0e38f))
    return fail(KVQ_ERR_INVALID_ARG, "softmax_scale must be finite");
  if (ws_bytes < need) return fail(KVQ_ERR_BUFFER_TOO_SMALL, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  kvq::PagedDecodeArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.requests = requests;
  a.q_heads = num_q_heads;
  a.group = num_q_heads / h->cfg.num_kv_heads;
  a.table = table;
  a.lens = lens;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_dtype == KVQ_F32;
  a.ws = workspace;
  a.sm_count = h->sm_count;
  return done(kvq::launch_paged_decode(layer_dev(h, layer), a, static_cast<cudaStream_t>(stream)), 2,
              "paged decode launch");
}

kvq_status kvq_prompt_attention(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, int32_t max_tokens, int32_t num_seqs, const int32_t* cu_tokens,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                                float softmax_scale, void* out, uint32_t* status, void* stream) {
  if (head_dim != 64 && head_dim != 128) return fail(KVQ_ERR_UNSUPPORTED, "head_dim %d must be 64 or 128", head_dim);
  if (dtype != KVQ_F16 && dtype != KVQ_BF16)
    return fail(KVQ_ERR_INVALID_ARG, "dtype %d must be KVQ_F16 or KVQ_BF16", dtype);
  if (num_kv_heads < 1 || num_kv_heads > 1024)
    return fail(KVQ_ERR_INVALID_ARG, "num_kv_heads %d must be in [1, 1024]", num_kv_heads);
  if (num_q_heads < num_kv_heads || num_q_heads % num_kv_heads != 0 || num_q_heads > 65535)
    return fail(KVQ_ERR_INVALID_ARG, "num_q_heads %d must be a multiple of num_kv_heads %d and at most 65535",
                num_q_heads, num_kv_heads);
  if (num_seqs < 1 || num_seqs > kvq::kMaxRequests)
    return fail(KVQ_ERR_INVALID_ARG, "num_seqs %d must be in [1, %d]", num_seqs, kvq::kMaxRequests);
  if (max_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "max_tokens must be >= 0");
  if (max_tokens > 1 << 26)  // the kernel's bounded waits are four times the longest block of such a prompt
    return fail(KVQ_ERR_UNSUPPORTED, "max_tokens %d exceeds 2^26", max_tokens);
  if (max_tokens == 0) return KVQ_OK;
  kvq_status s = check_row("q", q, q_stride, (int64_t)num_q_heads * head_dim);
  if (s == KVQ_OK) s = check_row("k", k, k_stride, (int64_t)num_kv_heads * head_dim);
  if (s == KVQ_OK) s = check_row("v", v, v_stride, (int64_t)num_kv_heads * head_dim);
  if (s != KVQ_OK) return s;
  if (!cu_tokens || !out) return fail(KVQ_ERR_INVALID_ARG, "cu_tokens and out must not be NULL");
  if (!aligned(out, 16) || !aligned(cu_tokens, 4) || !aligned(status, 4))
    return fail(KVQ_ERR_INVALID_ARG, "out must be 16-byte, cu_tokens and status 4-byte aligned");
  if (!(softmax_scale >= 0.0f && softmax_scale < 2.0e38f))
    return fail(KVQ_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  for (const void* p : {q, k, v, (const void*)out, (const void*)cu_tokens, (const void*)status}) {
    if (!p) continue;
    cudaPointerAttributes attr;
    e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
    if ((attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) || attr.device != dev)
      return fail(KVQ_ERR_INVALID_ARG, "q, k, v, out, cu_tokens and status must be memory of the current device %d",
                  dev);
  }
  kvq::PromptArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tokens = max_tokens;
  a.seqs = num_seqs;
  a.q_heads = num_q_heads;
  a.kv_heads = num_kv_heads;
  a.dim = head_dim;
  a.dtype = dtype;
  a.cu = cu_tokens;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out);
  a.status = status;
  return done(kvq::launch_prompt_attention(a, static_cast<cudaStream_t>(stream)), 1, "prompt attention launch");
}

}  // extern "C"
