// C ABI entry points: argument checks, kernel choice, launch accounting.
// Declarations and the meaning of every argument are in include/kvq.h.
#include <math.h>

#include "kvq_internal.h"
#include "paged.cuh"

namespace {

thread_local int32_t g_last_launches = 0;
thread_local const char *g_last_path = "";
thread_local uint64_t g_wait_limit_ns = 0;
thread_local int32_t g_drop_item = -1;

constexpr uint64_t kDefaultWaitNs = 1000000000ull;  // one second
constexpr double kLog2e = 1.4426950408889634;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 148;
  if (dev < 64) cache[dev] = n;
  return n;
}

kvq::KernelCtl make_ctl(int32_t *dev_status) {
  kvq::KernelCtl c;
  c.dev_status = dev_status;
  c.wait_limit_ns = g_wait_limit_ns ? g_wait_limit_ns : kDefaultWaitNs;
  c.drop_item = g_drop_item;
#ifdef KVQ_DEBUG
  c.n_bufs = 0;
#endif
  return c;
}

// The bounds-check table of a KVQ_DEBUG build: each device buffer of the
// call, as [p, p + bytes). Other builds keep no table and these do nothing.
void ctl_add(kvq::KernelCtl &c, const void *p, size_t bytes) {
#ifdef KVQ_DEBUG
  if (!p || bytes == 0 || c.n_bufs >= kvq::kMaxBufs) return;
  c.buf_lo[c.n_bufs] = reinterpret_cast<uintptr_t>(p);
  c.buf_hi[c.n_bufs] = reinterpret_cast<uintptr_t>(p) + bytes;
  ++c.n_bufs;
#else
  (void)c;
  (void)p;
  (void)bytes;
#endif
}

// Bytes of rows x d elements of type dt.
size_t rows_bytes(long rows, int d, int32_t dt) {
  return static_cast<size_t>(rows) * static_cast<size_t>(d) *
         (dt == KVQ_F32 ? 4u : dt == KVQ_BF16 ? 2u : 1u);
}

bool shape_ok(int32_t batch, int32_t kv_heads, int32_t n_tokens, int32_t head_dim, int32_t recent,
              int32_t kwin, int32_t vwin) {
  if (batch < 1 || kv_heads < 1 || n_tokens < 1) return false;
  if (head_dim < 32 || head_dim > 256 || head_dim % 32) return false;
  if (recent < 0 || recent > n_tokens) return false;
  if (kwin != KVQ_F32 && kwin != KVQ_BF16 && kwin != KVQ_MXFP8) return false;
  if (vwin != KVQ_F32 && vwin != KVQ_BF16) return false;
  return true;
}

size_t elem_bytes(int32_t dt) { return dt == KVQ_F32 ? 4 : dt == KVQ_BF16 ? 2 : 1; }

// Validates the cache descriptor's shape and the pointers its arrays need.
kvq_status check_cache(const kvq_cache *c) {
  if (!c) return KVQ_ERR_ARG;
  if (!shape_ok(c->batch, c->kv_heads, c->n_tokens, c->head_dim, c->recent, c->kwin_dtype,
                c->vwin_dtype))
    return KVQ_ERR_ARG;
  const int cut = c->n_tokens - c->recent;
  if (c->cap_groups < 0 || c->cap_window < 0) return KVQ_ERR_ARG;
  if (c->cap_groups > 0 && (c->cap_groups < (cut + 31) / 32 || c->cap_window < c->recent))
    return KVQ_ERR_ARG;
  if (c->cap_groups == 0 && c->cap_window != 0) return KVQ_ERR_ARG;
  if (cut > 0) {
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return KVQ_ERR_ARG;
    if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) ||
        !aligned16(c->v_scales))
      return KVQ_ERR_ALIGN;
  }
  if (c->recent > 0) {
    if (!c->k_window || !c->v_window) return KVQ_ERR_ARG;
    if (c->kwin_dtype == KVQ_MXFP8 && !c->k_window_e8m0) return KVQ_ERR_ARG;
    if (!aligned16(c->k_window) || !aligned16(c->v_window)) return KVQ_ERR_ALIGN;
    if (c->kwin_dtype == KVQ_MXFP8 && !aligned16(c->k_window_e8m0)) return KVQ_ERR_ALIGN;
  }
  return KVQ_OK;
}

kvq_status finish(int launches, const char *path) {
  if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  g_last_launches = launches;
  g_last_path = path;
  return KVQ_OK;
}

// The calls that fill a cache (kv_pack, kv_append) come before any decode,
// so they reserve the static decode scratch of the current device (loading
// its module) before a runtime hands the rest of HBM to its own pool. A
// failure here is not the caller's: it is cleared and kv_attend_decode_static
// retries, returning KVQ_ERR_CUDA if the array still cannot be had.
void reserve_static_scratch() {
  void *p = nullptr;
  (void)kvq::decode_static_scratch(&p);
}

float resolve_scale(float sm_scale, int head_dim) {
  return sm_scale > 0.0f ? sm_scale
                         : static_cast<float>(1.0 / sqrt(static_cast<double>(head_dim)));
}

// The cache's arrays, at the sizes its shape (and reserved room) gives.
void ctl_add_cache(kvq::KernelCtl &c, const kvq_cache &k) {
#ifdef KVQ_DEBUG
  size_t sz[8];
  const kvq_status st =
      k.cap_groups > 0
          ? kvq_cache_sizes_reserved(k.batch, k.kv_heads, k.head_dim, k.kwin_dtype, k.vwin_dtype,
                                     k.cap_groups, k.cap_window, sz)
          : kvq_cache_sizes(k.batch, k.kv_heads, k.n_tokens, k.head_dim, k.recent, k.kwin_dtype,
                            k.vwin_dtype, sz);
  if (st != KVQ_OK) return;
  ctl_add(c, k.k_codes, sz[0]);
  ctl_add(c, k.k_scales, sz[1]);
  ctl_add(c, k.v_codes, sz[2]);
  ctl_add(c, k.v_scales, sz[3]);
  ctl_add(c, k.k_window, sz[4]);
  ctl_add(c, k.v_window, sz[5]);
  ctl_add(c, k.k_window_e8m0, sz[6]);
#else
  (void)c;
  (void)k;
#endif
}

// Blocks of the int4 part.
int summary_blocks(const kvq_cache &c, int block) {
  return (c.n_tokens - c.recent + block - 1) / block;
}

kvq_status check_summary(const kvq_cache *c, const kvq_summary *s) {
  if (!s) return KVQ_ERR_ARG;
  if (s->block != 32 && s->block != 64 && s->block != 128) return KVQ_ERR_ARG;
  const int blocks = summary_blocks(*c, s->block);
  if (s->cap_blocks < blocks) return KVQ_ERR_WORKSPACE;
  if (blocks > 0) {
    if (!s->codes || !s->scales) return KVQ_ERR_ARG;
    if (!aligned16(s->codes) || !aligned16(s->scales)) return KVQ_ERR_ALIGN;
  }
  return KVQ_OK;
}

void ctl_add_summary(kvq::KernelCtl &c, const kvq_cache &k, const kvq_summary &s) {
  const size_t rows = static_cast<size_t>(k.batch) * k.kv_heads * s.cap_blocks;
  ctl_add(c, s.codes, rows * k.head_dim);
  ctl_add(c, s.scales, rows * sizeof(float));
}

bool page_state_ok(const kvq_page_state &s) {
  return s.slots >= 1 && s.slots <= KVQ_PAGES_MAX_SLOTS && s.n_pages >= 1 &&
         s.n_pages <= (1 << 28) && s.max_pages >= 1 &&
         (s.page == 32 || s.page == 64 || s.page == 128) && s.window >= 0 && s.window <= 65536 &&
         static_cast<long>(s.max_pages) * s.page + s.window + 64 <= 0x7fffffffL;
}

// (with these limits the sizes fit 64 bits)
bool paged_ok(const kvq_paged_cache &c) {
  return page_state_ok(c.state) && c.kv_heads >= 1 && c.kv_heads <= 65535 &&
         c.head_dim >= 32 && c.head_dim <= 256 && c.head_dim % 32 == 0 && (c.win_dtype == KVQ_F32 || c.win_dtype == KVQ_BF16);
}

kvq_status check_page_state(const kvq_page_state *s) {
  if (!s || !page_state_ok(*s)) return KVQ_ERR_ARG;
  if (!s->table || !s->lengths || !s->free_pages || !s->n_free) return KVQ_ERR_ARG;
  if (!aligned16(s->table) || !aligned16(s->lengths) || !aligned16(s->free_pages) ||
      !aligned16(s->n_free))
    return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

kvq_status check_paged(const kvq_paged_cache *c) {
  if (!c || !paged_ok(*c)) return KVQ_ERR_ARG;
  const kvq_status st = check_page_state(&c->state);
  if (st != KVQ_OK) return st;
  if (!c->pool || !c->ring) return KVQ_ERR_ARG;
  if (!aligned16(c->pool) || !aligned16(c->ring)) return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

kvq_status check_plan(const kvq_page_state &s, const kvq_page_plan *p) {
  if (!p || p->rows < 0 || p->rows > (1 << 28) || p->cap_work < 0) return KVQ_ERR_ARG;
  if (p->cap_work < kvq_page_work(&s, p->rows)) return KVQ_ERR_WORKSPACE;
  if (!p->offsets || !p->before || !p->after || !p->counts) return KVQ_ERR_ARG;
  if (p->rows > 0 && (!p->row_slot || !p->positions || !p->work)) return KVQ_ERR_ARG;
  if (!aligned16(p->offsets) || !aligned16(p->before) || !aligned16(p->after) ||
      !aligned16(p->row_slot) || !aligned16(p->positions) || !aligned16(p->work) ||
      !aligned16(p->counts))
    return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

void ctl_add_pages(kvq::KernelCtl &c, const kvq_paged_cache &k) {
#ifdef KVQ_DEBUG
  size_t sz[6];
  if (kvq_paged_sizes(&k, sz) != KVQ_OK) return;
  ctl_add(c, k.state.table, sz[0]);
  ctl_add(c, k.state.lengths, sz[1]);
  ctl_add(c, k.pool, sz[4]);
  ctl_add(c, k.ring, sz[5]);
#else
  (void)c;
  (void)k;
#endif
}

void ctl_add_plan(kvq::KernelCtl &c, const kvq_page_state &s, const kvq_page_plan &p) {
  ctl_add(c, p.offsets, 4 * (static_cast<size_t>(s.slots) + 1));
  ctl_add(c, p.before, 4 * static_cast<size_t>(s.slots));
  ctl_add(c, p.after, 4 * static_cast<size_t>(s.slots));
  ctl_add(c, p.work, 32 * static_cast<size_t>(p.cap_work));
  ctl_add(c, p.counts, 16);
}

}  // namespace

extern "C" {

kvq_status kvq_cache_sizes(int32_t batch, int32_t kv_heads, int32_t n_tokens, int32_t head_dim,
                           int32_t recent, int32_t kwin_dtype, int32_t vwin_dtype,
                           size_t sizes[8]) {
  if (!sizes || !shape_ok(batch, kv_heads, n_tokens, head_dim, recent, kwin_dtype, vwin_dtype))
    return KVQ_ERR_ARG;
  const size_t units = static_cast<size_t>(batch) * kv_heads;
  const size_t cut = static_cast<size_t>(n_tokens - recent);
  const size_t gk = (cut + 31) / 32;
  const size_t d = static_cast<size_t>(head_dim);
  sizes[0] = units * gk * 32 * d / 2;                 // k_codes
  sizes[1] = units * gk * d * sizeof(float);          // k_scales
  sizes[2] = units * cut * d / 2;                     // v_codes
  sizes[3] = units * cut * (d / 32) * sizeof(float);  // v_scales
  sizes[4] = units * recent * d * elem_bytes(kwin_dtype);
  sizes[5] = units * recent * d * elem_bytes(vwin_dtype);
  sizes[6] = kwin_dtype == KVQ_MXFP8 ? units * recent * (d / 32) : 0;
  sizes[7] = 16;                                      // {N, D, R, 32}
  return KVQ_OK;
}

kvq_status kvq_cache_sizes_reserved(int32_t batch, int32_t kv_heads, int32_t head_dim,
                                    int32_t kwin_dtype, int32_t vwin_dtype, int32_t cap_groups,
                                    int32_t cap_window, size_t sizes[8]) {
  if (!sizes || cap_groups < 1 || cap_window < 0 ||
      !shape_ok(batch, kv_heads, 1, head_dim, 0, kwin_dtype, vwin_dtype))
    return KVQ_ERR_ARG;
  const size_t units = static_cast<size_t>(batch) * kv_heads;
  const size_t gs = static_cast<size_t>(cap_groups), ws = static_cast<size_t>(cap_window);
  const size_t d = static_cast<size_t>(head_dim);
  sizes[0] = units * gs * 32 * d / 2;
  sizes[1] = units * gs * d * sizeof(float);
  sizes[2] = units * gs * 32 * d / 2;
  sizes[3] = units * gs * 32 * (d / 32) * sizeof(float);
  sizes[4] = units * ws * d * elem_bytes(kwin_dtype);
  sizes[5] = units * ws * d * elem_bytes(vwin_dtype);
  sizes[6] = kwin_dtype == KVQ_MXFP8 ? units * ws * (d / 32) : 0;
  sizes[7] = 16;
  return KVQ_OK;
}

size_t kvq_cache_bytes(int32_t batch, int32_t kv_heads, int32_t n_tokens, int32_t head_dim,
                       int32_t recent, int32_t kwin_dtype, int32_t vwin_dtype) {
  size_t s[8];
  if (kvq_cache_sizes(batch, kv_heads, n_tokens, head_dim, recent, kwin_dtype, vwin_dtype, s) !=
      KVQ_OK)
    return 0;
  size_t total = 0;
  for (int i = 0; i < 8; ++i) total += s[i];
  return total;
}

kvq_status kv_pack(const void *k, const void *v, int32_t in_dtype, kvq_cache *cache,
                   int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (in_dtype != KVQ_F32 && in_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (!k || !v) return KVQ_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  cache->header[0] = static_cast<uint32_t>(cache->n_tokens);
  cache->header[1] = static_cast<uint32_t>(cache->head_dim);
  cache->header[2] = static_cast<uint32_t>(cache->recent);
  cache->header[3] = 32u;
  reserve_static_scratch();
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_cache(ctl, *cache);
  const long units = static_cast<long>(cache->batch) * cache->kv_heads;
  ctl_add(ctl, k, rows_bytes(units * cache->n_tokens, cache->head_dim, in_dtype));
  ctl_add(ctl, v, rows_bytes(units * cache->n_tokens, cache->head_dim, in_dtype));
  const int n = kvq::launch_pack(k, v, in_dtype, *cache, ctl, sm_count(),
                                 reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "pack");
}

kvq_status kv_append(kvq_cache *cache, const void *k_new, const void *v_new, int32_t in_dtype,
                     int32_t n_new, int32_t window, int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (in_dtype != KVQ_F32 && in_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (n_new < 1 || window < 0 || !k_new || !v_new) return KVQ_ERR_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  if (cache->cap_groups <= 0) return KVQ_ERR_UNSUPPORTED;
  if ((cache->kwin_dtype != KVQ_F32 && cache->kwin_dtype != KVQ_BF16) ||
      (cache->vwin_dtype != KVQ_F32 && cache->vwin_dtype != KVQ_BF16))
    return KVQ_ERR_UNSUPPORTED;
  const int cut = cache->n_tokens - cache->recent;
  if (cut % 32) return KVQ_ERR_UNSUPPORTED;  // a padded last K group cannot grow
  if (n_new > 0x7fffffff - cache->n_tokens) return KVQ_ERR_ARG;
  const int n2 = cache->n_tokens + n_new;
  int cut2 = n2 > window ? 32 * ((n2 - window) / 32) : 0;
  if (cut2 < cut) cut2 = cut;
  const int r2 = n2 - cut2, m = (cut2 - cut) / 32;
  if (cut2 / 32 > cache->cap_groups || r2 > cache->cap_window) return KVQ_ERR_WORKSPACE;
  if (m > 0 && static_cast<long>(cache->batch) * cache->kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  reserve_static_scratch();
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_cache(ctl, *cache);
  const long units = static_cast<long>(cache->batch) * cache->kv_heads;
  ctl_add(ctl, k_new, rows_bytes(units * n_new, cache->head_dim, in_dtype));
  ctl_add(ctl, v_new, rows_bytes(units * n_new, cache->head_dim, in_dtype));
  const int n = kvq::launch_append(*cache, k_new, v_new, in_dtype, n_new, m, r2, ctl,
                                   reinterpret_cast<cudaStream_t>(stream));
  const kvq_status done = finish(n, "append");
  if (done != KVQ_OK) return done;
  cache->n_tokens = n2;
  cache->recent = r2;
  cache->header[0] = static_cast<uint32_t>(n2);
  cache->header[1] = static_cast<uint32_t>(cache->head_dim);
  cache->header[2] = static_cast<uint32_t>(r2);
  cache->header[3] = 32u;
  return KVQ_OK;
}

kvq_status kv_attend(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t q_heads,
                     int32_t n_q, float sm_scale, void *out, int32_t out_dtype,
                     const int32_t *region_bounds, int32_t n_regions, float *region_mass,
                     void *workspace, size_t *ws_bytes, int32_t *dev_status,
                     kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (region_bounds) {
    if (n_regions < 1 || n_regions > 16 || !region_mass) return KVQ_ERR_ARG;
    if (region_bounds[0] != 0 || region_bounds[n_regions] != cache->n_tokens) return KVQ_ERR_ARG;
    for (int i = 0; i < n_regions; ++i)
      if (region_bounds[i + 1] <= region_bounds[i]) return KVQ_ERR_ARG;
    if (!aligned16(region_mass)) return KVQ_ERR_ALIGN;
  }
  const bool regions = region_bounds != nullptr;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  const int sms = sm_count();

  enum { GENERIC, DECODE, CHUNK } path = GENERIC;
  // the chunk kernel's grid is (query tiles, batch * q_heads)
  if (kvq::chunk_supported(*cache, q_dtype, q_heads, n_q) &&
      static_cast<long>(cache->batch) * q_heads <= 65535 &&
      (!regions || n_regions <= kvq::chunk_max_regions()))
    path = CHUNK;
  else if (!regions && kvq::decode_supported(*cache, q_dtype, q_heads, n_q))
    path = DECODE;
  // the fp32 kernel's grid is (row blocks, q_heads, batch)
  if (path == GENERIC && (q_heads > 65535 || cache->batch > 65535)) return KVQ_ERR_UNSUPPORTED;
  size_t need = 0;
  if (path == DECODE) need = kvq::decode_workspace_bytes(*cache, q_heads, sms);
  if (path == CHUNK) need = kvq::chunk_workspace_bytes(*cache, q_heads, n_q);
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;

  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    if (regions) ctl_add(ctl, region_mass, rows_bytes(rows, n_regions, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (path == CHUNK) {
    const int n = kvq::launch_attend_chunk(*cache, q, q_heads, n_q,
                                           static_cast<float>(scale * kLog2e), out, out_dtype,
                                           region_bounds, n_regions, region_mass, workspace, ctl, s);
    if (n < 0) return KVQ_ERR_CUDA;
    return finish(n, cache->recent < cache->n_tokens   ? "chunk_int4"
                     : cache->kwin_dtype == KVQ_MXFP8 ? "chunk_mxfp8"
                                                      : "chunk_bf16");
  }
  if (path == DECODE) {
    const int n = kvq::launch_attend_decode(*cache, q, q_dtype,
                                            static_cast<float>(scale * kLog2e), out, out_dtype,
                                            workspace, ctl, sms, s);
    return finish(n, "decode");
  }
  const int n = kvq::launch_attend_generic(*cache, q, q_dtype, q_heads, n_q, scale, out,
                                           out_dtype, region_bounds, n_regions, region_mass, ctl, s);
  return finish(n, "generic");
}

kvq_status kv_attend_stats(const kvq_cache *cache, const void *q, int32_t q_dtype,
                           int32_t q_heads, int32_t n_q, float sm_scale,
                           const float *hadamard_signs, float *stats, void *workspace,
                           size_t *ws_bytes, int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1) return KVQ_ERR_ARG;
  if (q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  const int d = cache->head_dim;
  if ((d & (d - 1)) != 0 || cache->n_tokens > kvq::stats_max_tokens()) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<long>(cache->batch) * q_heads * n_q > 0x7fffffffL) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<long>(cache->batch) * q_heads > 65535) return KVQ_ERR_UNSUPPORTED;  // grid.y
  const size_t need = kvq::stats_workspace_bytes(*cache, q_heads, n_q);
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !stats) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(stats) || !aligned16(workspace) ||
      (hadamard_signs && !aligned16(hadamard_signs)) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, d);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, d, q_dtype));
    ctl_add(ctl, stats, rows_bytes(rows, KVQ_N_STATS, KVQ_F32));
    ctl_add(ctl, hadamard_signs, rows_bytes(1, d, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  const int n = kvq::launch_attend_stats(*cache, q, q_dtype, q_heads, n_q, scale, hadamard_signs,
                                         stats, workspace, ctl,
                                         reinterpret_cast<cudaStream_t>(stream));
  if (n < 0) return KVQ_ERR_UNSUPPORTED;
  return finish(n, "stats");
}

kvq_status kv_attend_candidates(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                int32_t q_heads, int32_t n_q, const int32_t *idx,
                                int32_t n_cand, int32_t validate, float sm_scale, void *out,
                                int32_t out_dtype, void *workspace, size_t *ws_bytes,
                                int32_t *dev_status, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1 || n_cand < 1) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (cache->recent > 0 && cache->kwin_dtype == KVQ_MXFP8) return KVQ_ERR_UNSUPPORTED;
  // the grid is (query rows, q_heads, batch)
  if (n_cand > 65536 || q_heads > 65535 || cache->batch > 65535) return KVQ_ERR_UNSUPPORTED;
  const int sms = sm_count();
  const bool uni = kvq::candidates_union_supported(*cache, q_dtype, q_heads, n_q, n_cand);
  const size_t need = uni ? kvq::candidates_union_workspace_bytes(*cache, n_cand, sms) : 0;
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out || !idx) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(idx) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, idx, rows_bytes(rows, n_cand, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  if (uni) {
    const int n = kvq::launch_candidates_union(*cache, q, idx, n_cand, validate,
                                               static_cast<float>(scale * kLog2e), out, out_dtype,
                                               workspace, ctl, sms, s);
    return finish(n, "candidates_union");
  }
  const int n = kvq::launch_attend_candidates(*cache, q, q_dtype, q_heads, n_q, idx, n_cand,
                                              validate, static_cast<float>(scale * kLog2e), out,
                                              out_dtype, ctl, s);
  return finish(n, "candidates");
}

kvq_status kv_attend_candidates_topk(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                     int32_t q_heads, int32_t n_q, const int32_t *idx,
                                     int32_t n_cand, int32_t top_k, float sm_scale, void *out,
                                     int32_t out_dtype, int32_t *selected, int32_t *dev_status,
                                     kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1 || n_cand < 1) return KVQ_ERR_ARG;
  if (top_k < 1 || top_k > n_cand) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (!q || !out || !idx) return KVQ_ERR_ARG;
  if (cache->recent > 0 && cache->kwin_dtype == KVQ_MXFP8) return KVQ_ERR_UNSUPPORTED;
  if (n_cand > kvq::candidates_topk_max() || q_heads > 65535 || cache->batch > 65535)
    return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !aligned16(idx) || (selected && !aligned16(selected)) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, idx, rows_bytes(rows, n_cand, KVQ_F32));
    ctl_add(ctl, selected, rows_bytes(rows, top_k, KVQ_F32));
  }
  const int n = kvq::launch_attend_candidates(
      *cache, q, q_dtype, q_heads, n_q, idx, n_cand, 0, static_cast<float>(scale * kLog2e), out,
      out_dtype, ctl, reinterpret_cast<cudaStream_t>(stream), top_k, selected);
  if (n < 0) return KVQ_ERR_UNSUPPORTED;
  return finish(n, "candidates_topk");
}

kvq_status kv_attend_candidates_block(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                      int32_t q_heads, int32_t n_q, const int32_t *idx,
                                      int32_t n_cand, int32_t block_q, float sm_scale, void *out,
                                      int32_t out_dtype, void *workspace, size_t *ws_bytes,
                                      int32_t *dev_status, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1 || n_cand < 1 || block_q < 1)
    return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (cache->recent > 0 && cache->kwin_dtype == KVQ_MXFP8) return KVQ_ERR_UNSUPPORTED;
  if (n_cand > 65536 || q_heads > 65535 || cache->batch > 65535) return KVQ_ERR_UNSUPPORTED;
  const long lists = static_cast<long>(cache->batch) * q_heads * ((n_q + block_q - 1) / block_q);
  const bool tensor = kvq::candidate_lists_supported(*cache, q_dtype, block_q) && lists <= 65535;
  const size_t need = tensor ? kvq::candidate_lists_workspace_bytes(lists, n_cand) : 0;
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out || !idx) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(idx) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, idx, rows_bytes(lists, n_cand, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  if (tensor) {
    const int n = kvq::launch_candidate_lists(*cache, q, q_heads, n_q, idx, n_cand, block_q,
                                              static_cast<float>(scale * kLog2e), out, out_dtype,
                                              workspace, ctl, s);
    if (n < 0) return KVQ_ERR_CUDA;
    return finish(n, "candidates_block_tensor");
  }
  const int n = kvq::launch_attend_candidates(*cache, q, q_dtype, q_heads, n_q, idx, n_cand, 0,
                                              static_cast<float>(scale * kLog2e), out, out_dtype,
                                              ctl, s, 0, nullptr, block_q);
  return finish(n, "candidates_block");
}

kvq_status kv_attend_region_drop(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                 int32_t q_heads, int32_t n_q, float sm_scale,
                                 const int32_t *region_bounds, int32_t n_regions,
                                 uint32_t drop_mask, void *out, int32_t out_dtype,
                                 void *workspace, size_t *ws_bytes, int32_t *dev_status,
                                 kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes || !region_bounds) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1) return KVQ_ERR_ARG;
  if (n_regions < 1 || n_regions > 16) return KVQ_ERR_ARG;
  if (region_bounds[0] != 0 || region_bounds[n_regions] != cache->n_tokens) return KVQ_ERR_ARG;
  for (int i = 0; i < n_regions; ++i)
    if (region_bounds[i + 1] <= region_bounds[i]) return KVQ_ERR_ARG;
  if (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  int kept = 0;
  for (int r = 0; r < n_regions; ++r)
    if (!(drop_mask & (1u << r))) kept += region_bounds[r + 1] - region_bounds[r];
  if (kept == 0 || (drop_mask >> n_regions) != 0) return KVQ_ERR_ARG;
  if (!kvq::candidate_lists_supported(*cache, q_dtype, 128) || q_heads > 65535 ||
      static_cast<long>(cache->batch) * cache->kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  const size_t need = kvq::region_drop_workspace_bytes(*cache, kept);
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  const int n = kvq::launch_region_drop(*cache, q, q_heads, n_q, region_bounds, n_regions,
                                        drop_mask, static_cast<float>(scale * kLog2e), out,
                                        out_dtype, workspace, ctl,
                                        reinterpret_cast<cudaStream_t>(stream));
  if (n < 0) return KVQ_ERR_CUDA;
  return finish(n, "region_drop");
}

kvq_status kv_attend_decode_static(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                   int32_t q_heads, float sm_scale, void *out,
                                   int32_t out_dtype, int32_t *dev_status, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (q_heads < 1 || q_heads % cache->kv_heads) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (!kvq::decode_supported(*cache, q_dtype, q_heads, 1)) return KVQ_ERR_UNSUPPORTED;
  if (!q || !out) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const int sms = sm_count();
  if (kvq::decode_workspace_bytes(*cache, q_heads, sms) > kvq::decode_static_scratch_limit())
    return KVQ_ERR_WORKSPACE;
  void *scratch = nullptr;
  if (kvq::decode_static_scratch(&scratch) != cudaSuccess) return KVQ_ERR_CUDA;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, scratch, kvq::decode_static_scratch_limit());
  }
  const int n = kvq::launch_attend_decode(*cache, q, q_dtype, static_cast<float>(scale * kLog2e),
                                          out, out_dtype, scratch, ctl, sms,
                                          reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "decode_static");
}

kvq_status kvq_rope_turns(int32_t rotary_dim, double base, const kvq_rope_scaling *scaling,
                          uint64_t *turns, float *amplitude) {
  if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2 || !turns || !amplitude)
    return KVQ_ERR_ARG;
  return kvq::rope_turns(rotary_dim, base, scaling, turns, amplitude) ? KVQ_OK : KVQ_ERR_ARG;
}

kvq_status kv_rope(const kvq_rope_tensor *tensors, int32_t n_tensors, int32_t dtype,
                   int32_t batch, int32_t n, int32_t head_dim, int32_t rotary_dim, int32_t layout,
                   const uint64_t *turns, float amplitude, int32_t inverse,
                   const int32_t *positions, int32_t *dev_status, kvq_stream_t stream) {
  if (!tensors || n_tensors < 1 || n_tensors > 3) return KVQ_ERR_ARG;
  if (dtype != KVQ_F32 && dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (batch < 0 || n < 0 || head_dim < 32 || head_dim > 256 || head_dim % 32) return KVQ_ERR_ARG;
  if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2) return KVQ_ERR_ARG;
  if (layout != KVQ_ROPE_HALF && layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_ARG;
  if (!turns || !(amplitude > 0.0f)) return KVQ_ERR_ARG;
  const int64_t unit = dtype == KVQ_F32 ? 4 : 8;  // elements in 16 bytes
  kvq::RopeTensors t = {};
  t.n = n_tensors;
  int64_t heads = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const kvq_rope_tensor &x = tensors[i];
    if (x.heads < 1 || x.stride_b < 0 || x.stride_h < 0 || x.stride_t < 0) return KVQ_ERR_ARG;
    heads += x.heads;
  }
  if (heads > 0x7fffffffL) return KVQ_ERR_ARG;
  if (batch == 0 || n == 0) {
    g_last_launches = 0;
    g_last_path = "rope";
    return KVQ_OK;
  }
  if (static_cast<int64_t>(batch) * n > 0x7fffffffL) return KVQ_ERR_UNSUPPORTED;
  if (!positions) return KVQ_ERR_ARG;
  for (int i = 0; i < n_tensors; ++i)
    if (!tensors[i].in || !tensors[i].out) return KVQ_ERR_ARG;
  if (!aligned16(turns) || !aligned16(positions) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  for (int i = 0; i < n_tensors; ++i) {
    const kvq_rope_tensor &x = tensors[i];
    if (!aligned16(x.in) || !aligned16(x.out) || x.stride_b % unit || x.stride_h % unit ||
        x.stride_t % unit)
      return KVQ_ERR_ALIGN;
    t.in[i] = x.in;
    t.out[i] = x.out;
    t.heads[i] = x.heads;
    t.rotate[i] = x.rotate;
    t.sb[i] = x.stride_b;
    t.sh[i] = x.stride_h;
    t.st[i] = x.stride_t;
    ctl_add(ctl, x.in,
            rows_bytes((batch - 1) * x.stride_b + (x.heads - 1) * x.stride_h +
                           (n - 1) * x.stride_t + head_dim, 1, dtype));
    ctl_add(ctl, x.out, rows_bytes(static_cast<long>(batch) * x.heads * n, head_dim, dtype));
  }
  t.total_heads = static_cast<int>(heads);
  ctl_add(ctl, turns, static_cast<size_t>(rotary_dim) * 4);
  ctl_add(ctl, positions, static_cast<size_t>(batch) * n * 4);
  const int k = kvq::launch_rope(t, dtype, batch, n, head_dim, rotary_dim, layout, turns,
                                 amplitude, inverse, positions, ctl, sm_count(),
                                 reinterpret_cast<cudaStream_t>(stream));
  return finish(k, "rope");
}

kvq_status kv_attend_tree(const kvq_cache *cache, const void *q, int32_t q_dtype,
                          int32_t q_heads, int32_t n_tree, const void *k_tree,
                          const void *v_tree, int32_t tree_dtype, const int32_t *parents,
                          float sm_scale, void *out, int32_t out_dtype, void *workspace,
                          size_t *ws_bytes, int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads) return KVQ_ERR_ARG;
  if (n_tree < 1 || n_tree > KVQ_TREE_MAX) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (tree_dtype != KVQ_F32 && tree_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  const int sms = sm_count();
  const bool tensor = kvq::tree_tensor_supported(*cache, q_dtype, tree_dtype, q_heads, n_tree);
  if (!tensor && (q_heads > 65535 || cache->batch > 65535)) return KVQ_ERR_UNSUPPORTED;
  const size_t need = tensor ? kvq::tree_workspace_bytes(*cache, q_heads, n_tree, sms) : 0;
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out || !k_tree || !v_tree || !parents) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_tree) || !aligned16(v_tree) ||
      !aligned16(parents) || !aligned16(workspace) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_tree;
    const long tree = static_cast<long>(cache->batch) * cache->kv_heads * n_tree;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, k_tree, rows_bytes(tree, cache->head_dim, tree_dtype));
    ctl_add(ctl, v_tree, rows_bytes(tree, cache->head_dim, tree_dtype));
    ctl_add(ctl, parents, rows_bytes(cache->batch, n_tree, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tensor) {
    const int n = kvq::launch_attend_tree(*cache, q, q_heads, n_tree, k_tree, v_tree, parents,
                                          static_cast<float>(scale * kLog2e), out, out_dtype,
                                          workspace, ctl, sms, s);
    if (n < 0) return KVQ_ERR_CUDA;
    return finish(n, "tree_tensor");
  }
  const int n = kvq::launch_tree_rows(*cache, q, q_dtype, q_heads, n_tree, k_tree, v_tree,
                                      tree_dtype, parents, scale, out, out_dtype, ctl, s);
  return finish(n, "tree_rows");
}

kvq_status kv_block_summary(const kvq_cache *cache, const kvq_summary *summary,
                            int32_t first_block, int32_t *dev_status, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  st = check_summary(cache, summary);
  if (st != KVQ_OK) return st;
  if (first_block < 0) return KVQ_ERR_ARG;
  if (dev_status && !aligned16(dev_status)) return KVQ_ERR_ALIGN;
  const int blocks = summary_blocks(*cache, summary->block);
  if (first_block >= blocks) {
    g_last_launches = 0;
    g_last_path = "block_summary";
    return KVQ_OK;
  }
  // one warp per block: the grid's x holds 2^31 - 1 CTAs of eight
  if (static_cast<long>(cache->batch) * cache->kv_heads * blocks > 0x7fffffffL)
    return KVQ_ERR_UNSUPPORTED;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_cache(ctl, *cache);
  ctl_add_summary(ctl, *cache, *summary);
  const int n = kvq::launch_block_summary(*cache, *summary, first_block, blocks, ctl,
                                          reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "block_summary");
}

kvq_status kv_block_values(const kvq_cache *cache, const kvq_summary *summary,
                           int32_t first_block, float *values, int32_t *dev_status,
                           kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  st = check_summary(cache, summary);
  if (st != KVQ_OK) return st;
  if (first_block < 0) return KVQ_ERR_ARG;
  if (dev_status && !aligned16(dev_status)) return KVQ_ERR_ALIGN;
  const int blocks = summary_blocks(*cache, summary->block);
  if (first_block >= blocks) {
    g_last_launches = 0;
    g_last_path = "block_values";
    return KVQ_OK;
  }
  if (!values) return KVQ_ERR_ARG;
  if (!aligned16(values)) return KVQ_ERR_ALIGN;
  if (static_cast<long>(cache->batch) * cache->kv_heads * blocks > 0x7fffffffL)
    return KVQ_ERR_UNSUPPORTED;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_summary(ctl, *cache, *summary);
  ctl_add(ctl, values,
          rows_bytes(static_cast<long>(cache->batch) * cache->kv_heads * (blocks - first_block),
                     cache->head_dim, KVQ_F32));
  const int n = kvq::launch_block_values(*cache, *summary, first_block, blocks, values, ctl,
                                         reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "block_values");
}

kvq_status kv_select_blocks(const kvq_cache *cache, const kvq_summary *summary, const void *q,
                            int32_t q_dtype, int32_t q_heads, int32_t n_q, int32_t top_k,
                            int32_t n_sink, int32_t *selected, void *workspace, size_t *ws_bytes,
                            int32_t *dev_status, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  st = check_summary(cache, summary);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1) return KVQ_ERR_ARG;
  if (q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (top_k < 1 || n_sink < 0 || n_sink > top_k) return KVQ_ERR_ARG;
  if (q_heads / cache->kv_heads > kvq::select_max_group()) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<long>(cache->batch) * cache->kv_heads * n_q > 65535) return KVQ_ERR_UNSUPPORTED;
  const int blocks = summary_blocks(*cache, summary->block);
  const size_t need = blocks > top_k ? kvq::select_workspace_bytes(*cache, blocks, n_q) : 0;
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !selected) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(selected) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_summary(ctl, *cache, *summary);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, selected,
            rows_bytes(static_cast<long>(cache->batch) * cache->kv_heads * n_q, top_k, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  const int n = kvq::launch_select_blocks(*cache, *summary, blocks, q, q_dtype, q_heads, n_q,
                                          top_k, n_sink, selected, workspace, ctl,
                                          reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "select_blocks");
}

kvq_status kv_attend_blocks(const kvq_cache *cache, const void *q, int32_t q_dtype,
                            int32_t q_heads, int32_t n_q, const int32_t *selected, int32_t top_k,
                            int32_t block, float sm_scale, void *out, int32_t out_dtype,
                            void *workspace, size_t *ws_bytes, int32_t *dev_status,
                            kvq_stream_t stream) {
  const kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_q < 1 || top_k < 1) return KVQ_ERR_ARG;
  if (block != 32 && block != 64 && block != 128) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  const int sms = sm_count();
  const bool decode = kvq::blocks_decode_supported(*cache, q_dtype, q_heads, n_q, top_k, block);
  if (!decode && (q_heads > 65535 || cache->batch > 65535)) return KVQ_ERR_UNSUPPORTED;
  const size_t need =
      decode ? kvq::blocks_decode_workspace_bytes(*cache, n_q, top_k, block, sms) : 0;
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!q || !out || !selected) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(selected) || !aligned16(workspace) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  {
    const long rows = static_cast<long>(cache->batch) * q_heads * n_q;
    ctl_add_cache(ctl, *cache);
    ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
    ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
    ctl_add(ctl, selected,
            rows_bytes(static_cast<long>(cache->batch) * cache->kv_heads * n_q, top_k, KVQ_F32));
    ctl_add(ctl, workspace, *ws_bytes);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = summary_blocks(*cache, block);
  if (decode) {
    const int n = kvq::launch_attend_blocks(*cache, q, q_heads, n_q, selected, top_k, block,
                                            blocks, static_cast<float>(scale * kLog2e), out,
                                            out_dtype, workspace, ctl, sms, s);
    return finish(n, "blocks_decode");
  }
  const int n = kvq::launch_block_rows(*cache, q, q_dtype, q_heads, n_q, selected, top_k, block,
                                       blocks, scale, out, out_dtype, ctl, s);
  return finish(n, "blocks_rows");
}

kvq_status kvq_paged_sizes(const kvq_paged_cache *cache, size_t sizes[6]) {
  if (!cache || !sizes || !paged_ok(*cache)) return KVQ_ERR_ARG;
  const kvq_page_state &s = cache->state;
  const size_t d = static_cast<size_t>(cache->head_dim), h = static_cast<size_t>(cache->kv_heads);
  const size_t slots = static_cast<size_t>(s.slots), pages = static_cast<size_t>(s.n_pages);
  sizes[0] = 4 * slots * s.max_pages;
  sizes[1] = 4 * slots;
  sizes[2] = 4 * pages;
  sizes[3] = 16;
  sizes[4] = pages * h * (s.page / 32) * 40 * d;
  sizes[5] = slots * h * kvq::paged_tiles(s.window) * 64 * d * elem_bytes(cache->win_dtype);
  return KVQ_OK;
}

int32_t kvq_page_work(const kvq_page_state *s, int32_t rows) {
  if (!s || !page_state_ok(*s) || rows < 0 || rows > (1 << 28)) return 0;
  return kvq::page_work_bound(s->window, s->slots, rows);
}

kvq_status kv_page_tables(const kvq_page_state *state, const int32_t *n_new,
                          const kvq_page_plan *plan, int32_t advance, int32_t *dev_status,
                          kvq_stream_t stream) {
  kvq_status st = check_page_state(state);
  if (st != KVQ_OK) return st;
  st = check_plan(*state, plan);
  if (st != KVQ_OK) return st;
  if (!n_new) return KVQ_ERR_ARG;
  if (!aligned16(n_new) || (dev_status && !aligned16(dev_status))) return KVQ_ERR_ALIGN;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  const size_t slots = static_cast<size_t>(state->slots);
  ctl_add(ctl, state->table, 4 * slots * state->max_pages);
  ctl_add(ctl, state->lengths, 4 * slots);
  ctl_add(ctl, state->free_pages, 4 * static_cast<size_t>(state->n_pages));
  ctl_add(ctl, state->n_free, 16);
  ctl_add(ctl, n_new, 4 * slots);
  ctl_add_plan(ctl, *state, *plan);
  ctl_add(ctl, plan->row_slot, 4 * static_cast<size_t>(plan->rows));
  ctl_add(ctl, plan->positions, 4 * static_cast<size_t>(plan->rows));
  const int n = kvq::launch_page_tables(*state, n_new, *plan, advance != 0, ctl, sm_count(),
                                        reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "page_tables");
}

kvq_status kv_append_pages(const kvq_paged_cache *cache, const kvq_page_plan *plan,
                           const kvq_page_rows *rows, int32_t in_dtype, int32_t *dev_status,
                           kvq_stream_t stream) {
  kvq_status st = check_paged(cache);
  if (st != KVQ_OK) return st;
  st = check_plan(cache->state, plan);
  if (st != KVQ_OK) return st;
  if (!rows || (in_dtype != KVQ_F32 && in_dtype != KVQ_BF16)) return KVQ_ERR_ARG;
  if (rows->k_stride_row < 0 || rows->k_stride_head < 0 || rows->v_stride_row < 0 ||
      rows->v_stride_head < 0)
    return KVQ_ERR_ARG;
  if (plan->rows == 0) {
    g_last_launches = 0;
    g_last_path = "append_pages";
    return KVQ_OK;
  }
  if (!rows->k_new || !rows->v_new) return KVQ_ERR_ARG;
  const int64_t unit = in_dtype == KVQ_F32 ? 4 : 8;  // elements in 16 bytes
  if (!aligned16(rows->k_new) || !aligned16(rows->v_new) || rows->k_stride_row % unit ||
      rows->k_stride_head % unit || rows->v_stride_row % unit || rows->v_stride_head % unit ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const int64_t most = 0x7fffffffL;
  if (2 * static_cast<int64_t>(plan->cap_work) * cache->kv_heads > most || rows->k_stride_row > most ||
      rows->k_stride_head > most || rows->v_stride_row > most || rows->v_stride_head > most)
    return KVQ_ERR_UNSUPPORTED;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_pages(ctl, *cache);
  ctl_add_plan(ctl, cache->state, *plan);
  const int64_t n1 = plan->rows - 1, h1 = cache->kv_heads - 1;
  ctl_add(ctl, rows->k_new,
          rows_bytes(n1 * rows->k_stride_row + h1 * rows->k_stride_head + cache->head_dim, 1,
                     in_dtype));
  ctl_add(ctl, rows->v_new,
          rows_bytes(n1 * rows->v_stride_row + h1 * rows->v_stride_head + cache->head_dim, 1,
                     in_dtype));
  const kvq::PageRows r = {rows->k_new,
                           rows->v_new,
                           static_cast<int>(rows->k_stride_row),
                           static_cast<int>(rows->k_stride_head),
                           static_cast<int>(rows->v_stride_row),
                           static_cast<int>(rows->v_stride_head),
                           in_dtype};
  const int n = kvq::launch_append_pages(kvq::paged_dims(*cache), *plan, r, ctl, sm_count(),
                                         reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "append_pages");
}

kvq_status kv_page_values(const kvq_paged_cache *cache, const int32_t *row_slot,
                          const int32_t *positions, int32_t n_rows, void *k, void *v,
                          int32_t out_dtype, int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_paged(cache);
  if (st != KVQ_OK) return st;
  if (n_rows < 0 || n_rows > (1 << 28) || (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (n_rows == 0) {
    g_last_launches = 0;
    g_last_path = "page_values";
    return KVQ_OK;
  }
  if (!row_slot || !positions || !k || !v) return KVQ_ERR_ARG;
  if (static_cast<long>(n_rows) * cache->kv_heads > 1L << 34) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(row_slot) || !aligned16(positions) || !aligned16(k) || !aligned16(v) ||
      (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  kvq::KernelCtl ctl = make_ctl(dev_status);
  ctl_add_pages(ctl, *cache);
  ctl_add(ctl, row_slot, 4 * static_cast<size_t>(n_rows));
  ctl_add(ctl, positions, 4 * static_cast<size_t>(n_rows));
  const size_t bytes = rows_bytes(static_cast<long>(n_rows) * cache->kv_heads, cache->head_dim,
                                  out_dtype);
  ctl_add(ctl, k, bytes);
  ctl_add(ctl, v, bytes);
  const int n = kvq::launch_page_values(kvq::paged_dims(*cache), row_slot, positions, n_rows, k, v,
                                        out_dtype, ctl,
                                        reinterpret_cast<cudaStream_t>(stream));
  return finish(n, "page_values");
}

kvq_status kv_attend_pages(const kvq_paged_cache *cache, const void *q, int32_t q_dtype,
                           int32_t q_heads, int32_t n_rows, const int32_t *row_slot,
                           const int32_t *positions, float sm_scale, void *out,
                           int32_t out_dtype, void *workspace, size_t *ws_bytes,
                           int32_t *dev_status, kvq_stream_t stream) {
  const kvq_status st = check_paged(cache);
  if (st != KVQ_OK) return st;
  if (!ws_bytes) return KVQ_ERR_ARG;
  if (q_heads < 1 || q_heads % cache->kv_heads || n_rows < 0 || n_rows > 65535) return KVQ_ERR_ARG;
  if (!row_slot && n_rows > cache->state.slots) return KVQ_ERR_ARG;
  if ((q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) ||
      (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16))
    return KVQ_ERR_ARG;
  if (q_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  const int sms = sm_count();
  const kvq::PagedDims d = kvq::paged_dims(*cache);
  const bool tensor = kvq::attend_pages_supported(d, q_heads, n_rows);
  const size_t need = n_rows == 0 ? 0
                      : tensor    ? kvq::attend_pages_workspace(d, q_heads, n_rows, sms)
                                  : kvq::page_rows_workspace(d, q_heads, n_rows, sms);
  if (!workspace) {
    *ws_bytes = need;
    return KVQ_OK;
  }
  if (*ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (n_rows == 0) {
    g_last_launches = 0;
    g_last_path = tensor ? "pages_tensor" : "pages_rows";
    return KVQ_OK;
  }
  if (!q || !out) return KVQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned16(row_slot) ||
      !aligned16(positions) || (dev_status && !aligned16(dev_status)))
    return KVQ_ERR_ALIGN;
  const float scale = resolve_scale(sm_scale, cache->head_dim);
  kvq::KernelCtl ctl = make_ctl(dev_status);
  const long rows = static_cast<long>(n_rows) * q_heads;
  ctl_add_pages(ctl, *cache);
  ctl_add(ctl, q, rows_bytes(rows, cache->head_dim, q_dtype));
  ctl_add(ctl, out, rows_bytes(rows, cache->head_dim, out_dtype));
  ctl_add(ctl, row_slot, 4 * static_cast<size_t>(n_rows));
  ctl_add(ctl, positions, 4 * static_cast<size_t>(n_rows));
  ctl_add(ctl, workspace, *ws_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tensor) {
    const int n = kvq::launch_attend_pages(d, q, q_dtype, q_heads, n_rows, row_slot, positions,
                                           static_cast<float>(scale * kLog2e), out, out_dtype,
                                           workspace, ctl, sms, s);
    return finish(n, "pages_tensor");
  }
  const int n = kvq::launch_page_rows(d, q, q_dtype, q_heads, n_rows, row_slot, positions, scale,
                                      out, out_dtype, workspace, ctl, sms, s);
  return finish(n, "pages_rows");
}

int32_t kvq_last_launch_count(void) { return g_last_launches; }

const char *kvq_last_path(void) { return g_last_path; }

int32_t kvq_debug_checks(void) {
#ifdef KVQ_DEBUG
  return 1;
#else
  return 0;
#endif
}

void kvq_debug_set(uint32_t wait_limit_ns, int32_t drop_item) {
  g_wait_limit_ns = wait_limit_ns;
  g_drop_item = drop_item;
}

}  // extern "C"
