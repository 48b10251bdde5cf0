// The paged cache's arithmetic, shared by its kernels and the C ABI layer: what a
// request's length says about where its tokens are, and where the elements of a page's
// records and of a window's tiles lie (include/kvq.h, kvq_paged_cache).
#pragma once

#include <type_traits>

#include "kvq_internal.h"

namespace kvq {

__host__ __device__ __forceinline__ int paged_cut(int len, int window) {
  return len >= window ? ((len - window) >> 5) << 5 : 0;
}
__host__ __device__ __forceinline__ int paged_tiles(int window) { return (window + 63) >> 5; }
// Pages that hold a request's int4 tokens (unsigned: any length may be asked about).
__host__ __device__ __forceinline__ int paged_pages(int len, int window, int page_log2) {
  const uint32_t cut = static_cast<uint32_t>(paged_cut(len, window));
  return static_cast<int>((cut + (1u << page_log2) - 1u) >> page_log2);
}

// Shape and arrays of one layer's cache, as kernels take them.
struct PagedDims {
  int slots, n_pages, page_log2, max_pages, window, tiles;
  int Hkv, D, win_dt;
  const int32_t *table;
  const int32_t *lengths;
  uint8_t *pool;
  void *ring;

  __host__ __device__ __forceinline__ int gpp_log2() const { return page_log2 - 5; }
  __host__ __device__ __forceinline__ int record() const { return 40 * D; }
  // whether a table row can hold a request of this length
  __host__ __device__ __forceinline__ bool holds(int len) const {
    return len >= 0 && paged_pages(len, window, page_log2) <= max_pages;
  }
  // record of group g (of its page) and head h
  __host__ __device__ __forceinline__ uint8_t *record_at(int page, int sub, int h) const {
    return pool + (((static_cast<size_t>(page) * Hkv + h) << gpp_log2()) + sub) * record();
  }
  // first element of the window tile that holds group g of slot s, head h (K; V is 32 D on)
  __host__ __device__ __forceinline__ size_t tile_at(int s, int h, int g) const {
    return ((static_cast<size_t>(s) * Hkv + h) * tiles + g % tiles) * (64 * static_cast<size_t>(D));
  }
};

inline PagedDims paged_dims(const kvq_paged_cache &c) {
  PagedDims d;
  d.slots = c.state.slots;
  d.n_pages = c.state.n_pages;
  d.page_log2 = c.state.page == 32 ? 5 : c.state.page == 64 ? 6 : 7;
  d.max_pages = c.state.max_pages;
  d.window = c.state.window;
  d.tiles = paged_tiles(c.state.window);
  d.Hkv = c.kv_heads;
  d.D = c.head_dim;
  d.win_dt = c.win_dtype;
  d.table = c.state.table;
  d.lengths = c.state.lengths;
  d.pool = c.pool;
  d.ring = c.ring;
  return d;
}

// Entries of the work list of a step: a request with n new tokens writes at most n / 32
// groups and its window's tiles and a part of a group at either end, and no more than two
// groups for each token.
inline int page_work_bound(int window, int slots, int rows) {
  const int64_t requests = slots < rows ? slots : rows;
  const int64_t most = rows / 32 + (paged_tiles(window) + 3) * requests;
  return static_cast<int>(most < 2 * static_cast<int64_t>(rows) ? most : 2 * static_cast<int64_t>(rows));
}

// ---- a group's record: byte offsets of its four parts
__host__ __device__ __forceinline__ int rec_kscale(int D) { return 16 * D; }
__host__ __device__ __forceinline__ int rec_vcode(int D) { return 20 * D; }
__host__ __device__ __forceinline__ int rec_vscale(int D) { return 36 * D; }

// K scale of channel c: the order in which a lane of the score MMAs reads them.
__host__ __device__ __forceinline__ int kscale_at(int c, int D) {
  const int t = c / (D / 4), r = c - t * (D / 4), i = r >> 3, k = r & 7;
  return (2 * i + (k >> 1 & 1)) * 16 + 4 * t + 2 * (k & 1) + (k >> 2);
}
// V code word (m, g, t, f).
__host__ __device__ __forceinline__ int vword_at(int m, int g, int t, int f, int D) {
  const int cl = D % 64 == 0 ? 2 : 1;  // log2 of the words a lane has side by side
  return (((m * ((D / 16) >> cl) + (f >> cl)) * 32 + 4 * g + t) << cl) + (f & ((1 << cl) - 1));
}
// V scale of token t (of the group) and 32-feature block b.
__host__ __device__ __forceinline__ int vscale_at(int t, int b, int D) {
  return (((t >> 3) * 4 + ((t & 7) >> 1)) * (D / 32) + b) * 2 + (t & 1);
}

// ---- a window tile: element offsets
__host__ __device__ __forceinline__ int ringk_at(int r, int c, int D) {
  const int t = c / (D / 4), q = c - t * (D / 4), i = q >> 3, k = q & 7;
  const int x = D % 64 == 0 ? r & 1 : 0;
  return r * D + ((i ^ x) * 4 + t) * 8 + 2 * (k & 3) + (k >> 2);
}
__host__ __device__ __forceinline__ int ringv_at(int r, int d, int D) {
  const int b = d >> 5, j = (d >> 3) & 3, g = d & 7;
  return (((((r >> 3) * (D / 32) + b) * 8 + g) * 4 + ((r & 7) >> 1)) * 4 + j) * 2 + (r & 1);
}

// ---- launchers (arguments are already validated)
struct PageRows {
  const void *k, *v;
  int ksr, ksh, vsr, vsh;  // strides in elements
  int dtype;
};
int launch_page_tables(const kvq_page_state &st, const int32_t *n_new, const kvq_page_plan &p,
                       int advance, const KernelCtl &ctl, int num_sms, cudaStream_t s);
int launch_append_pages(const PagedDims &d, const kvq_page_plan &p, const PageRows &r,
                        const KernelCtl &ctl, int num_sms, cudaStream_t s);
int launch_page_values(const PagedDims &d, const int32_t *slot, const int32_t *pos, int n,
                       void *k, void *v, int out_dt, const KernelCtl &ctl, cudaStream_t s);
bool attend_pages_supported(const PagedDims &d, int Hq, int rows);
size_t attend_pages_workspace(const PagedDims &d, int Hq, int rows, int num_sms);
int launch_attend_pages(const PagedDims &d, const void *q, int q_dt, int Hq, int rows,
                        const int32_t *slot, const int32_t *pos, float scale_log2, void *out,
                        int out_dt, void *ws, const KernelCtl &ctl, int num_sms, cudaStream_t s);
int launch_page_rows(const PagedDims &d, const void *q, int q_dt, int Hq, int rows,
                     const int32_t *slot, const int32_t *pos, float scale, void *out, int out_dt,
                     void *ws, const KernelCtl &ctl, int num_sms, cudaStream_t s);
size_t page_rows_workspace(const PagedDims &d, int Hq, int rows, int num_sms);

}  // namespace kvq
