// kv_page_tables: one step's block tables, slot map and list of groups, from the
// requests' lengths (include/kvq.h states the rules).
//
// Everything is a sum over the requests in slot order: the first row of a request is the
// sum of the new tokens before it, the first page it takes the sum of the pages asked for
// before it, and so on. Each CTA takes the sums of all requests (a few thousand integers,
// in shared memory) and then its share of the rows, pages and groups, each found by a
// binary search over the sums; the tables of a decoding step are one CTA. Nothing is
// ordered by atomics, so the tables are a function of the inputs. The lengths and the
// count of free pages are written by the CTA that is the last to have read them.
#include <algorithm>

#include "paged.cuh"

namespace kvq {
namespace {

struct TablesArgs {
  int32_t *table, *lengths, *free_pages, *n_free;
  const int32_t *n_new;
  int32_t *offsets, *before, *after, *row_slot, *positions, *work, *counts;
  int S, n_pages, page_log2, max_pages, window, rows, cap_work, advance;
  KernelCtl ctl;
};

// Exclusive sum over the block's threads; *total receives the sum of all.
__device__ __forceinline__ long long block_sum(long long x, long long *buf, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // (buf may still be read from the sum before)
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < warps ? buf[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += y;
    }
    buf[lane] = w;
  }
  __syncthreads();
  *total = buf[31];
  return v - x + (warp ? buf[warp - 1] : 0);
}

// Last index i in [0, n) with sum[i] <= k.
__device__ __forceinline__ int find_run(const int *sum, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(const TablesArgs &a, int len) {
  return (paged_cut(len, a.window) + (1 << a.page_log2) - 1) >> a.page_log2;
}

__device__ __forceinline__ bool holds(const TablesArgs &a, int len) {
  return len >= 0 && pages_of(a, len) <= a.max_pages;
}

__device__ __forceinline__ int clamp_int(long long x) {
  return static_cast<int>(x < 0x7fffffffLL ? x : 0x7fffffffLL);
}

__device__ __forceinline__ int load_entry(const TablesArgs &a, const int32_t *e) {
  return in_bounds(a.ctl, e, 4) ? *e : -1;
}

// The k-th page that the step takes: from the top of the free ones, on which the pages of
// ended requests (their sums in backp) are put first.
__device__ __forceinline__ int taken_page(const TablesArgs &a, const int *backp, int k, int n_free,
                                          long long have) {
  const long long at = have - 1 - k;
  if (at < n_free) return load_entry(a, a.free_pages + at);
  const int j = static_cast<int>(at - n_free), b = find_run(backp, a.S, j);
  return load_entry(a, a.table + static_cast<size_t>(b) * a.max_pages + (j - backp[b]));
}

__global__ void __launch_bounds__(1024) page_tables_kernel(const TablesArgs a) {
  extern __shared__ int sm[];
  __shared__ long long buf[32];
  __shared__ int last;
  const int S = a.S;
  int *rowp = sm, *takep = rowp + S + 1, *backp = takep + S + 1, *workp = backp + S + 1;
  int *bef = workp + S + 1, *aft = bef + S;
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  wait_prior_grid();
  allow_next_grid();

  // what each request asks for: aft[s] holds n_new until it is decided
  long long rows = 0, back = 0, total;
  for (int s = s0; s < s1; ++s) {
    int len = 0, n = 0;
    if (in_bounds(a.ctl, a.lengths + s, 4)) len = a.lengths[s];
    if (in_bounds(a.ctl, a.n_new + s, 4)) n = a.n_new[s];
    if (!holds(a, len) || n < -1) {
      if (blockIdx.x == 0) flag_error(a.ctl, KVQ_DEV_INDEX);
      n = max(n, 0);  // (its rows stand for none)
    }
    bef[s] = len;
    aft[s] = n;
    rows += max(n, 0);
    if (n == -1) back += pages_of(a, len);
  }
  int n_free = 0;
  if (in_bounds(a.ctl, a.n_free, 4)) n_free = min(max(a.n_free[0], 0), a.n_pages);
  long long row_at = block_sum(rows, buf, &total);
  if (threadIdx.x == 0) rowp[S] = clamp_int(total);
  long long back_total;
  long long back_at = block_sum(back, buf, &back_total);
  if (threadIdx.x == 0) backp[S] = clamp_int(back_total);
  long long take = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = aft[s], len = bef[s];
    rowp[s] = clamp_int(row_at);
    backp[s] = clamp_int(back_at);
    row_at += max(n, 0);
    if (n == -1) back_at += pages_of(a, len);
    if (n > 0) {
      int bit = 0;
      const long long grown = static_cast<long long>(len) + n;
      if (row_at > a.rows || !holds(a, len))
        bit = KVQ_DEV_INDEX;
      else if (grown > 0x7fffffffLL || pages_of(a, static_cast<int>(grown)) > a.max_pages)
        bit = KVQ_DEV_PAGES;
      if (bit) {
        if (blockIdx.x == 0) flag_error(a.ctl, bit);
        aft[s] = 0;
      } else {
        take += pages_of(a, static_cast<int>(grown)) - pages_of(a, len);
      }
    }
  }
  // pages: served while the sum of what is asked for does not pass what there is
  const long long have = n_free + back_total;
  long long take_at = block_sum(take, buf, &total);
  long long work = 0, served = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = aft[s], len = bef[s];
    takep[s] = clamp_int(take_at < have ? take_at : have);
    int end = n == -1 ? 0 : len;
    if (n > 0) {
      const int need = pages_of(a, len + n) - pages_of(a, len);
      take_at += need;
      if (need > 0 && take_at > have) {
        if (blockIdx.x == 0) flag_error(a.ctl, KVQ_DEV_PAGES);
      } else {
        end = len + n;
        served += need;
        const int c0 = paged_cut(len, a.window) >> 5, c1 = paged_cut(end, a.window) >> 5;
        work += c1 - c0 + max(0, ((end + 31) >> 5) - max(len >> 5, c1));
      }
    }
    aft[s] = end;
  }
  // (requests that were refused come behind the served ones in the sum of pages)
  long long work_at = block_sum(work, buf, &total);
  if (threadIdx.x == 0) workp[S] = clamp_int(total);
  for (int s = s0; s < s1; ++s) {
    const int len = bef[s], end = aft[s];
    workp[s] = clamp_int(work_at);
    if (end > len) {
      const int c0 = paged_cut(len, a.window) >> 5, c1 = paged_cut(end, a.window) >> 5;
      work_at += c1 - c0 + max(0, ((end + 31) >> 5) - max(len >> 5, c1));
    }
  }
  long long served_total;
  block_sum(served, buf, &served_total);
  if (threadIdx.x == 0) takep[S] = clamp_int(served_total);
  __syncthreads();

  // the state is read: whoever is last moves it on
  if (threadIdx.x == 0) {
    last = 1;
    if (gridDim.x > 1) {
      __threadfence();
      last = 0;
      if (in_bounds(a.ctl, a.counts, 16))
        last = atomicAdd(a.counts + 2, 1) == static_cast<int>(gridDim.x) - 1;
      if (last) a.counts[2] = 0;
    }
  }
  __syncthreads();
  const int n_work = min(workp[S], a.cap_work), n_back = backp[S], n_take = takep[S];
  if (last) {
    for (int s = threadIdx.x; s <= S; s += blockDim.x) {
      if (in_bounds(a.ctl, a.offsets + s, 4)) a.offsets[s] = rowp[s];
      if (s == S) break;
      if (in_bounds(a.ctl, a.before + s, 4)) a.before[s] = bef[s];
      if (in_bounds(a.ctl, a.after + s, 4)) a.after[s] = aft[s];
      if (a.advance && aft[s] != bef[s] && in_bounds(a.ctl, a.lengths + s, 4))
        a.lengths[s] = aft[s];
    }
    if (threadIdx.x == 0) {
      const int left = static_cast<int>(min(have - n_take, static_cast<long long>(a.n_pages)));
      if (in_bounds(a.ctl, a.counts, 16)) {
        a.counts[0] = left;
        a.counts[1] = n_work;
      }
      if (a.advance && in_bounds(a.ctl, a.n_free, 4)) a.n_free[0] = left;
    }
  }

  const int t0 = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  // rows
  for (int r = t0; r < a.rows; r += step) {
    int slot = -1, pos = 0;
    if (r < rowp[S]) {
      const int s = find_run(rowp, S, r);
      if (aft[s] > bef[s]) {
        slot = s;
        pos = bef[s] + r - rowp[s];
      }
    }
    if (in_bounds(a.ctl, a.row_slot + r, 4)) a.row_slot[r] = slot;
    if (in_bounds(a.ctl, a.positions + r, 4)) a.positions[r] = pos;
  }
  // groups to write: those that are packed, then those of the window
  for (int k = t0; k < n_work; k += step) {
    const int s = find_run(workp, S, k), e = k - workp[s];
    const int c0 = paged_cut(bef[s], a.window) >> 5, c1 = paged_cut(aft[s], a.window) >> 5;
    const int g = e < c1 - c0 ? c0 + e : max(bef[s] >> 5, c1) + e - (c1 - c0);
    int page = -1;
    if (g < c1) {
      const int j = g >> (a.page_log2 - 5), held = pages_of(a, bef[s]);
      page = j < held ? load_entry(a, a.table + static_cast<size_t>(s) * a.max_pages + j)
                      : taken_page(a, backp, takep[s] + j - held, n_free, have);
    }
    int4 *o = reinterpret_cast<int4 *>(a.work + 8 * static_cast<size_t>(k));
    if (in_bounds(a.ctl, o, 32)) {
      o[0] = make_int4(s, g, page, bef[s]);
      o[1] = make_int4(aft[s], rowp[s], 0, 0);
    }
  }
  // pages of ended requests go on top of the free ones
  for (int k = t0; k < n_back; k += step) {
    const int s = find_run(backp, S, k);
    const int32_t *e = a.table + static_cast<size_t>(s) * a.max_pages + (k - backp[s]);
    if (n_free + k < a.n_pages && in_bounds(a.ctl, e, 4) &&
        in_bounds(a.ctl, a.free_pages + n_free + k, 4))
      a.free_pages[n_free + k] = *e;
  }
  // and requests that grow take from the top
  for (int k = t0; k < n_take; k += step) {
    const int s = find_run(takep, S, k);
    const int page = taken_page(a, backp, k, n_free, have);
    int32_t *o = a.table + static_cast<size_t>(s) * a.max_pages + pages_of(a, bef[s]) +
                 (k - takep[s]);
    if (in_bounds(a.ctl, o, 4)) *o = page;
  }
}

}  // namespace

int launch_page_tables(const kvq_page_state &st, const int32_t *n_new, const kvq_page_plan &p,
                       int advance, const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  TablesArgs a;
  a.table = st.table;
  a.lengths = st.lengths;
  a.free_pages = st.free_pages;
  a.n_free = st.n_free;
  a.n_new = n_new;
  a.offsets = p.offsets;
  a.before = p.before;
  a.after = p.after;
  a.row_slot = p.row_slot;
  a.positions = p.positions;
  a.work = p.work;
  a.counts = p.counts;
  a.S = st.slots;
  a.n_pages = st.n_pages;
  a.page_log2 = st.page == 32 ? 5 : st.page == 64 ? 6 : 7;
  a.max_pages = st.max_pages;
  a.window = st.window;
  a.rows = p.rows;
  a.cap_work = p.cap_work;
  a.advance = advance;
  a.ctl = ctl;
  const int threads = st.slots <= 256 ? 256 : 1024;
  const int grid = std::max(1, std::min(num_sms, (p.rows + 2 * threads - 1) / (2 * threads)));
  const size_t smem = sizeof(int) * (6 * static_cast<size_t>(st.slots) + 4);
  if (smem > 48 * 1024) opt_in_smem(page_tables_kernel, smem);
  launch_dependent(page_tables_kernel, dim3(grid), dim3(threads), smem, s, a);
  return 1;
}

}  // namespace kvq
