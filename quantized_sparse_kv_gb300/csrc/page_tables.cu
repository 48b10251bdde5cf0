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
//
// Who is served depends on the sums themselves (the rows and the pages that are left). When
// there are rows and pages for all that is asked for, as in the usual step, one sum of
// four numbers says it; only else two more follow, of what the requests before were granted.
//
// 64 requests of a decoding step: 3.3 us (3.8 with three sums), a launch and a row of
// dependent steps (two loads, a sum, a search, a write). 1,024 requests with 24 prompts, 99,151
// rows: 6.2 us (6.7).
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

// Sums stop at kMost: whatever n_new holds, they fit 32 bits and keep their order (the sum
// of the smaller of a sum and kMost is the same in any grouping). Rows and pages end at 2^28.
constexpr uint32_t kMost = 1u << 30;
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// Exclusive sums of N numbers over the block's threads and, in t, the sums of all. One
// barrier: every call has a buffer of its own.
template <int N>
struct SumBuffer {
  uint32_t x[N][32];
};
template <int N>
__device__ __forceinline__ void block_sums(uint32_t (&x)[N], uint32_t (&t)[N], SumBuffer<N> &buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const auto scan = [lane](uint32_t (&y)[N]) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t p = __shfl_up_sync(~0u, y[i], o);
        if (lane >= o) y[i] = add(y[i], p);
      }
  };
  scan(x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (lane == 31) buf.x[i][warp] = x[i];
    x[i] = __shfl_up_sync(~0u, x[i], 1);
    if (lane == 0) x[i] = 0;
  }
  __syncthreads();
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = lane < warps ? buf.x[i][lane] : 0;
  scan(w);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = __shfl_sync(~0u, w[i], 31);
    const uint32_t p = __shfl_sync(~0u, w[i], max(warp - 1, 0));
    if (warp) x[i] = add(x[i], p);
  }
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
  return paged_pages(len, a.window, a.page_log2);
}

__device__ __forceinline__ bool holds(const TablesArgs &a, int len) {
  return len >= 0 && pages_of(a, len) <= a.max_pages;
}

// Groups that a request's step from len to end tokens writes, in pages and window.
__device__ __forceinline__ int groups_of(const TablesArgs &a, int len, int end) {
  if (end <= len) return 0;
  const int c0 = paged_cut(len, a.window) >> 5, c1 = paged_cut(end, a.window) >> 5;
  return c1 - c0 + max(0, ((end + 31) >> 5) - max(len >> 5, c1));
}

// The length that a request of n new tokens asks for: its own when it rests or cannot be
// served whatever the others ask for (bit: why).
__device__ __forceinline__ int asked(const TablesArgs &a, int len, int n, int &bit) {
  bit = 0;
  if (n <= 0) return n == -1 ? 0 : len;
  const uint32_t grown = static_cast<uint32_t>(len) + static_cast<uint32_t>(n);
  if (!holds(a, len))
    bit = KVQ_DEV_INDEX;
  else if (grown > 0x7fffffffu || pages_of(a, static_cast<int>(grown)) > a.max_pages)
    bit = KVQ_DEV_PAGES;
  return bit ? len : static_cast<int>(grown);
}
// Sums that are taken of the requests: rows, pages that come back, pages asked for, groups.
__device__ __forceinline__ void count(const TablesArgs &a, int len, int n, int end, uint32_t (&x)[4]) {
  x[0] = add(x[0], min(static_cast<uint32_t>(max(n, 0)), kMost));
  if (n == -1) x[1] = add(x[1], pages_of(a, len));
  if (end > len) {
    x[2] = add(x[2], pages_of(a, end) - pages_of(a, len));
    x[3] = add(x[3], groups_of(a, len, end));
  }
}

__device__ __forceinline__ int load_entry(const TablesArgs &a, const int32_t *e) {
  return in_bounds(a.ctl, e, 4) ? *e : -1;
}

// The k-th page that the step takes: from the top of the free ones, on which the pages of
// ended requests (their sums in backp) are put first.
__device__ __forceinline__ int taken_page(const TablesArgs &a, const int *backp, int k, int n_free,
                                          int have) {
  const int at = have - 1 - k;
  if (at < n_free) return load_entry(a, a.free_pages + at);
  const int j = at - n_free, b = find_run(backp, a.S, j);
  return load_entry(a, a.table + static_cast<size_t>(b) * a.max_pages + (j - backp[b]));
}

__global__ void __launch_bounds__(1024) page_tables_kernel(const TablesArgs a) {
  extern __shared__ int sm[];
  __shared__ SumBuffer<4> buf4;
  __shared__ SumBuffer<1> buf1;
  __shared__ SumBuffer<2> buf2;
  __shared__ int last;
  const int S = a.S;
  int *rowp = sm, *takep = rowp + S + 1, *backp = takep + S + 1, *workp = backp + S + 1;
  int *bef = workp + S + 1, *aft = bef + S;
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  wait_prior_grid();
  allow_next_grid();

  // what each request asks for: aft[s] holds n_new until it is decided
  uint32_t x[4] = {0, 0, 0, 0}, total[4];
  int n_free = 0, bit;
  if (in_bounds(a.ctl, a.n_free, 4)) n_free = min(max(a.n_free[0], 0), a.n_pages);
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
    count(a, len, n, asked(a, len, n, bit), x);
  }
  block_sums(x, total, buf4);
  const uint32_t have = min(n_free + total[1], kMost - 1);
  int n_back = total[1], n_take = total[2], work_total = total[3];
  if (total[0] <= static_cast<uint32_t>(a.rows) && total[2] <= have) {
    // the usual step: there are rows and pages for all
    for (int s = s0; s < s1; ++s) {
      const int n = aft[s], len = bef[s], end = asked(a, len, n, bit);
      if (bit && blockIdx.x == 0) flag_error(a.ctl, bit);
      rowp[s] = x[0];
      backp[s] = x[1];
      takep[s] = x[2];
      workp[s] = x[3];
      count(a, len, n, end, x);
      aft[s] = end;
    }
  } else {
    uint32_t take[1] = {0}, take_total[1];
    for (int s = s0; s < s1; ++s) {
      const int n = aft[s], len = bef[s];
      rowp[s] = x[0];
      backp[s] = x[1];
      count(a, len, n, len, x);
      if (n > 0) {
        const int end = asked(a, len, n, bit);
        if (x[0] > static_cast<uint32_t>(a.rows)) bit = KVQ_DEV_INDEX;
        if (bit) {
          if (blockIdx.x == 0) flag_error(a.ctl, bit);
          aft[s] = 0;
        } else {
          take[0] = add(take[0], pages_of(a, end) - pages_of(a, len));
        }
      }
    }
    // pages: served while the sum of what is asked for does not pass what there is
    block_sums(take, take_total, buf1);
    uint32_t y[2] = {0, 0}, served[2];  // pages, groups
    for (int s = s0; s < s1; ++s) {
      const int n = aft[s], len = bef[s];
      takep[s] = min(take[0], have);
      int end = n == -1 ? 0 : len;
      if (n > 0) {
        const int need = pages_of(a, len + n) - pages_of(a, len);
        take[0] = add(take[0], need);
        if (need > 0 && take[0] > have) {
          if (blockIdx.x == 0) flag_error(a.ctl, KVQ_DEV_PAGES);
        } else {
          end = len + n;
          y[0] = add(y[0], need);
          y[1] = add(y[1], groups_of(a, len, end));
        }
      }
      aft[s] = end;
    }
    // (requests that were refused come behind the served ones in the sum of pages)
    block_sums(y, served, buf2);
    for (int s = s0; s < s1; ++s) {
      workp[s] = y[1];
      y[1] = add(y[1], groups_of(a, bef[s], aft[s]));
    }
    n_take = served[0];
    work_total = served[1];
  }
  if (threadIdx.x == 0) {
    rowp[S] = total[0];
    backp[S] = n_back;
    takep[S] = n_take;
    workp[S] = work_total;
  }
  __syncthreads();
  const int n_work = min(work_total, a.cap_work);

  // the state is read: the CTA that is the last to have done so moves it on. (Its count
  // comes back while the tables are written.)
  int arrived = 0;
  if (threadIdx.x == blockDim.x - 1 && gridDim.x > 1 && in_bounds(a.ctl, a.counts, 16)) {
    __threadfence();
    arrived = atomicAdd(a.counts + 2, 1);
  }
  if (blockIdx.x == 0) {
    for (int s = threadIdx.x; s <= S; s += blockDim.x) {
      if (in_bounds(a.ctl, a.offsets + s, 4)) a.offsets[s] = rowp[s];
      if (s == S) break;
      if (in_bounds(a.ctl, a.before + s, 4)) a.before[s] = bef[s];
      if (in_bounds(a.ctl, a.after + s, 4)) a.after[s] = aft[s];
    }
  }

  // Rows, groups and pages, each from another thread on: those of one kind are few, and a
  // thread that has one of each would wait for four chains of loads in a row.
  const int t0 = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
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
  for (int k = step - 1 - t0; k < n_work; k += step) {
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
  for (int k = (t0 + step / 2) % step; k < n_back; k += step) {
    const int s = find_run(backp, S, k);
    const int32_t *e = a.table + static_cast<size_t>(s) * a.max_pages + (k - backp[s]);
    if (n_free + k < a.n_pages && in_bounds(a.ctl, e, 4) &&
        in_bounds(a.ctl, a.free_pages + n_free + k, 4))
      a.free_pages[n_free + k] = *e;
  }
  // and requests that grow take from the top
  for (int k = (t0 + step / 4) % step; k < n_take; k += step) {
    const int s = find_run(takep, S, k);
    const int page = taken_page(a, backp, k, n_free, have);
    int32_t *o = a.table + static_cast<size_t>(s) * a.max_pages + pages_of(a, bef[s]) +
                 (k - takep[s]);
    if (in_bounds(a.ctl, o, 4)) *o = page;
  }

  if (threadIdx.x == blockDim.x - 1) last = arrived == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  const int left = min(static_cast<int>(have) - n_take, a.n_pages);
  if (a.advance)
    for (int s = threadIdx.x; s < S; s += blockDim.x)
      if (aft[s] != bef[s] && in_bounds(a.ctl, a.lengths + s, 4)) a.lengths[s] = aft[s];
  if (threadIdx.x == 0) {
    if (in_bounds(a.ctl, a.counts, 16)) {
      a.counts[0] = left;
      a.counts[1] = n_work;
      a.counts[2] = 0;
    }
    if (a.advance && in_bounds(a.ctl, a.n_free, 4)) a.n_free[0] = left;
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
  // (1,024 slots: 512 threads 0.5 us faster than 256, 1.1 than 1,024)
  const int threads = st.slots <= 256 ? 256 : 512;
  const int grid = std::max(1, std::min(num_sms, (p.rows + threads - 1) / threads));
  const size_t smem = sizeof(int) * (6 * static_cast<size_t>(st.slots) + 4);
  if (smem > 48 * 1024) opt_in_smem(page_tables_kernel, smem);
  launch_dependent(page_tables_kernel, dim3(grid), dim3(threads), smem, s, a);
  return 1;
}

}  // namespace kvq
