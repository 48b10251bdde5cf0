// kv_attend_pages in fp32 for the shapes the tensor-core kernel leaves out (other head
// dims, fp32 windows): O = softmax(scale q K^T) V over the first tokens of a request in
// the paged cache.
//
// A CTA takes one query row, up to eight query heads of one KV head and an equal share of
// the row's 32-token groups; each group's keys and values are staged in shared memory as
// floats. Warp h scores head h (lane = token) and keeps its running maximum and sum; then
// every thread adds the group's values to its elements of the output. A second kernel
// merges the shares' partial results. It is bound by its arithmetic, an fp32 product at a
// time: 64 requests of 16 to 32 thousand tokens take 5.4 ms (91 us on the tensor cores).
#include <math_constants.h>

#include <algorithm>

#include "paged.cuh"

namespace kvq {
namespace {

constexpr int kPrThreads = 256;
constexpr int kPrHeads = 8;

struct PageRowsArgs {
  PagedDims d;
  const void *q;
  void *out;
  const int32_t *slot, *pos;
  float *part;  // [row][kv head][chunk][split][heads of the chunk (8)][D + 2]
  float scale_log2;
  int q_dt, out_dt, Hq, G, chunks, splits;
  KernelCtl ctl;
};

// Tokens the row attends, and its request; -1: the row is left as it was.
__device__ __forceinline__ int row_tokens(const PageRowsArgs &a, int row, int &s, bool flag) {
  s = row;
  if (a.slot) s = in_bounds(a.ctl, a.slot + row, 4) ? a.slot[row] : -1;
  if (s == -1) return -1;
  int len = -1;
  if (s >= 0 && s < a.d.slots && in_bounds(a.ctl, a.d.lengths + s, 4)) len = a.d.lengths[s];
  int n = len;
  bool ok = a.d.holds(len);
  if (a.pos && ok) {
    const int p = in_bounds(a.ctl, a.pos + row, 4) ? a.pos[row] : -1;
    ok = p >= 0 && p < len;
    n = p + 1;
  }
  if (!ok && flag) flag_error(a.ctl, KVQ_DEV_INDEX);
  return ok ? n : -1;
}

__device__ __forceinline__ float *part_of(const PageRowsArgs &a, int row, int hc, int split) {
  return a.part + ((static_cast<size_t>(row) * a.d.Hkv * a.chunks + hc) * a.splits + split) *
                      (kPrHeads * (a.d.D + 2));
}

__device__ __forceinline__ void store_out(const PageRowsArgs &a, size_t o, float y) {
  const size_t b = a.out_dt == KVQ_F32 ? 4 : 2;
  if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.out) + o * b, b)) return;
  if (a.out_dt == KVQ_F32)
    static_cast<float *>(a.out)[o] = y;
  else
    static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(y);
}

__global__ void __launch_bounds__(kPrThreads) page_rows_kernel(const PageRowsArgs a) {
  extern __shared__ float sm[];
  wait_prior_grid();
  allow_next_grid();
  const int D = a.d.D, ld = D + 1, gl = a.d.gpp_log2();
  float *ks = sm, *vs = ks + 32 * ld, *qs = vs + 32 * D, *ps = qs + kPrHeads * D;
  float *corr = ps + kPrHeads * 32;
  const int row = blockIdx.x, hc = blockIdx.y, kvh = hc / a.chunks, chunk = hc % a.chunks;
  const int h0 = kvh * a.G + kPrHeads * chunk, nh = min(kPrHeads, a.G - kPrHeads * chunk);
  int s;
  const int n = row_tokens(a, row, s, threadIdx.x == 0 && hc == 0 && blockIdx.z == 0);
  if (n < 0) return;
  const int groups = (n + 31) >> 5, cut = paged_cut(a.d.lengths[s], a.d.window) >> 5;
  const int g0 = static_cast<int>(static_cast<long>(groups) * blockIdx.z / a.splits);
  const int g1 = static_cast<int>(static_cast<long>(groups) * (blockIdx.z + 1) / a.splits);
  for (int i = threadIdx.x; i < nh * D; i += kPrThreads) {
    const size_t e = (static_cast<size_t>(row) * a.Hq + h0) * D + i, b = a.q_dt == KVQ_F32 ? 4 : 2;
    float x = 0.0f;
    if (in_bounds(a.ctl, static_cast<const uint8_t *>(a.q) + e * b, b))
      x = a.q_dt == KVQ_F32 ? static_cast<const float *>(a.q)[e]
                            : bf16_to_f32(static_cast<const uint16_t *>(a.q)[e]);
    qs[i] = x * a.scale_log2;
  }
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -CUDART_INF_F, l = 0.0f;
  for (int g = g0; g < g1; ++g) {
    int valid = min(32, n - 32 * g);
    const uint8_t *rec = nullptr;
    size_t tile = 0;
    if (g < cut) {
      const int32_t *pe = a.d.table + static_cast<size_t>(s) * a.d.max_pages + (g >> gl);
      const int page = in_bounds(a.ctl, pe, 4) ? *pe : -1;
      if (page < 0 || page >= a.d.n_pages) {
        if (threadIdx.x == 0) flag_error(a.ctl, KVQ_DEV_INDEX);
        continue;
      }
      rec = a.d.record_at(page, g & ((1 << gl) - 1), kvh);
      if (!in_bounds(a.ctl, rec, a.d.record())) continue;
    } else {
      tile = a.d.tile_at(s, kvh, g);
      const size_t b = a.d.win_dt == KVQ_F32 ? 4 : 2;
      if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.d.ring) + tile * b, 64 * D * b)) continue;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * D; i += kPrThreads) {
      const int r = i / D, d = i - r * D;
      float k = 0.0f, v = 0.0f;
      if (r < valid) {
        if (rec) {
          const int kc = rec[r * (D / 2) + d / 2] >> (4 * (d & 1)) & 15;
          k = (kc - 8) * reinterpret_cast<const float *>(rec + rec_kscale(D))[kscale_at(d, D)];
          const uint32_t w = reinterpret_cast<const uint32_t *>(
              rec + rec_vcode(D))[vword_at(r >> 4, d & 7, (r & 7) >> 1, d >> 4, D)];
          const int vc = w >> (4 * (4 * (r & 1) + 2 * (d >> 3 & 1) + (r >> 3 & 1))) & 15;
          v = (vc - 8) * reinterpret_cast<const float *>(rec + rec_vscale(D))[vscale_at(r, d >> 5, D)];
        } else {
          const size_t ek = tile + ringk_at(r, d, D), ev = tile + 32 * D + ringv_at(r, d, D);
          if (a.d.win_dt == KVQ_F32) {
            k = static_cast<const float *>(a.d.ring)[ek];
            v = static_cast<const float *>(a.d.ring)[ev];
          } else {
            k = bf16_to_f32(static_cast<const uint16_t *>(a.d.ring)[ek]);
            v = bf16_to_f32(static_cast<const uint16_t *>(a.d.ring)[ev]);
          }
        }
      }
      ks[r * ld + d] = k;
      vs[r * D + d] = v;
    }
    __syncthreads();
    if (warp < nh) {
      float x = 0.0f;
      for (int d = 0; d < D; ++d) x = fmaf(qs[warp * D + d], ks[lane * ld + d], x);
      if (lane >= valid) x = -CUDART_INF_F;
      const float mx = fmaxf(m, warp_max(x));
      const float ref = mx == -CUDART_INF_F ? 0.0f : mx;
      const float p = lane < valid ? exp2f(x - ref) : 0.0f, c = exp2f(m - ref);
      ps[warp * 32 + lane] = p;
      l = l * c + warp_sum(p);
      m = mx;
      if (lane == 0) corr[warp] = c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = threadIdx.x + k * kPrThreads;
      if (i < nh * D) {
        const int h = i / D, d = i - h * D;
        float y = acc[k] * corr[h];
        for (int r = 0; r < valid; ++r) y = fmaf(ps[h * 32 + r], vs[r * D + d], y);
        acc[k] = y;
      }
    }
  }
  if (a.splits == 1) {  // the row's only share
    __syncthreads();
    if (warp < nh && lane == 0) corr[warp] = l == 0.0f ? 0.0f : 1.0f / l;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = threadIdx.x + k * kPrThreads;
      if (i < nh * D) store_out(a, (static_cast<size_t>(row) * a.Hq + h0) * D + i, acc[k] * corr[i / D]);
    }
    return;
  }
  float *part = part_of(a, row, hc, blockIdx.z);
  if (!in_bounds(a.ctl, part, sizeof(float) * kPrHeads * (D + 2))) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = threadIdx.x + k * kPrThreads;
    if (i < nh * D) part[i / D * (D + 2) + i % D] = acc[k];
  }
  if (warp < nh && lane == 0) {
    part[warp * (D + 2) + D] = m;
    part[warp * (D + 2) + D + 1] = l;
  }
}

__global__ void __launch_bounds__(kPrThreads) page_rows_combine_kernel(const PageRowsArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int D = a.d.D, row = blockIdx.x, hc = blockIdx.y, kvh = hc / a.chunks;
  const int chunk = hc % a.chunks;
  const int h0 = kvh * a.G + kPrHeads * chunk, nh = min(kPrHeads, a.G - kPrHeads * chunk);
  int s;
  const int n = row_tokens(a, row, s, false);
  if (n < 0) return;
  for (int i = threadIdx.x; i < nh * D; i += kPrThreads) {
    const int h = i / D, d = i - h * D;
    const float *p = part_of(a, row, hc, 0) + h * (D + 2);
    const size_t step = kPrHeads * (D + 2);
    if (!in_bounds(a.ctl, p, sizeof(float) * ((a.splits - 1) * step + D + 2))) return;
    float m = -CUDART_INF_F;
    for (int z = 0; z < a.splits; ++z) m = fmaxf(m, p[z * step + D]);
    if (m == -CUDART_INF_F) m = 0.0f;
    float y = 0.0f, l = 0.0f;
    for (int z = 0; z < a.splits; ++z) {
      // (a share without keys has m = -inf and weight 0; one of NaN scores keeps its NaN)
      const float c = exp2f(p[z * step + D] - m), lz = p[z * step + D + 1];
      y += lz != lz ? lz : c * p[z * step + d];
      l += lz != lz ? lz : c * lz;
    }
    y = l == 0.0f ? 0.0f : y / l;
    store_out(a, (static_cast<size_t>(row) * a.Hq + h0) * D + i, y);
  }
}

// Shares of a row: enough CTAs for four waves of the SMs, at most 64.
int row_splits(const PagedDims &d, int Hq, int rows, int num_sms) {
  const int chunks = (Hq / d.Hkv + kPrHeads - 1) / kPrHeads;
  const long units = static_cast<long>(rows) * d.Hkv * chunks;
  return static_cast<int>(std::max<long>(1, std::min<long>(64, 4L * num_sms / std::max(1L, units))));
}

}  // namespace

size_t page_rows_workspace(const PagedDims &d, int Hq, int rows, int num_sms) {
  const int chunks = (Hq / d.Hkv + kPrHeads - 1) / kPrHeads;
  const int splits = row_splits(d, Hq, rows, num_sms);
  if (splits == 1) return 0;
  return sizeof(float) * rows * d.Hkv * chunks * splits * kPrHeads * (static_cast<size_t>(d.D) + 2);
}

int launch_page_rows(const PagedDims &d, const void *q, int q_dt, int Hq, int rows,
                     const int32_t *slot, const int32_t *pos, float scale, void *out, int out_dt,
                     void *ws, const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  PageRowsArgs a;
  a.d = d;
  a.q = q;
  a.out = out;
  a.slot = slot;
  a.pos = pos;
  a.part = static_cast<float *>(ws);
  a.scale_log2 = scale * 1.44269504088896f;
  a.q_dt = q_dt;
  a.out_dt = out_dt;
  a.Hq = Hq;
  a.G = Hq / d.Hkv;
  a.chunks = (a.G + kPrHeads - 1) / kPrHeads;
  a.splits = row_splits(d, Hq, rows, num_sms);
  a.ctl = ctl;
  const size_t smem = sizeof(float) * (32 * (2 * static_cast<size_t>(d.D) + 1) +
                                       kPrHeads * (d.D + 33));
  opt_in_smem(page_rows_kernel, smem);
  const dim3 grid(rows, d.Hkv * a.chunks, a.splits);
  launch_dependent(page_rows_kernel, grid, dim3(kPrThreads), smem, s, a);
  if (a.splits == 1) return 1;
  launch_dependent(page_rows_combine_kernel, dim3(rows, d.Hkv * a.chunks), dim3(kPrThreads), 0, s,
                   a);
  return 2;
}

}  // namespace kvq
