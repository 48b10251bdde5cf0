// kv_attend_pages in fp32 for the shapes the tensor-core kernel leaves out (other head
// dims, fp32 windows): O = softmax(scale q K^T) V over the first tokens of a request in
// the paged cache.
//
// A CTA takes one query row, up to eight query heads of one KV head and an equal share of
// the row's 32-token groups; each group's keys and values are staged in shared memory as
// floats, a word of eight codes at a time. A warp has an eighth of the channels of all
// scores (lane = token), so that K is read once for the heads; the parts meet in shared
// memory, where warp h takes head h's maximum and sum. A warp then has four of the tokens
// of the output, all heads in registers over all groups, and the warps' sums meet at the end. A
// second kernel merges the shares, a lane a share. The fp32 products and the latency
// of the staging at 16 warps per SM bound it: 64 requests of 24 thousand tokens, 16 heads over 2,
// D = 128, fp32 windows: 1.74 ms (codes one by one and K read by every head 4.3; the tensor
// cores, with bf16 windows, 0.09); 8 of 8 thousand, D = 256: 174 us (573).
#include <math_constants.h>

#include <algorithm>

#include "paged.cuh"

namespace kvq {
namespace {

constexpr int kPrThreads = 256;
constexpr int kPrWarps = kPrThreads / 32;
constexpr int kPrHeads = 8;
constexpr int kPrSplits = 64;  // shares of a row at most: two a lane of the merge
static_assert(kPrHeads <= kPrWarps);

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

// K and V of an int4 group as floats, rows of ld: a word of eight codes at a time. K: eight
// channels of a token; V: tokens x, x + 8 and the ones behind them, features y and y + 8.
__device__ __forceinline__ void stage_group(const PageRowsArgs &a, const uint8_t *rec, float *ks,
                                            float *vs, int ld) {
  const int D = a.d.D, pieces = D / 8, cl = D % 64 == 0 ? 2 : 1, fw = (D / 16) >> cl;
  const float *kscale = reinterpret_cast<const float *>(rec + rec_kscale(D));
  const float *vscale = reinterpret_cast<const float *>(rec + rec_vscale(D));
  const uint32_t *vw = reinterpret_cast<const uint32_t *>(rec + rec_vcode(D));
  for (int i = threadIdx.x; i < 4 * D; i += kPrThreads) {
    const int r = i / pieces, p = i - r * pieces;
    const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + 4 * i);
    const float *sc = kscale + kscale_at(8 * p, D);  // channels 0 4 1 5, and behind 16: 2 6 3 7
    const float4 x = *reinterpret_cast<const float4 *>(sc);
    const float4 y = *reinterpret_cast<const float4 *>(sc + 16);
    const auto code = [w](int j) { return static_cast<float>(static_cast<int>(w >> (4 * j) & 15) - 8); };
    float4 *o = reinterpret_cast<float4 *>(ks + r * ld + 8 * p);
    o[0] = make_float4(code(0) * x.x, code(1) * x.z, code(2) * y.x, code(3) * y.z);
    o[1] = make_float4(code(4) * x.y, code(5) * x.w, code(6) * y.y, code(7) * y.w);
  }
  // (a lane takes the words it has side by side: stores of a warp fall into 32 banks)
  for (int i = threadIdx.x; i < 4 * D >> cl; i += kPrThreads) {
    const int lane = i & 31, mf = i >> 5, m = mf / fw, f0 = (mf - m * fw) << cl;
    const int x = 16 * m + 2 * (lane & 3);
    uint32_t w[4];
    if (cl == 2) {
      const uint4 u = reinterpret_cast<const uint4 *>(vw)[i];
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = reinterpret_cast<const uint2 *>(vw)[i];
      w[0] = u.x, w[1] = u.y, w[2] = w[3] = 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= 1 << cl) break;
      const int f = f0 + k;
      const float2 sa = *reinterpret_cast<const float2 *>(vscale + vscale_at(x, f >> 1, D));
      const float2 sb = *reinterpret_cast<const float2 *>(vscale + vscale_at(x + 8, f >> 1, D));
      const auto code = [&](int j) { return static_cast<float>(static_cast<int>(w[k] >> (4 * j) & 15) - 8); };
      float *o = vs + x * ld + 16 * f + (lane >> 2);
      o[0] = code(0) * sa.x;
      o[8] = code(2) * sa.x;
      o[8 * ld] = code(1) * sb.x;
      o[8 * ld + 8] = code(3) * sb.x;
      o[ld] = code(4) * sa.y;
      o[ld + 8] = code(6) * sa.y;
      o[9 * ld] = code(5) * sb.y;
      o[9 * ld + 8] = code(7) * sb.y;
    }
  }
}

// The same of a window tile: eight elements of K are channels 0 4 1 5 2 6 3 7 of a token, eight
// of V features 8 apart of two tokens.
template <typename Win>
__device__ __forceinline__ void stage_tile(const PageRowsArgs &a, size_t tile, float *ks, float *vs,
                                           int ld) {
  const int D = a.d.D, pieces = D / 8;
  const Win *x = static_cast<const Win *>(a.d.ring) + tile;
  float e[8];
  const auto load8 = [&e](const Win *p) {
    if constexpr (sizeof(Win) == 4) {
      const float4 u = reinterpret_cast<const float4 *>(p)[0], w = reinterpret_cast<const float4 *>(p)[1];
      e[0] = u.x, e[1] = u.y, e[2] = u.z, e[3] = u.w, e[4] = w.x, e[5] = w.y, e[6] = w.z, e[7] = w.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e[2 * k] = __uint_as_float(w[k] << 16);
        e[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  };
  for (int i = threadIdx.x; i < 4 * D; i += kPrThreads) {
    const int r = i / pieces, p = i - r * pieces;
    load8(x + ringk_at(r, 8 * p, D));
    float4 *o = reinterpret_cast<float4 *>(ks + r * ld + 8 * p);
    o[0] = make_float4(e[0], e[2], e[4], e[6]);
    o[1] = make_float4(e[1], e[3], e[5], e[7]);
  }
  for (int i = threadIdx.x; i < 4 * D; i += kPrThreads) {
    const int t = i & 3, g = i >> 2 & 7, rb = i >> 5, r8 = rb / (D / 32), b = rb - r8 * (D / 32);
    load8(x + 32 * D + 8 * i);
    float *o = vs + (8 * r8 + 2 * t) * ld + 32 * b + g;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[8 * k] = e[2 * k];
      o[ld + 8 * k] = e[2 * k + 1];
    }
  }
}

// kCols: float4 columns of the output a lane has (2 for D > 128).
template <int kCols>
__global__ void __launch_bounds__(kPrThreads, 2) page_rows_kernel(const PageRowsArgs a) {
  extern __shared__ __align__(16) float sm[];
  wait_prior_grid();
  allow_next_grid();
  const int D = a.d.D, ld = D + 4, gl = a.d.gpp_log2();
  float *ks = sm, *vs = ks + 32 * ld, *qs = vs + 32 * ld, *ps = qs + kPrHeads * D;
  float *red = ps + kPrHeads * 32, *corr = red + kPrWarps * kPrHeads * 32;
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
  // of the tokens 4 warp .. 4 warp + 3 of every group: features 4 (lane + 32 k) and on
  const int cols = D / 4;
  float acc[kCols][kPrHeads][4];
#pragma unroll
  for (int k = 0; k < kCols; ++k)
#pragma unroll
    for (int h = 0; h < kPrHeads; ++h) acc[k][h][0] = acc[k][h][1] = acc[k][h][2] = acc[k][h][3] = 0.0f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -CUDART_INF_F, l = 0.0f;
  for (int g = g0; g < g1; ++g) {
    const int valid = min(32, n - 32 * g);
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
    // (rows behind the attended ones are staged as they are and not used)
    __syncthreads();
    if (rec)
      stage_group(a, rec, ks, vs, ld);
    else if (a.d.win_dt == KVQ_F32)
      stage_tile<float>(a, tile, ks, vs, ld);
    else
      stage_tile<uint16_t>(a, tile, ks, vs, ld);
    __syncthreads();
    {  // a warp's eighth of the channels of every score; lane = token
      float x[kPrHeads];
#pragma unroll
      for (int h = 0; h < kPrHeads; ++h) x[h] = 0.0f;
      const int c0 = warp * (cols / kPrWarps);
      const float4 *k4 = reinterpret_cast<const float4 *>(ks + lane * ld);
      const float4 *q4 = reinterpret_cast<const float4 *>(qs);
      for (int d = c0; d < c0 + cols / kPrWarps; ++d) {
        const float4 k = k4[d];
#pragma unroll
        for (int h = 0; h < kPrHeads; ++h) {
          if (h >= nh) break;
          const float4 q = q4[h * cols + d];
          x[h] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, x[h]))));
        }
      }
#pragma unroll
      for (int h = 0; h < kPrHeads; ++h)
        if (h < nh) red[(warp * kPrHeads + h) * 32 + lane] = x[h];
    }
    __syncthreads();
    if (warp < nh) {  // a head's scores; lane = token
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < kPrWarps; ++w) x += red[(w * kPrHeads + warp) * 32 + lane];
      if (lane >= valid) x = -CUDART_INF_F;
      const float mx = fmaxf(m, warp_max(x));
      const float ref = mx == -CUDART_INF_F ? 0.0f : mx;
      const float p = lane < valid ? exp2f(x - ref) : 0.0f, f = exp2f(m - ref);
      ps[warp * 32 + lane] = p;
      l = l * f + warp_sum(p);
      m = mx;
      if (lane == 0) corr[warp] = f;
    }
    __syncthreads();
    float4 p[kPrHeads];
#pragma unroll
    for (int h = 0; h < kPrHeads; ++h) {
      if (h >= nh) break;
      p[h] = *reinterpret_cast<const float4 *>(ps + h * 32 + 4 * warp);
      const float f = corr[h];
#pragma unroll
      for (int k = 0; k < kCols; ++k)
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[k][h][z] *= f;
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      if (lane + 32 * k >= cols) break;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 4 * warp + t;
        if (r >= valid) break;  // (what is staged there may be anything)
        const float4 v = *reinterpret_cast<const float4 *>(vs + r * ld + 4 * (lane + 32 * k));
#pragma unroll
        for (int h = 0; h < kPrHeads; ++h) {
          if (h >= nh) break;
          const float y = t == 0 ? p[h].x : t == 1 ? p[h].y : t == 2 ? p[h].z : p[h].w;
          acc[k][h][0] = fmaf(y, v.x, acc[k][h][0]);
          acc[k][h][1] = fmaf(y, v.y, acc[k][h][1]);
          acc[k][h][2] = fmaf(y, v.z, acc[k][h][2]);
          acc[k][h][3] = fmaf(y, v.w, acc[k][h][3]);
        }
      }
    }
  }
  // the warps' sums meet in the space of K and V, [warp][head][D]
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    if (lane + 32 * k >= cols) break;
#pragma unroll
    for (int h = 0; h < kPrHeads; ++h)
      if (h < nh)
        *reinterpret_cast<float4 *>(sm + (warp * kPrHeads + h) * D + 4 * (lane + 32 * k)) =
            make_float4(acc[k][h][0], acc[k][h][1], acc[k][h][2], acc[k][h][3]);
  }
  if (warp < nh && lane == 0) corr[warp] = l == 0.0f ? 0.0f : 1.0f / l;
  __syncthreads();
  float *part = part_of(a, row, hc, blockIdx.z);
  if (a.splits > 1 && !in_bounds(a.ctl, part, sizeof(float) * kPrHeads * (D + 2))) return;
  for (int i = threadIdx.x; i < nh * D; i += kPrThreads) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kPrWarps; ++w) y += sm[w * kPrHeads * D + i];
    const int h = i / D;
    if (a.splits == 1)  // the row's only share
      store_out(a, (static_cast<size_t>(row) * a.Hq + h0) * D + i, y * corr[h]);
    else
      part[h * (D + 2) + i - h * D] = y;
  }
  if (a.splits > 1 && warp < nh && lane == 0) {
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
  __shared__ float weight[kPrHeads][kPrSplits], inv[kPrHeads];
  const float *p = part_of(a, row, hc, 0);
  const size_t step = kPrHeads * (D + 2);
  if (!in_bounds(a.ctl, p, sizeof(float) * a.splits * step)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < nh) {  // a head's weights; lane = share
    const float *ph = p + warp * (D + 2) + D;
    float pm[2], pl[2], mx = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int z = lane + 32 * k;
      pm[k] = z < a.splits ? ph[z * step] : -CUDART_INF_F;
      pl[k] = z < a.splits ? ph[z * step + 1] : 0.0f;
      mx = fmaxf(mx, pm[k]);
    }
    mx = warp_max(mx);
    if (mx == -CUDART_INF_F) mx = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // (a share without keys has m = -inf and weight 0; one of NaN scores keeps its NaN)
      const float c = pl[k] != pl[k] ? pl[k] : exp2f(pm[k] - mx);
      weight[warp][lane + 32 * k] = c;
      l += c * pl[k];
    }
    l = warp_sum(l);
    if (lane == 0) inv[warp] = l == 0.0f ? 0.0f : 1.0f / l;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * D; i += kPrThreads) {
    const int h = i / D, d = i - h * D;
    const float *pd = p + h * (D + 2) + d;
    float y = 0.0f;
#pragma unroll 16
    for (int z = 0; z < a.splits; ++z) y = fmaf(weight[h][z], pd[z * step], y);
    store_out(a, (static_cast<size_t>(row) * a.Hq + h0) * D + i, y * inv[h]);
  }
}

// Shares of a row: enough CTAs for four waves of the SMs, at most 64.
int row_splits(const PagedDims &d, int Hq, int rows, int num_sms) {
  const int chunks = (Hq / d.Hkv + kPrHeads - 1) / kPrHeads;
  const long units = static_cast<long>(rows) * d.Hkv * chunks;
  return static_cast<int>(std::max<long>(1, std::min<long>(kPrSplits, 4L * num_sms / std::max(1L, units))));
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
  const size_t smem = sizeof(float) * (64 * (static_cast<size_t>(d.D) + 4) + kPrHeads * (d.D + 33) +
                                       32 * kPrWarps * kPrHeads);
  auto *const kernel = d.D > 128 ? page_rows_kernel<2> : page_rows_kernel<1>;
  opt_in_smem(kernel, smem);
  const dim3 grid(rows, d.Hkv * a.chunks, a.splits);
  launch_dependent(kernel, grid, dim3(kPrThreads), smem, s, a);
  if (a.splits == 1) return 1;
  launch_dependent(page_rows_combine_kernel, dim3(rows, d.Hkv * a.chunks), dim3(kPrThreads), 0, s,
                   a);
  return 2;
}

}  // namespace kvq
