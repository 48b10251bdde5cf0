// fp32 attention of single rows over chosen keys, for any supported shape: the
// path of kv_attend_tree and kv_attend_blocks for the shapes and types their
// tensor-core kernels do not take (fp32 queries, other head dims, fp32 or MXFP8
// windows).
//
// One CTA of 8 warps per query token, sequence and (up to) four of the query heads
// that share a KV head, which see the same keys: each key and value is read and
// dequantized once for all of them. The keys are walked in chunks of 32: the
// cache's tokens and then the drafted ones (tree), or the listed blocks' groups
// and then the window (blocks); warp w takes chunks w, w + 8, ... Lane j of a warp
// scores key j of the chunk against the whole q rows in shared memory, the warp
// keeps an online softmax per row (running maximum, rescaled sum) and each lane
// owns D / 32 output features. The warps' states meet in shared memory. Keys a
// token does not see are never read into a sum, so their contents do not matter.
// It is bound by its instructions: 8 sequences x 16 drafted tokens x 16 heads over
// 8,192 keys, D = 128, fp32 queries: 691 us (one head a CTA, values loaded key by
// key: 2,916 us); 32 listed blocks of 64 keys, 8 sequences: 35.5 us.
#include <math_constants.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRowWarps = 8;

struct RowsArgs {
  const uint8_t *k_codes;
  const float *k_scales;
  const uint8_t *v_codes;
  const float *v_scales;
  const void *k_window;
  const void *v_window;
  const uint8_t *k_e8m0;
  int kwin, vwin;
  int Hkv, N, R, cut, Gs, Vs, Ws;
  int Hq, group, n_q;
  const void *q;
  int q_dtype;
  void *out;
  int out_dtype;
  float scale;
  // tree
  const void *k_tree, *v_tree;
  int tree_dtype;
  const int32_t *parents;
  // blocks
  const int32_t *selected;
  int top_k, block, n_blocks;
  KernelCtl ctl;
};

__device__ __forceinline__ float nibble(uint32_t byte, int odd) {
  return static_cast<float>(static_cast<int>(odd ? (byte >> 4) & 15u : byte & 15u) - 8);
}
__device__ __forceinline__ float elem(const void *p, int dtype, long i) {
  return dtype == KVQ_F32 ? static_cast<const float *>(p)[i]
                          : bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}
__device__ __forceinline__ size_t elem_size(int dtype) {
  return dtype == KVQ_F32 ? 4 : dtype == KVQ_BF16 ? 2 : 1;
}

// s[r] += q[r][d .. d + 3] . (x0 .. x3)
template <int D, int kRows>
__device__ __forceinline__ void dot4(float (&s)[kRows], const float (*q)[D], int d, float x0,
                                     float x1, float x2, float x3) {
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float4 y = *reinterpret_cast<const float4 *>(&q[r][d]);
    s[r] = fmaf(y.w, x3, fmaf(y.z, x2, fmaf(y.y, x1, fmaf(y.x, x0, s[r]))));
  }
}

// s[r] = q[r] . (row `row` of a dense [rows][D] tensor)
template <int D, int kRows>
__device__ __forceinline__ void dot_row(const KernelCtl &ctl, const void *p, int dtype, long row,
                                        const float (*q)[D], float (&s)[kRows]) {
  if (!in_bounds(ctl, static_cast<const uint8_t *>(p) + row * D * elem_size(dtype),
                 D * elem_size(dtype)))
    return;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    if (dtype == KVQ_F32) {
      const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + row * D + d);
      dot4<D, kRows>(s, q, d, x.x, x.y, x.z, x.w);
    } else {
      const uint2 x =
          *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + row * D + d);
      dot4<D, kRows>(s, q, d, __uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                     __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
    }
  }
}

// s[r] = q[r] . K of cache token t
template <int D, int kRows>
__device__ __forceinline__ void dot_cache(const RowsArgs &a, long u, int t, const float (*q)[D],
                                          float (&s)[kRows]) {
  if (t < a.cut) {
    const long g = u * a.Gs + t / kGroup;
    const uint32_t *c =
        reinterpret_cast<const uint32_t *>(a.k_codes + (g * kGroup + t % kGroup) * (D / 2));
    const float *sc = a.k_scales + g * D;
    if (!in_bounds(a.ctl, c, D / 2) || !in_bounds(a.ctl, sc, D * sizeof(float))) return;
#pragma unroll 4
    for (int w = 0; w < D / 8; ++w) {
      const uint32_t x = c[w];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = *reinterpret_cast<const float4 *>(sc + 8 * w + 4 * h);
        const uint32_t b0 = x >> (16 * h), b1 = x >> (16 * h + 8);
        dot4<D, kRows>(s, q, 8 * w + 4 * h, nibble(b0, 0) * f.x, nibble(b0, 1) * f.y,
                       nibble(b1, 0) * f.z, nibble(b1, 1) * f.w);
      }
    }
    return;
  }
  const long row = u * a.Ws + (t - a.cut);
  if (a.kwin != KVQ_MXFP8) return dot_row<D, kRows>(a.ctl, a.k_window, a.kwin, row, q, s);
  const uint8_t *c = static_cast<const uint8_t *>(a.k_window) + row * D;
  const uint8_t *e8 = a.k_e8m0 + row * (D / 32);
  if (!in_bounds(a.ctl, c, D) || !in_bounds(a.ctl, e8, D / 32)) return;
  for (int d = 0; d < D; d += 4) {
    const uint8_t e = e8[d / 32];
    dot4<D, kRows>(s, q, d, mxfp8_value(c[d], e), mxfp8_value(c[d + 1], e),
                   mxfp8_value(c[d + 2], e), mxfp8_value(c[d + 3], e));
  }
}

// Element d of V of cache token t
template <int D>
__device__ __forceinline__ float v_cache(const RowsArgs &a, long u, int t, int d) {
  if (t < a.cut) {
    const long row = u * a.Vs + t;
    const uint8_t *c = a.v_codes + row * (D / 2) + d / 2;
    const float *sc = a.v_scales + row * (D / 32) + d / 32;
    if (!in_bounds(a.ctl, c, 1) || !in_bounds(a.ctl, sc, sizeof(float))) return 0.0f;
    return nibble(*c, d & 1) * *sc;
  }
  const long i = (u * a.Ws + (t - a.cut)) * D + d;
  if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.v_window) + i * elem_size(a.vwin),
                 elem_size(a.vwin)))
    return 0.0f;
  return elem(a.v_window, a.vwin, i);
}

template <int DPL, bool kTree, int kRows>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const RowsArgs a) {
  wait_prior_grid();
  allow_next_grid();
  constexpr int D = 32 * DPL;
  __shared__ __align__(16) float qs[kRows][D];
  __shared__ float wo[kRowWarps][kRows][D], wm[kRowWarps][kRows], wl[kRowWarps][kRows];
  __shared__ int par[KVQ_TREE_MAX];
  __shared__ uint32_t seen[KVQ_TREE_MAX / 32];
  __shared__ int row_ok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // query token i of sequence b; heads kvh * group + h0 + 0 .. kRows - 1 (below h0 + heads)
  const int i = blockIdx.x, b = blockIdx.z, per = (a.group + kRows - 1) / kRows;
  const int kvh = blockIdx.y / per, h0 = (blockIdx.y - kvh * per) * kRows;
  const int heads = min(kRows, a.group - h0);
  const long u = static_cast<long>(b) * a.Hkv + kvh;
  const size_t qe = elem_size(a.q_dtype), oe = elem_size(a.out_dtype);
  auto row_of = [&](int r) {
    return (static_cast<long>(b) * a.Hq + kvh * a.group + h0 + r) * a.n_q + i;
  };
  auto q_ok = [&](int r) {
    return r < heads &&
           in_bounds(a.ctl, static_cast<const uint8_t *>(a.q) + row_of(r) * D * qe, D * qe);
  };
  for (int e = tid; e < kRows * D; e += kRowWarps * 32) {
    const int r = e / D, d = e % D;
    qs[r][d] = q_ok(r) ? elem(a.q, a.q_dtype, row_of(r) * D + d) : 0.0f;
  }
  if (kTree) {
    const int32_t *p = a.parents + static_cast<long>(b) * a.n_q;
    const bool ok = in_bounds(a.ctl, p, sizeof(int32_t) * a.n_q);
    for (int j = tid; j < a.n_q; j += kRowWarps * 32) par[j] = ok ? p[j] : -2;
    if (tid < KVQ_TREE_MAX / 32) seen[tid] = 0u;
  }
  __syncthreads();
  if (kTree && tid == 0) {
    // up the parents, each below its child, to the cache (-1); a row that
    // meets anything else holds no token
    int j = i;
    bool bad = false;
    for (;;) {
      const int p = par[j];
      if (p < -1 || p >= j) {
        bad = p != -2 || j != i;  // -2 on the row itself: an unused row
        row_ok = 0;
        break;
      }
      seen[j >> 5] |= 1u << (j & 31);
      if (p == -1) {
        row_ok = 1;
        break;
      }
      j = p;
    }
    if (bad) flag_error(a.ctl, KVQ_DEV_INDEX);
  }
  if (a.kwin == KVQ_MXFP8) {  // Q takes the same MXFP8 rounding as the K window
    for (int j = warp; j < kRows * DPL; j += kRowWarps) {
      float &x = qs[j / DPL][32 * (j % DPL) + lane];
      x = mxfp8_round_warp(x);
    }
  }
  __syncthreads();
  if (kTree && row_ok == 0) return;  // the output of a row without a token stays

  float m[kRows], l[kRows], o[kRows][DPL];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.0f;
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[r][k] = 0.0f;
  }

  const int32_t *list = nullptr;
  int per_block = 1, list_chunks = 0;
  if (!kTree) {
    list = a.selected + (u * a.n_q + i) * a.top_k;
    per_block = a.block / 32;
    // (increasing blocks: a list's entries past the n_blocks-th hold none)
    const int ents = min(a.top_k, a.n_blocks);
    list_chunks = in_bounds(a.ctl, list, sizeof(int32_t) * a.top_k) ? ents * per_block : 0;
  }
  const int cache_chunks = kTree ? (a.N + 31) / 32 : list_chunks;
  const int tail_keys = kTree ? i + 1 : a.R;  // a drafted token sees none after itself
  const int chunks = cache_chunks + (tail_keys + 31) / 32;
  for (int c = warp; c < chunks; c += kRowWarps) {
    int t = -1, tj = -1;  // this lane's cache token, or drafted token
    if (c < cache_chunks) {
      if (kTree) {
        t = 32 * c + lane < a.N ? 32 * c + lane : -1;
      } else {
        const int e = c / per_block, blk = list[e];
        const int prev = e > 0 ? list[e - 1] : -1;
        int bit = 0;
        if (blk != -1 && (blk < 0 || blk >= a.n_blocks)) bit = KVQ_DEV_INDEX;
        else if (blk != -1 && e > 0 && blk <= prev) bit = KVQ_DEV_DUP;
        else if (blk != -1 && e > 0 && prev == -1) bit = KVQ_DEV_INDEX;
        if (bit != 0 && lane == 0 && c % per_block == 0) flag_error(a.ctl, bit);
        if (blk == -1 || bit != 0) continue;
        const int t0 = blk * a.block + 32 * (c % per_block);
        t = t0 + lane < a.cut ? t0 + lane : -1;
      }
    } else {
      const int k = 32 * (c - cache_chunks) + lane;
      if (kTree) {
        if (k < tail_keys && (seen[k >> 5] >> (k & 31) & 1u)) tj = k;
      } else {
        t = k < a.R ? a.cut + k : -1;
      }
    }
    const bool live = t >= 0 || tj >= 0;
    const uint32_t lives = __ballot_sync(0xffffffffu, live);
    if (lives == 0u) continue;
    float p[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) p[r] = 0.0f;
    if (t >= 0) dot_cache<D, kRows>(a, u, t, qs, p);
    if (tj >= 0) dot_row<D, kRows>(a.ctl, a.k_tree, a.tree_dtype, u * a.n_q + tj, qs, p);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float s = live ? p[r] * a.scale : -CUDART_INF_F;
      const float mx = warp_max(s);
      // (all scores -inf: probabilities against 0 are exp(-inf) = 0)
      const float m_new = fmaxf(m[r], mx), ref = m_new == -CUDART_INF_F ? 0.0f : m_new;
      const float corr = m[r] == -CUDART_INF_F ? 0.0f : expf(m[r] - ref);
      p[r] = live ? expf(s - ref) : 0.0f;
      l[r] = l[r] * corr + warp_sum(p[r]);
#pragma unroll
      for (int k = 0; k < DPL; ++k) o[r][k] *= corr;
      m[r] = m_new;
    }
    // 32 keys of the int4 part in a row: their values' loads overlap
    const int t0 = __shfl_sync(0xffffffffu, t, 0);
    const long v0 = u * a.Vs + t0;
    if (__all_sync(0xffffffffu, t >= 0 && t < a.cut) &&
        in_bounds(a.ctl, a.v_codes + v0 * (D / 2), 16 * D) &&
        in_bounds(a.ctl, a.v_scales + v0 * DPL, 128 * DPL)) {
      const uint8_t *c = a.v_codes + v0 * (D / 2) + lane / 2;
      const float *sc = a.v_scales + v0 * DPL;
#pragma unroll 8
      for (int j = 0; j < 32; ++j) {
        float pj[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) pj[r] = __shfl_sync(0xffffffffu, p[r], j);
#pragma unroll
        for (int k = 0; k < DPL; ++k) {
          const float v = nibble(c[j * (D / 2) + 16 * k], lane & 1) * sc[j * DPL + k];
#pragma unroll
          for (int r = 0; r < kRows; ++r) o[r][k] = fmaf(pj[r], v, o[r][k]);
        }
      }
      continue;
    }
    for (int j = 0; j < 32; ++j) {
      if (!(lives >> j & 1u)) continue;
      float pj[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) pj[r] = __shfl_sync(0xffffffffu, p[r], j);
      const int tt = __shfl_sync(0xffffffffu, t, j), tr = __shfl_sync(0xffffffffu, tj, j);
#pragma unroll
      for (int k = 0; k < DPL; ++k) {
        const int d = lane + 32 * k;
        float v = 0.0f;
        if (tr >= 0) {
          const long e = (u * a.n_q + tr) * D + d;
          if (in_bounds(a.ctl, static_cast<const uint8_t *>(a.v_tree) + e * elem_size(a.tree_dtype),
                        elem_size(a.tree_dtype)))
            v = elem(a.v_tree, a.tree_dtype, e);
        } else {
          v = v_cache<D>(a, u, tt, d);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) o[r][k] = fmaf(pj[r], v, o[r][k]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int k = 0; k < DPL; ++k) wo[warp][r][lane + 32 * k] = o[r][k];
    if (lane == 0) {
      wm[warp][r] = m[r];
      wl[warp][r] = l[r];
    }
  }
  __syncthreads();
  for (int e = tid; e < kRows * D; e += kRowWarps * 32) {
    const int r = e / D, d = e % D;
    const long at = row_of(r) * D;
    if (!q_ok(r) || !in_bounds(a.ctl, static_cast<uint8_t *>(a.out) + at * oe, D * oe)) continue;
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) mx = fmaxf(mx, wm[w][r]);
    float ls = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      if (wl[w][r] == 0.0f) continue;  // no key (a NaN sum stays in)
      const float f = wm[w][r] == -CUDART_INF_F ? 1.0f : expf(wm[w][r] - mx);
      ls += f * wl[w][r];
      acc += f * wo[w][r][d];
    }
    const float x = ls == 0.0f ? 0.0f : acc / ls;  // no key at all: zero
    if (a.out_dtype == KVQ_F32)
      static_cast<float *>(a.out)[at + d] = x;
    else
      static_cast<__nv_bfloat16 *>(a.out)[at + d] = __float2bfloat16_rn(x);
  }
}

// Query heads of a KV head that share a CTA (one head alone does not pay for the
// other rows' arithmetic).
constexpr int kShared = 4;

template <bool kTree, int kRows>
int launch_rows_of(const RowsArgs &a, int D, int batch, cudaStream_t s) {
  const dim3 grid(a.n_q, a.Hkv * ((a.group + kRows - 1) / kRows), batch), block(kRowWarps * 32);
  switch (D / 32) {
    case 1: launch_dependent(rows_kernel<1, kTree, kRows>, grid, block, 0, s, a); break;
    case 2: launch_dependent(rows_kernel<2, kTree, kRows>, grid, block, 0, s, a); break;
    case 3: launch_dependent(rows_kernel<3, kTree, kRows>, grid, block, 0, s, a); break;
    case 4: launch_dependent(rows_kernel<4, kTree, kRows>, grid, block, 0, s, a); break;
    case 5: launch_dependent(rows_kernel<5, kTree, kRows>, grid, block, 0, s, a); break;
    case 6: launch_dependent(rows_kernel<6, kTree, kRows>, grid, block, 0, s, a); break;
    case 7: launch_dependent(rows_kernel<7, kTree, kRows>, grid, block, 0, s, a); break;
    default: launch_dependent(rows_kernel<8, kTree, kRows>, grid, block, 0, s, a); break;
  }
  return 1;
}

template <bool kTree>
int launch_rows(const RowsArgs &a, int D, int batch, cudaStream_t s) {
  return a.group == 1 ? launch_rows_of<kTree, 1>(a, D, batch, s)
                      : launch_rows_of<kTree, kShared>(a, D, batch, s);
}

RowsArgs rows_args(const kvq_cache &c, const void *q, int q_dtype, int Hq, int n_q, float scale,
                   void *out, int out_dtype, const KernelCtl &ctl) {
  const CacheDims d = dims_of(c);
  RowsArgs a = {};
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.v_codes = c.v_codes;
  a.v_scales = c.v_scales;
  a.k_window = c.k_window;
  a.v_window = c.v_window;
  a.k_e8m0 = c.k_window_e8m0;
  a.kwin = c.kwin_dtype;
  a.vwin = c.vwin_dtype;
  a.Hkv = d.Hkv;
  a.N = d.N;
  a.R = d.R;
  a.cut = d.cut;
  a.Gs = d.Gs;
  a.Vs = d.Vs;
  a.Ws = d.Ws;
  a.Hq = Hq;
  a.group = Hq / d.Hkv;
  a.n_q = n_q;
  a.q = q;
  a.q_dtype = q_dtype;
  a.out = out;
  a.out_dtype = out_dtype;
  a.scale = scale;
  a.ctl = ctl;
  return a;
}

}  // namespace

int launch_tree_rows(const kvq_cache &c, const void *q, int q_dtype, int Hq, int T,
                     const void *k_tree, const void *v_tree, int tree_dtype,
                     const int32_t *parents, float scale, void *out, int out_dtype,
                     const KernelCtl &ctl, cudaStream_t s) {
  RowsArgs a = rows_args(c, q, q_dtype, Hq, T, scale, out, out_dtype, ctl);
  a.k_tree = k_tree;
  a.v_tree = v_tree;
  a.tree_dtype = tree_dtype;
  a.parents = parents;
  return launch_rows<true>(a, c.head_dim, c.batch, s);
}

int launch_block_rows(const kvq_cache &c, const void *q, int q_dtype, int Hq, int n_q,
                      const int32_t *selected, int top_k, int block, int n_blocks, float scale,
                      void *out, int out_dtype, const KernelCtl &ctl, cudaStream_t s) {
  RowsArgs a = rows_args(c, q, q_dtype, Hq, n_q, scale, out, out_dtype, ctl);
  a.selected = selected;
  a.top_k = top_k;
  a.block = block;
  a.n_blocks = n_blocks;
  return launch_rows<false>(a, c.head_dim, c.batch, s);
}

}  // namespace kvq
