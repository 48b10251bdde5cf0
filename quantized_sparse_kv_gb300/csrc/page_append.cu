// kv_append_pages and kv_page_values: new tokens into the pages and windows of one layer,
// and listed tokens read back.
//
// int4 rule of kv_pack ("KV殘差窗口", section 固定預算): scale = fl(amax / 7), code =
// clamp(rint(fl(x / scale)), -7, 7), K per channel over the 32 tokens of a group, V per
// token over 32 features.
#include <algorithm>

#include "int4_round.cuh"
#include "paged.cuh"

namespace kvq {
namespace {

struct AppendPagesArgs {
  PagedDims d;
  PageRows r;
  const int32_t *offsets, *before, *after, *work, *counts;
  int cap_work;
  KernelCtl ctl;
};

__device__ __forceinline__ float int4_scale(float amax) { return __fdiv_rn(amax, 7.0f); }
__device__ __forceinline__ int int4_code(float x, float scale) {
  if (scale == 0.0f) return 0;
  return max(-7, min(7, __float2int_rn(__fdiv_rn(x, scale))));
}

__device__ __forceinline__ float load_elem(const void *p, size_t i, int dt) {
  return dt == KVQ_F32 ? static_cast<const float *>(p)[i]
                       : bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}
__device__ __forceinline__ size_t el_bytes(int dt) { return dt == KVQ_F32 ? 4 : 2; }

// One work entry and head: what the step does with 32-token group g of slot s.
struct GroupWork {
  int s, g, h, before, after, c1, w0, w1, row0;
};

// Value of token pos, feature d as the cache keeps it (rounded to the window's type).
template <bool kV>
__device__ __forceinline__ float source(const AppendPagesArgs &a, const GroupWork &w, int pos,
                                        int d) {
  const int D = a.d.D;
  if (pos < w.before) {
    const size_t e = a.d.tile_at(w.s, w.h, pos >> 5) +
                     (kV ? 32 * D + ringv_at(pos & 31, d, D) : ringk_at(pos & 31, d, D));
    const size_t b = el_bytes(a.d.win_dt);
    if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.d.ring) + e * b, b)) return 0.0f;
    return load_elem(a.d.ring, e, a.d.win_dt);
  }
  const int64_t row = w.row0 + pos - w.before;
  const void *p = kV ? a.r.v : a.r.k;
  const size_t e = static_cast<size_t>(row * (kV ? a.r.vsr : a.r.ksr) +
                                       w.h * (kV ? a.r.vsh : a.r.ksh) + d);
  const size_t b = el_bytes(a.r.dtype);
  if (!in_bounds(a.ctl, static_cast<const uint8_t *>(p) + e * b, b)) return 0.0f;
  const float x = load_elem(p, e, a.r.dtype);
  return a.d.win_dt == KVQ_F32 ? x : __bfloat162float(__float2bfloat16_rn(x));
}

// The new tokens of window group g into its tile.
__device__ __forceinline__ void write_tile(const AppendPagesArgs &a, const GroupWork &w, int g) {
  const int D = a.d.D, p0 = max(w.before, 32 * g), p1 = min(w.after, 32 * g + 32);
  const size_t tile = a.d.tile_at(w.s, w.h, g);
  for (int i = threadIdx.x; i < 2 * D * (p1 - p0); i += blockDim.x) {
    const int pos = p0 + i / (2 * D), e = i % (2 * D), d = e < D ? e : e - D, r = pos & 31;
    const float x = e < D ? source<false>(a, w, pos, d) : source<true>(a, w, pos, d);
    const size_t o = tile + (e < D ? ringk_at(r, d, D) : 32 * D + ringv_at(r, d, D));
    const size_t b = el_bytes(a.d.win_dt);
    if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.d.ring) + o * b, b)) continue;
    if (a.d.win_dt == KVQ_F32)
      static_cast<float *>(a.d.ring)[o] = x;
    else
      static_cast<__nv_bfloat16 *>(a.d.ring)[o] = __float2bfloat16_rn(x);
  }
}

constexpr int kApThreads = 256;

// A CTA per (group of the work list, head). A group that is packed may have tokens in a
// tile of the window that the step's new tokens take over: the CTA that packs it writes
// them too, behind its own reads, and the tile's own entry leaves them to it, so no
// order between CTAs is needed.
__global__ void __launch_bounds__(kApThreads) append_pages_kernel(const AppendPagesArgs a) {
  extern __shared__ float xs[];  // [32][D + 1], then codes
  wait_prior_grid();
  allow_next_grid();
  const int D = a.d.D, ld = D + 1, T = a.d.tiles, nb = D / 32;
  uint8_t *codes = reinterpret_cast<uint8_t *>(xs + 32 * ld);  // [32][D]
  int n = 0;
  if (in_bounds(a.ctl, a.counts, 16)) n = min(a.counts[1], a.cap_work);
  for (int it = blockIdx.x; it < n * a.d.Hkv; it += gridDim.x) {
    GroupWork w;
    w.h = it % a.d.Hkv;
    const int32_t *e = a.work + 2 * (it / a.d.Hkv);
    if (!in_bounds(a.ctl, e, 8)) continue;
    w.s = e[0];
    w.g = e[1];
    if (w.s < 0 || w.s >= a.d.slots) continue;
    w.before = a.before[w.s];
    w.after = a.after[w.s];
    w.row0 = a.offsets[w.s];
    w.c1 = paged_cut(w.after, a.d.window) >> 5;
    w.w0 = max(w.before >> 5, w.c1);
    w.w1 = (w.after + 31) >> 5;
    const int c0 = paged_cut(w.before, a.d.window) >> 5, ob = (w.before + 31) >> 5;
    if (w.g >= w.c1) {
      // the old group in this tile, if it moves into the pages, has its CTA write here
      const int o = ob - 1 - (((ob - 1 - w.g) % T) + T) % T;
      if (!(ob > c0 && o >= c0 && o < w.c1)) write_tile(a, w, w.g);
      continue;
    }
    const int32_t *pe = a.d.table + static_cast<size_t>(w.s) * a.d.max_pages +
                        (w.g >> a.d.gpp_log2());
    const int page = in_bounds(a.ctl, pe, 4) ? *pe : -1;
    uint8_t *rec = nullptr;
    if (page >= 0 && page < a.d.n_pages)
      rec = a.d.record_at(page, w.g & ((1 << a.d.gpp_log2()) - 1), w.h);
    else if (threadIdx.x == 0)
      flag_error(a.ctl, KVQ_DEV_INDEX);
    if (rec && !in_bounds(a.ctl, rec, a.d.record())) rec = nullptr;
    __syncthreads();  // (the staged values of the item before are read)
    for (int i = threadIdx.x; i < 32 * D; i += kApThreads)
      xs[i / D * ld + i % D] = source<false>(a, w, 32 * w.g + i / D, i % D);
    __syncthreads();
    if (rec) {
      for (int c = threadIdx.x; c < D; c += kApThreads) {
        float m = 0.0f;
        for (int t = 0; t < 32; ++t) m = fmaxf(m, fabsf(xs[t * ld + c]));
        const float sc = int4_scale(m);
        reinterpret_cast<float *>(rec + rec_kscale(D))[kscale_at(c, D)] = sc;
        for (int t = 0; t < 32; ++t)
          codes[t * D + c] = static_cast<uint8_t>(int4_code(xs[t * ld + c], sc) + 8);
      }
    }
    __syncthreads();
    if (rec)
      for (int i = threadIdx.x; i < 16 * D; i += kApThreads)
        rec[i] = codes[2 * i] | codes[2 * i + 1] << 4;
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * D; i += kApThreads)
      xs[i / D * ld + i % D] = source<true>(a, w, 32 * w.g + i / D, i % D);
    __syncthreads();
    if (rec) {
      for (int i = threadIdx.x; i < 32 * nb; i += kApThreads) {
        const int t = i / nb, b = i % nb;
        float m = 0.0f;
        for (int k = 0; k < 32; ++k) m = fmaxf(m, fabsf(xs[t * ld + 32 * b + k]));
        const float sc = int4_scale(m);
        reinterpret_cast<float *>(rec + rec_vscale(D))[vscale_at(t, b, D)] = sc;
        for (int k = 0; k < 32; ++k)
          codes[t * D + 32 * b + k] =
              static_cast<uint8_t>(int4_code(xs[t * ld + 32 * b + k], sc) + 8);
      }
    }
    __syncthreads();
    if (rec) {
      for (int i = threadIdx.x; i < 4 * D; i += kApThreads) {
        const int f = i % (D / 16), t = i / (D / 16) % 4, g = i / (D / 4) % 8, m = i / (2 * D);
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x |= static_cast<uint32_t>(
                   codes[(16 * m + 2 * t + (k >> 2) + 8 * (k & 1)) * D + 16 * f + 8 * (k >> 1 & 1) + g])
               << (4 * k);
        reinterpret_cast<uint32_t *>(rec + rec_vcode(D))[vword_at(m, g, t, f, D)] = x;
      }
    }
    // the window group that takes over this group's tile
    if (32 * w.g < w.before) {
      const int g = w.w0 + (((w.g - w.w0) % T) + T) % T;
      __syncthreads();  // every value of the tile has been read
      if (g < w.w1) write_tile(a, w, g);
    }
  }
}

struct PageValuesArgs {
  PagedDims d;
  const int32_t *slot, *pos;
  void *k, *v;
  int n, out_dt;
  KernelCtl ctl;
};

// A thread per (row, head, eight features) of K and V.
__global__ void __launch_bounds__(256) page_values_kernel(const PageValuesArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int D = a.d.D, pieces = a.d.Hkv * D / 8;
  const long total = static_cast<long>(a.n) * pieces;
  const long stride = static_cast<long>(gridDim.x) * blockDim.x;
  for (long i = blockIdx.x * static_cast<long>(blockDim.x) + threadIdx.x; i < total; i += stride) {
    const int row = static_cast<int>(i / pieces), x = static_cast<int>(i - static_cast<long>(row) * pieces);
    const int h = x / (D / 8), p = x - h * (D / 8), d0 = 8 * p;
    if (!in_bounds(a.ctl, a.slot + row, 4) || !in_bounds(a.ctl, a.pos + row, 4)) continue;
    const int s = a.slot[row], pos = a.pos[row];
    if (s == -1) continue;
    int len = -1;
    if (s >= 0 && s < a.d.slots && in_bounds(a.ctl, a.d.lengths + s, 4)) len = a.d.lengths[s];
    if (!a.d.holds(len) || pos < 0 || pos >= len) {
      if (x == 0) flag_error(a.ctl, KVQ_DEV_INDEX);
      continue;
    }
    const int g = pos >> 5, r = pos & 31;
    float k[8], v[8];
    if (pos < paged_cut(len, a.d.window)) {
      const int32_t *pe = a.d.table + static_cast<size_t>(s) * a.d.max_pages + (g >> a.d.gpp_log2());
      const int page = in_bounds(a.ctl, pe, 4) ? *pe : -1;
      const uint8_t *rec = a.d.record_at(page, g & ((1 << a.d.gpp_log2()) - 1), h);
      if (page < 0 || page >= a.d.n_pages) {
        if (x == 0) flag_error(a.ctl, KVQ_DEV_INDEX);
        continue;
      }
      if (!in_bounds(a.ctl, rec, a.d.record())) continue;
      const uint32_t kw = *reinterpret_cast<const uint32_t *>(rec + r * (D / 2) + 4 * p);
      const float *ks = reinterpret_cast<const float *>(rec + rec_kscale(D));
      const uint32_t *vw = reinterpret_cast<const uint32_t *>(rec + rec_vcode(D));
      const float vs = reinterpret_cast<const float *>(rec + rec_vscale(D))[vscale_at(r, d0 >> 5, D)];
      // token r, features d0 + g: nibble 4 (r % 2) + 2 (d0 / 8 % 2) + (r / 8 % 2)
      const int sh = 4 * (4 * (r & 1) + 2 * (p & 1) + (r >> 3 & 1));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] = (static_cast<int>(kw >> (4 * j) & 15) - 8) * ks[kscale_at(d0 + j, D)];
        v[j] = (static_cast<int>(vw[vword_at(r >> 4, j, (r & 7) >> 1, d0 >> 4, D)] >> sh & 15) - 8) * vs;
      }
    } else {
      const size_t tile = a.d.tile_at(s, h, g), b = el_bytes(a.d.win_dt);
      if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.d.ring) + tile * b, 64 * D * b)) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] = load_elem(a.d.ring, tile + ringk_at(r, d0 + j, D), a.d.win_dt);
        v[j] = load_elem(a.d.ring, tile + 32 * D + ringv_at(r, d0 + j, D), a.d.win_dt);
      }
    }
    const size_t o = (static_cast<size_t>(row) * a.d.Hkv + h) * D + d0, ob = el_bytes(a.out_dt);
    for (int z = 0; z < 2; ++z) {
      void *out = z ? a.v : a.k;
      const float *y = z ? v : k;
      if (!in_bounds(a.ctl, static_cast<const uint8_t *>(out) + o * ob, 8 * ob)) continue;
      if (a.out_dt == KVQ_F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
        q[0] = make_float4(y[0], y[1], y[2], y[3]);
        q[1] = make_float4(y[4], y[5], y[6], y[7]);
      } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o) =
            make_uint4(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]), pack_bf2(y[4], y[5]),
                       pack_bf2(y[6], y[7]));
      }
    }
  }
}

}  // namespace

int launch_append_pages(const PagedDims &d, const kvq_page_plan &p, const PageRows &r,
                        const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  AppendPagesArgs a;
  a.d = d;
  a.r = r;
  a.offsets = p.offsets;
  a.before = p.before;
  a.after = p.after;
  a.work = p.work;
  a.counts = p.counts;
  a.cap_work = p.cap_work;
  a.ctl = ctl;
  const size_t smem = 32 * (4 * (static_cast<size_t>(d.D) + 1) + d.D);
  const long items = static_cast<long>(p.cap_work) * d.Hkv;
  const int grid = static_cast<int>(std::min<long>(items, 6L * num_sms));
  launch_dependent(append_pages_kernel, dim3(grid), dim3(kApThreads), smem, s, a);
  return 1;
}

int launch_page_values(const PagedDims &d, const int32_t *slot, const int32_t *pos, int n,
                       void *k, void *v, int out_dt, const KernelCtl &ctl, int num_sms,
                       cudaStream_t s) {
  PageValuesArgs a;
  a.d = d;
  a.slot = slot;
  a.pos = pos;
  a.k = k;
  a.v = v;
  a.n = n;
  a.out_dt = out_dt;
  a.ctl = ctl;
  const long total = static_cast<long>(n) * d.Hkv * d.D / 8;
  const int grid = static_cast<int>(std::min<long>((total + 255) / 256, 8L * num_sms));
  launch_dependent(page_values_kernel, dim3(grid), dim3(256), 0, s, a);
  return 1;
}

}  // namespace kvq
