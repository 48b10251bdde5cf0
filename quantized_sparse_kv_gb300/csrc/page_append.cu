// kv_append_pages and kv_page_values: new tokens into the pages and windows of one layer,
// and listed tokens read back.
//
// int4 rule of kv_pack ("KV殘差窗口", section 固定預算): scale = fl(amax / 7), code =
// clamp(rint(fl(x / scale)), -7, 7), K per channel over the 32 tokens of a group, V per
// token over 32 features. Values that are bf16 take the reciprocal and one correction step,
// others the reciprocal where the code is clear, else the division (int4_round.cuh: the
// same codes).
//
// Append. A CTA of about D / 2 threads has K or V of one 32-token group of one head. For K
// a thread has a pair of channels of all 32 tokens in registers, so the maxima need no
// exchange and a warp reads whole rows. For V a thread has four features of 16 tokens;
// eight lanes share a token's 32 features, their maxima meet in three lane exchanges for two
// tokens at a time and their scales come back through shared memory. V codes are made from
// (token, token + 8) pairs of one feature, which is the byte a record's words hold; lanes of
// features y and y + 8 exchange half of their bytes and each keeps half of the words. Each
// half of the record (20 D bytes) is put together in shared memory and leaves as one bulk
// copy. All of a thread's loads are issued before the first is used, and with bf16 windows 16
// CTAs share an SM at 64 registers, for which the compiler spills 44 bytes a thread (12 at D =
// 64, 36 at other head dims; 28 to 124 with fp32 rows); with fp32 windows eight at 128.
//
// 112,000 rows of two heads, D = 128 (151 MB in and out): 33.3 us, 4.5 TB/s; the loads of
// 32 warps an SM and 1.4 thousand instructions a half group, half of the issue slots, overlap
// in part. Rows staged in shared memory a group ahead (49 us, 42 without as it was then), 16
// values a thread (38) and 80 registers (56) were slower. One token of each of 64 requests:
// 4.5 us, of which the launch is 2 and a group that completes the rest.
#include <algorithm>

#include "int4_round.cuh"
#include "paged.cuh"

namespace kvq {
namespace {

struct AppendPagesArgs {
  PagedDims d;
  PageRows r;
  const int32_t *work, *counts;
  int cap_work;
  KernelCtl ctl;
};

__device__ __forceinline__ float int4_scale(float amax) { return __fdiv_rn(amax, 7.0f); }
__device__ __forceinline__ int int4_code(float x, float scale) {
  if (scale == 0.0f) return 0;
  return max(-7, min(7, __float2int_rn(__fdiv_rn(x, scale))));
}
// Two codes + 8 as a byte, by the division (out of line: the usual bf16 values do without).
__device__ __noinline__ uint32_t code_byte_div(float lo, float hi, float s_lo, float s_hi) {
  return static_cast<uint32_t>(int4_code(lo, s_lo) + 8 + 16 * (int4_code(hi, s_hi) + 8));
}

// The same without a division where the codes are clear (r: reciprocals of the scales, NaN for
// one that has none to be used).
__device__ __forceinline__ uint32_t code_byte_f32(float lo, float hi, float s_lo, float s_hi,
                                                  float r_lo, float r_hi) {
  uint32_t a, b;
  const bool ok = code8_clear(lo, r_lo, a) & code8_clear(hi, r_hi, b);
  return ok ? b * 16u + a : code_byte_div(lo, hi, s_lo, s_hi);
}
__device__ __forceinline__ float recip_or_nan(float amax, float s) {
  return recip_ok(amax) ? recip_of(s) : __int_as_float(0x7fc00000);
}

__device__ __forceinline__ size_t el_bytes(int dt) { return dt == KVQ_F32 ? 4 : 2; }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The larger magnitudes of two bf16 pairs (with signs that mean nothing).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The lowest bytes of four words.
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A pair of values as the cache keeps them: bf16 pairs in one register.
struct PairB {
  uint32_t w;
  __device__ __forceinline__ void set(float x, float y) { w = pack_bf2(x, y); }
  __device__ __forceinline__ float lo() const { return bf_lo(w); }
  __device__ __forceinline__ float hi() const { return bf_hi(w); }
};
struct PairF {
  float2 f;
  __device__ __forceinline__ void set(float x, float y) { f = make_float2(x, y); }
  __device__ __forceinline__ float lo() const { return f.x; }
  __device__ __forceinline__ float hi() const { return f.y; }
};

// Types of the step's rows and of the windows.
template <typename In, typename Win>
struct Types {
  static constexpr bool kBf16 = sizeof(Win) == 2;  // the values are bf16
  using Pair = typename std::conditional<kBf16, PairB, PairF>::type;

  // two elements of a row of the step
  static __device__ __forceinline__ Pair row2(const AppendPagesArgs &a, const In *p) {
    Pair x;
    x.set(0.0f, 0.0f);
    if (!in_bounds(a.ctl, p, 2 * sizeof(In))) return x;
    if constexpr (sizeof(In) == 4) {
      const float2 f = *reinterpret_cast<const float2 *>(p);
      x.set(f.x, f.y);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
      if constexpr (kBf16)
        x.w = w;
      else
        x.set(bf_lo(w), bf_hi(w));
    }
    return x;
  }
  // four elements of a row
  static __device__ __forceinline__ void row4(const AppendPagesArgs &a, const In *p, Pair (&x)[2]) {
    if constexpr (sizeof(In) == 2 && kBf16) {
      const uint2 w = in_bounds(a.ctl, p, 8) ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
      x[0].w = w.x;
      x[1].w = w.y;
    } else {
      x[0] = row2(a, p);
      x[1] = row2(a, p + 2);
    }
  }
  // two elements of the windows
  static __device__ __forceinline__ Pair win2(const AppendPagesArgs &a, const Win *p, const Win *q) {
    Pair x;
    x.set(0.0f, 0.0f);
    if (in_bounds(a.ctl, p, sizeof(Win)) && in_bounds(a.ctl, q, sizeof(Win)))
      x.set(load_f32(p), load_f32(q));
    return x;
  }
  // K of channels c and c + 1 (c even) of window row r. bf16: one load of channels k, k + 4,
  // k + 1, k + 5, which lie together.
  static __device__ __forceinline__ Pair win_k(const AppendPagesArgs &a, const Win *tile, int r, int c,
                                               int D) {
    if constexpr (kBf16) {
      Pair x;
      const Win *p = tile + ringk_at(r, c & ~4, D);
      const uint2 y = in_bounds(a.ctl, p, 8) ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
      x.w = __byte_perm(y.x, y.y, c & 4 ? 0x7632 : 0x5410);
      return x;
    } else {
      return win2(a, tile + ringk_at(r, c, D), tile + ringk_at(r, c + 1, D));
    }
  }
  // V of features d and d + 1 of window rows r and r + 1 (r even), bf16: one load a feature,
  // whose tokens lie in pairs.
  static __device__ __forceinline__ void win_v(const AppendPagesArgs &a, const Win *tile, int r, int d,
                                               int D, Pair &t0, Pair &t1) {
    const Win *p = tile + ringv_at(r, d, D), *q = tile + ringv_at(r, d + 1, D);
    uint32_t y = 0, z = 0;
    if (in_bounds(a.ctl, p, 4) && in_bounds(a.ctl, q, 4)) {
      y = *reinterpret_cast<const uint32_t *>(p);
      z = *reinterpret_cast<const uint32_t *>(q);
    }
    t0.w = __byte_perm(y, z, 0x5410);
    t1.w = __byte_perm(y, z, 0x7632);
  }
};

// One work entry and head: what the step does with 32-token group g of slot s.
struct GroupWork {
  int s, g, h, before, after, c1, w0, w1, row0;
};

__device__ __forceinline__ size_t row_elem(const AppendPagesArgs &a, const GroupWork &w, int pos,
                                           bool v) {
  const int64_t row = w.row0 + pos - w.before;
  return static_cast<size_t>(v ? row * a.r.vsr + static_cast<int64_t>(w.h) * a.r.vsh
                               : row * a.r.ksr + static_cast<int64_t>(w.h) * a.r.ksh);
}

// K or V of the new tokens of window group g into its tile, eight elements of a row at a
// time (a tile's K keeps them together, its V has them apart).
template <typename In, typename Win, int kD>
__device__ __forceinline__ void write_tile(const AppendPagesArgs &a, const GroupWork &w, bool v,
                                           int g) {
  using T = Types<In, Win>;
  const int D = kD ? kD : a.d.D, p0 = max(w.before, 32 * g), p1 = min(w.after, 32 * g + 32), pieces = D / 8;
  const size_t tile = a.d.tile_at(w.s, w.h, g);
  Win *ring = static_cast<Win *>(a.d.ring);
  for (int i = threadIdx.x; i < (p1 - p0) * pieces; i += blockDim.x) {
    const int pos = p0 + i / pieces, d = 8 * (i % pieces), r = pos & 31;
    const In *row = static_cast<const In *>(v ? a.r.v : a.r.k) + row_elem(a, w, pos, v) + d;
    typename T::Pair y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = T::row2(a, row + 2 * k);
    if (v) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        Win *o = ring + tile + 32 * D + ringv_at(r, d + k, D);
        if (in_bounds(a.ctl, o, sizeof(Win))) store_from_f32(o, k & 1 ? y[k / 2].hi() : y[k / 2].lo());
      }
    } else {
      Win *o = ring + tile + ringk_at(r, d, D);  // order 0 4 1 5 2 6 3 7
      if (!in_bounds(a.ctl, o, 8 * sizeof(Win))) continue;
      if constexpr (T::kBf16) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(
            __byte_perm(y[0].w, y[2].w, 0x5410), __byte_perm(y[0].w, y[2].w, 0x7632),
            __byte_perm(y[1].w, y[3].w, 0x5410), __byte_perm(y[1].w, y[3].w, 0x7632));
      } else {
        reinterpret_cast<float4 *>(o)[0] = make_float4(y[0].lo(), y[2].lo(), y[0].hi(), y[2].hi());
        reinterpret_cast<float4 *>(o)[1] = make_float4(y[1].lo(), y[3].lo(), y[1].hi(), y[3].hi());
      }
    }
  }
}

// K of a group, the first half of its record: thread p has channels 2p and 2p + 1.
template <typename In, typename Win, int kD>
__device__ __forceinline__ void pack_k(const AppendPagesArgs &a, const GroupWork &w, uint8_t *rec,
                                       int p) {
  using T = Types<In, Win>;
  const int D = kD ? kD : a.d.D, t0 = 32 * w.g;
  if (2 * p >= D) return;
  typename T::Pair x[32];
  if (t0 >= w.before) {  // (the usual group of a prompt)
    const In *row = static_cast<const In *>(a.r.k) + row_elem(a, w, t0, false) + 2 * p;
#pragma unroll
    for (int t = 0; t < 32; ++t) x[t] = T::row2(a, row + static_cast<int64_t>(t) * a.r.ksr);
  } else {
    const In *row = static_cast<const In *>(a.r.k) + row_elem(a, w, t0, false) + 2 * p;
    const Win *tile = static_cast<const Win *>(a.d.ring) + a.d.tile_at(w.s, w.h, w.g);
#pragma unroll
    for (int t = 0; t < 32; ++t)
      x[t] = t0 + t < w.before ? T::win_k(a, tile, t, 2 * p, D)
                               : T::row2(a, row + static_cast<int64_t>(t) * a.r.ksr);
  }
  float a0, a1;
  if constexpr (T::kBf16) {
    uint32_t m = x[0].w;
#pragma unroll
    for (int t = 1; t < 32; ++t) m = max_abs2(m, x[t].w);
    a0 = fmaxf(fabsf(bf_lo(m)), 0.0f);  // (of NaNs alone: 0)
    a1 = fmaxf(fabsf(bf_hi(m)), 0.0f);
  } else {
    a0 = a1 = 0.0f;
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      a0 = fmaxf(a0, fabsf(x[t].lo()));
      a1 = fmaxf(a1, fabsf(x[t].hi()));
    }
  }
  const bool fast = T::kBf16 && recip_ok(a0) && recip_ok(a1);
  const float s0 = fast ? scale_recip(a0) : int4_scale(a0);
  const float s1 = fast ? scale_recip(a1) : int4_scale(a1);
  float *ks = reinterpret_cast<float *>(rec + rec_kscale(D));
  ks[kscale_at(2 * p, D)] = s0;
  ks[kscale_at(2 * p + 1, D)] = s1;
  if (fast) {
    if constexpr (T::kBf16) {
      const uint64_t ns = pair64(-s0, -s1), r = pair64(recip_of(s0), recip_of(s1));
#pragma unroll
      for (int t = 0; t < 32; ++t)
        rec[t * (D / 2) + p] =
            static_cast<uint8_t>(code_byte_pair(x[t].w << 16, x[t].w & 0xffff0000u, ns, r));
    }
  } else if constexpr (T::kBf16) {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      rec[t * (D / 2) + p] = static_cast<uint8_t>(code_byte_div(x[t].lo(), x[t].hi(), s0, s1));
  } else {
    const float r0 = recip_or_nan(a0, s0), r1 = recip_or_nan(a1, s1);
#pragma unroll
    for (int t = 0; t < 32; ++t)
      rec[t * (D / 2) + p] =
          static_cast<uint8_t>(code_byte_f32(x[t].lo(), x[t].hi(), s0, s1, r0, r1));
  }
}

// V of a group, the second half of its record: thread i has features 32 b + 4 e .. + 3 of the 16 tokens of half m, i = (m,
// b, e); every lane of a warp takes part in the exchanges.
template <typename In, typename Win, int kD>
__device__ __forceinline__ void pack_v(const AppendPagesArgs &a, const GroupWork &w, uint8_t *rec,
                                       int i) {
  using T = Types<In, Win>;
  const int D = kD ? kD : a.d.D, nb = D / 32, m = i / (8 * nb), b = i / 8 % nb, e = i & 7, d0 = 32 * b + 4 * e;
  const bool live = m < 2;
  const int t0 = 32 * w.g + 16 * m;
  typename T::Pair x[16][2];
  const In *row = static_cast<const In *>(a.r.v) + row_elem(a, w, t0, true) + d0;
  if (!live) {
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      x[t][0].set(0.0f, 0.0f);
      x[t][1].set(0.0f, 0.0f);
    }
  } else if (t0 >= w.before) {
#pragma unroll
    for (int t = 0; t < 16; ++t)
      T::row4(a, row + static_cast<int64_t>(t) * a.r.vsr, x[t]);
  } else {
    const Win *tile = static_cast<const Win *>(a.d.ring) + a.d.tile_at(w.s, w.h, w.g) + 32 * D;
    if constexpr (T::kBf16) {
      // (the window has both tokens of a pair, written or not)
#pragma unroll
      for (int t = 0; t < 16; t += 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (t0 + t < w.before)
            T::win_v(a, tile, 16 * m + t, d0 + 2 * k, D, x[t][k], x[t + 1][k]);
          else
            x[t][k] = T::row2(a, row + static_cast<int64_t>(t) * a.r.vsr + 2 * k);
          if (t0 + t + 1 >= w.before)
            x[t + 1][k] = T::row2(a, row + static_cast<int64_t>(t + 1) * a.r.vsr + 2 * k);
        }
    } else {
#pragma unroll
      for (int t = 0; t < 16; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          x[t][k] = t0 + t < w.before ? T::win2(a, tile + ringv_at(16 * m + t, d0 + 2 * k, D),
                                                tile + ringv_at(16 * m + t, d0 + 2 * k + 1, D))
                                      : T::row2(a, row + static_cast<int64_t>(t) * a.r.vsr + 2 * k);
    }
  }
  // maxima of tokens 2n and 2n + 1; lane e keeps those of its own two
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    float u, v;
    if constexpr (T::kBf16) {
      const uint32_t p = max_abs2(x[2 * n][0].w, x[2 * n][1].w);
      const uint32_t q = max_abs2(x[2 * n + 1][0].w, x[2 * n + 1][1].w);
      uint32_t y = max_abs2(__byte_perm(p, q, 0x5410), __byte_perm(p, q, 0x7632));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) y = max_abs2(y, __shfl_xor_sync(~0u, y, o));
      u = bf_lo(y);
      v = bf_hi(y);
    } else {
      u = fmaxf(fmaxf(fabsf(x[2 * n][0].lo()), fabsf(x[2 * n][0].hi())),
                fmaxf(fabsf(x[2 * n][1].lo()), fabsf(x[2 * n][1].hi())));
      v = fmaxf(fmaxf(fabsf(x[2 * n + 1][0].lo()), fabsf(x[2 * n + 1][0].hi())),
                fmaxf(fabsf(x[2 * n + 1][1].lo()), fabsf(x[2 * n + 1][1].hi())));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        u = fmaxf(u, __shfl_xor_sync(~0u, u, o));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
      }
    }
    if (n == e) {
      m0 = fmaxf(fabsf(u), 0.0f);  // (of NaNs alone: 0)
      m1 = fmaxf(fabsf(v), 0.0f);
    }
  }
  // (the eight lanes of a token have all of its tokens' maxima between them)
  const bool fast = __all_sync(~0u, T::kBf16 && recip_ok(m0) && recip_ok(m1));
  const float s0 = fast ? scale_recip(m0) : int4_scale(m0);
  const float s1 = fast ? scale_recip(m1) : int4_scale(m1);
  // [half and block][t][token 2t or 2t + 1]: -scale of the token and of the one 8 behind it,
  // then their reciprocals
  float *aux = reinterpret_cast<float *>(rec + 20 * D) + (i >> 3) * 32;
  {
    float *o = aux + (e & 3) * 8 + (e >> 2);
    o[0] = -s0;
    o[4] = -s1;
    if (T::kBf16) {
      o[2] = fast ? recip_of(s0) : 0.0f;
      o[6] = fast ? recip_of(s1) : 0.0f;
    } else {
      o[2] = recip_or_nan(m0, s0);
      o[6] = recip_or_nan(m1, s1);
    }
  }
  __syncwarp();
  if (live) {
    float *vs = reinterpret_cast<float *>(rec + rec_vscale(D) - rec_vcode(D));
    vs[vscale_at(16 * m + 2 * e, b, D)] = s0;
    vs[vscale_at(16 * m + 2 * e + 1, b, D)] = s1;
  }
  uint32_t *words = reinterpret_cast<uint32_t *>(rec);
  const bool upper = e & 2;  // features y + 8
  const int f = 2 * b + (e >> 2), g0 = 4 * (e & 1) + (upper ? 2 : 0);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    // bytes: features j, j + 1 of token 2t, then of 2t + 1; low nibbles are the tokens
    // themselves, high ones those 8 behind
    uint32_t c01 = 0, c23 = 0;
    if constexpr (T::kBf16) {
      if (fast) {  // (low and high codes apart: one mask for four bytes)
        uint32_t lo[2][4], hi[2][4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float4 sc = *reinterpret_cast<const float4 *>(aux + 8 * t + 4 * z);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t p = x[2 * t + z][j >> 1].w, q = x[2 * t + z + 8][j >> 1].w;
            lo[z][j] = j & 1 ? p & 0xffff0000u : p << 16;
            hi[z][j] = j & 1 ? q & 0xffff0000u : q << 16;
            code8_pair(lo[z][j], hi[z][j], pair64(sc.x, sc.y), pair64(sc.z, sc.w));
          }
        }
        c01 = (four_bytes(hi[0][0], hi[0][1], hi[1][0], hi[1][1]) << 4 & 0xf0f0f0f0u) |
              (four_bytes(lo[0][0], lo[0][1], lo[1][0], lo[1][1]) & 0x0f0f0f0fu);
        c23 = (four_bytes(hi[0][2], hi[0][3], hi[1][2], hi[1][3]) << 4 & 0xf0f0f0f0u) |
              (four_bytes(lo[0][2], lo[0][3], lo[1][2], lo[1][3]) & 0x0f0f0f0fu);
      }
    }
    if (!fast) {
      uint32_t c[2][4];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float4 sc = *reinterpret_cast<const float4 *>(aux + 8 * t + 4 * z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const auto &p = x[2 * t + z][j >> 1], &q = x[2 * t + z + 8][j >> 1];
          const float y0 = j & 1 ? p.hi() : p.lo(), y8 = j & 1 ? q.hi() : q.lo();
          if constexpr (T::kBf16)
            c[z][j] = code_byte_div(y0, y8, -sc.x, -sc.y);
          else
            c[z][j] = code_byte_f32(y0, y8, -sc.x, -sc.y, sc.z, sc.w);
        }
      }
      c01 = four_bytes(c[0][0], c[0][1], c[1][0], c[1][1]);
      c23 = four_bytes(c[0][2], c[0][3], c[1][2], c[1][3]);
    }
    const uint32_t other = __shfl_xor_sync(~0u, upper ? c01 : c23, 2);
    const uint32_t lo = upper ? other : c01, hi = upper ? c23 : other;
    if (live) {
      words[vword_at(m, g0, t, f, D)] = __byte_perm(lo, hi, 0x6240);
      words[vword_at(m, g0 + 1, t, f, D)] = __byte_perm(lo, hi, 0x7351);
    }
  }
}

__device__ __forceinline__ void bulk_s2g(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A CTA per (group of the work list, head, K or V). A group that is packed may have
// tokens in a tile of the window that the step's new tokens take over: the CTA that packs
// it writes them too, behind its own reads, and the tile's own entry leaves them to it, so
// no order between CTAs is needed.
template <typename In, typename Win, int kD>
__global__ void __launch_bounds__(128, sizeof(Win) == 2 ? 8 : 4)
    append_pages_kernel(const AppendPagesArgs a) {
  extern __shared__ __align__(16) uint8_t rec[];
  wait_prior_grid();
  allow_next_grid();
  const int T = a.d.tiles, D = kD ? kD : a.d.D;
  unsigned items = 0;
  if (in_bounds(a.ctl, a.counts, 16)) items = 2u * max(0, min(a.counts[1], a.cap_work)) * a.d.Hkv;
  for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {  // (up to 2^31 of them)
    GroupWork w;
    const bool v = it & 1;
    const int e = static_cast<int>((it >> 1) / a.d.Hkv);
    w.h = static_cast<int>((it >> 1) - static_cast<unsigned>(e) * a.d.Hkv);
    const int4 *p = reinterpret_cast<const int4 *>(a.work) + 2 * static_cast<size_t>(e);
    if (!in_bounds(a.ctl, p, 32)) continue;
    const int4 e0 = p[0], e1 = p[1];
    w.s = e0.x;
    w.g = e0.y;
    const int page = e0.z;
    w.before = e0.w;
    w.after = e1.x;
    w.row0 = e1.y;
    w.c1 = paged_cut(w.after, a.d.window) >> 5;
    w.w0 = max(w.before >> 5, w.c1);
    w.w1 = (w.after + 31) >> 5;
    if (w.g >= w.c1) {
      // the old group in this tile, if it moves into the pages, has its CTA write here
      const int c0 = paged_cut(w.before, a.d.window) >> 5, ob = (w.before + 31) >> 5;
      const int o = ob - 1 - (((ob - 1 - w.g) % T) + T) % T;
      if (!(ob > c0 && o >= c0 && o < w.c1)) write_tile<In, Win, kD>(a, w, v, w.g);
      continue;
    }
    if (v)
      pack_v<In, Win, kD>(a, w, rec, threadIdx.x);
    else
      pack_k<In, Win, kD>(a, w, rec, threadIdx.x);
    __syncthreads();
    if (threadIdx.x == 0) {
      uint8_t *dst = nullptr;
      if (page >= 0 && page < a.d.n_pages)
        dst = a.d.record_at(page, w.g & ((1 << a.d.gpp_log2()) - 1), w.h) + (v ? rec_vcode(D) : 0);
      if (!dst)
        flag_error(a.ctl, KVQ_DEV_INDEX);
      else if (in_bounds(a.ctl, dst, 20 * D))
        bulk_s2g(dst, smem_u32(rec), 20 * D);
    }
    // the window group that takes over this group's tile, whose values have all been read
    if (32 * w.g < w.before) {
      const int g = w.w0 + (((w.g - w.w0) % T) + T) % T;
      if (g < w.w1) write_tile<In, Win, kD>(a, w, v, g);
    }
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();  // the record is free again
  }
  if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

struct PageValuesArgs {
  PagedDims d;
  const int32_t *slot, *pos;
  void *k, *v;
  int n, out_dt;
  KernelCtl ctl;
};

constexpr int kVlRows = 16;  // list rows of a pair of warps

// 8 or 16 consecutive values (wide: the address is a multiple of 32 bytes).
template <typename Out>
__device__ __forceinline__ void store8(const KernelCtl &ctl, Out *o, const float (&y)[8]) {
  if (!in_bounds(ctl, o, 8 * sizeof(Out))) return;
  if constexpr (sizeof(Out) == 4) {
    reinterpret_cast<float4 *>(o)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4 *>(o)[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    *reinterpret_cast<uint4 *>(o) = make_uint4(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]),
                                               pack_bf2(y[4], y[5]), pack_bf2(y[6], y[7]));
  }
}
template <typename Out>
__device__ __forceinline__ void store16(const KernelCtl &ctl, Out *o, const float (&lo)[8],
                                        const float (&hi)[8], bool wide) {
  if (sizeof(Out) == 4 || !wide) {
    store8(ctl, o, lo);
    store8(ctl, o + 8, hi);
  } else if (in_bounds(ctl, o, 32)) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o),
                 "r"(pack_bf2(lo[0], lo[1])), "r"(pack_bf2(lo[2], lo[3])),
                 "r"(pack_bf2(lo[4], lo[5])), "r"(pack_bf2(lo[6], lo[7])),
                 "r"(pack_bf2(hi[0], hi[1])), "r"(pack_bf2(hi[2], hi[3])),
                 "r"(pack_bf2(hi[4], hi[5])), "r"(pack_bf2(hi[6], hi[7]))
                 : "memory");
  }
}

// The scales of eight channels from d0 on, as a record has them: channels 0 4 1 5, and 64
// bytes on 2 6 3 7.
__device__ __forceinline__ void load_kscales(const uint8_t *rec, int d0, int D, float (&sc)[8]) {
  const float *ks = reinterpret_cast<const float *>(rec + rec_kscale(D)) + kscale_at(d0, D);
  const float4 x = *reinterpret_cast<const float4 *>(ks), y = *reinterpret_cast<const float4 *>(ks + 16);
  sc[0] = x.x;
  sc[1] = x.z;
  sc[2] = y.x;
  sc[3] = y.z;
  sc[4] = x.y;
  sc[5] = x.w;
  sc[6] = y.y;
  sc[7] = y.w;
}

// Tokens [16 m, 16 m + 16) of a record, those with list index i0 + token in [0, 16), to
// the list rows from row0 on: K, or V. A lane takes 16 channels of K of every token in its
// turn, or the eight words of V of 16 features and four tokens: every byte is read once.
template <typename Out, int D>
__device__ __forceinline__ void read_half(const PageValuesArgs &a, const uint8_t *rec, bool v, int m,
                                          int i0, long row0, int h, bool wide, int lane) {
  constexpr int kChunks = D / 16, kRows = 32 / kChunks;
  float lo[8], hi[8];
  const size_t o0 = (static_cast<size_t>(row0) * a.d.Hkv + h) * D;
  const size_t step = static_cast<size_t>(a.d.Hkv) * D;
  if (!v) {
    const int c = lane & (kChunks - 1), r0 = lane / kChunks;
    uint2 w[16 / kRows];
#pragma unroll
    for (int x = 0; x < 16 / kRows; ++x)
      w[x] = *reinterpret_cast<const uint2 *>(rec + (16 * m + kRows * x + r0) * (D / 2) + 8 * c);
    float s0[8], s1[8];
    load_kscales(rec, 16 * c, D, s0);
    load_kscales(rec, 16 * c + 8, D, s1);
#pragma unroll
    for (int x = 0; x < 16 / kRows; ++x) {
      const int i = i0 + kRows * x + r0;
      if (i0 + kRows * x <= -kRows || i0 + kRows * x >= kVlRows) continue;  // (none of them)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo[j] = (static_cast<int>(w[x].x >> (4 * j) & 15) - 8) * s0[j];
        hi[j] = (static_cast<int>(w[x].y >> (4 * j) & 15) - 8) * s1[j];
      }
      if (i >= 0 && i < kVlRows)
        store16(a.ctl, static_cast<Out *>(a.k) + o0 + i * step + 16 * c, lo, hi, wide);
    }
    return;
  }
  if (lane >= 4 * kChunks) return;
  const int t = lane >> 2 & 3, f = (lane >> 4) * 4 + (lane & 3);
  const uint32_t *vw = reinterpret_cast<const uint32_t *>(rec + rec_vcode(D)) + vword_at(m, 0, t, f, D);
  const float *vs = reinterpret_cast<const float *>(rec + rec_vscale(D));
  uint32_t w[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) w[g] = vw[16 * g];
  const float2 sa = *reinterpret_cast<const float2 *>(vs + vscale_at(16 * m + 2 * t, f >> 1, D));
  const float2 sb = *reinterpret_cast<const float2 *>(vs + vscale_at(16 * m + 2 * t + 8, f >> 1, D));
#pragma unroll
  for (int z = 0; z < 4; ++z) {  // tokens 2t, 2t + 8, 2t + 1, 2t + 9
    const int i = i0 + 2 * t + 8 * (z & 1) + (z >> 1), sh = 4 * (z & 1) + 16 * (z >> 1);
    const float s = z == 0 ? sa.x : z == 1 ? sb.x : z == 2 ? sa.y : sb.y;
    if (i - 2 * t < -6 || i - 2 * t >= kVlRows) continue;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      lo[g] = (static_cast<int>(w[g] >> sh & 15) - 8) * s;
      hi[g] = (static_cast<int>(w[g] >> (sh + 8) & 15) - 8) * s;
    }
    if (i >= 0 && i < kVlRows)
      store16(a.ctl, static_cast<Out *>(a.v) + o0 + i * step + 16 * f, lo, hi, wide);
  }
}

// Two warps per 16 list rows of one head. Lane i < 16 finds row i's record or tile (or that
// it has none). Rows that are consecutive int4 tokens of one request (a prefix) are read
// half a record at a time, K by one warp and V by the other; others one by one, eight
// rows a warp: a token alone touches four times the bytes of its V codes. kD: the head
// dim, or 0 for one of the others. 56 registers: 112,000 rows of two heads (153 MB in and
// out, runs that start inside a half record) 31.9 us, 4.7 TB/s; with 64 registers 33.1.
// What it waits for are three loads in a row (list, then length and page together, then the
// record): 4,099 scattered rows 4.8 us, 5.0 with the page read after the length was checked.
template <typename Out, int kD>
__global__ void __launch_bounds__(128, 9) page_values_kernel(const PageValuesArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int D = kD ? kD : a.d.D, pieces = D / 8, lane = threadIdx.x & 31;
  const long unit = (blockIdx.x * static_cast<long>(blockDim.x) + threadIdx.x) >> 6;
  const int h = static_cast<int>(unit % a.d.Hkv), second = threadIdx.x >> 5 & 1;
  const long row0 = unit / a.d.Hkv * kVlRows;
  if (row0 >= a.n) return;
  // at: byte offset of the record, or (kind 2) element offset of the tile; kind 0: none
  size_t at = 0;
  int kind = 0, s = -1, pos = 0;
  if (lane < kVlRows && row0 + lane < a.n) {
    const int32_t *ps = a.slot + row0 + lane, *pp = a.pos + row0 + lane;
    if (in_bounds(a.ctl, ps, 4) && in_bounds(a.ctl, pp, 4)) {
      s = *ps;
      pos = *pp;
      // (the length and the page are on the way together)
      const int g = pos >> 5, j = pos >> a.d.page_log2;
      const bool there = s >= 0 && s < a.d.slots && pos >= 0;
      int len = -1, page = -1;
      if (there && in_bounds(a.ctl, a.d.lengths + s, 4)) len = a.d.lengths[s];
      if (there && j < a.d.max_pages) {
        const int32_t *pe = a.d.table + static_cast<size_t>(s) * a.d.max_pages + j;
        if (in_bounds(a.ctl, pe, 4)) page = *pe;
      }
      if (s == -1) {
        kind = 0;
      } else if (!a.d.holds(len) || pos < 0 || pos >= len) {
        flag_error(a.ctl, KVQ_DEV_INDEX);
      } else if (pos < paged_cut(len, a.d.window)) {
        if (page < 0 || page >= a.d.n_pages) {
          flag_error(a.ctl, KVQ_DEV_INDEX);
        } else {
          const uint8_t *rec = a.d.record_at(page, g & ((1 << a.d.gpp_log2()) - 1), h);
          at = rec - a.d.pool;
          kind = in_bounds(a.ctl, rec, 40 * D);
        }
      } else {
        at = a.d.tile_at(s, h, g);
        const size_t b = el_bytes(a.d.win_dt);
        kind = in_bounds(a.ctl, static_cast<const uint8_t *>(a.d.ring) + at * b, 64 * D * b) ? 2 : 0;
      }
    }
  }
  if constexpr (kD != 0) {
    const int s0 = __shfl_sync(~0u, s, 0), p0 = __shfl_sync(~0u, pos, 0);
    if (__all_sync(~0u, lane >= kVlRows || (kind == 1 && s == s0 && pos == p0 + lane))) {
      const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 31) == 0;
      for (int q = p0 >> 4; q <= (p0 + kVlRows - 1) >> 4; ++q) {
        const int i0 = 16 * q - p0;
        const size_t off = __shfl_sync(~0u, static_cast<unsigned long long>(at), max(0, i0));
        read_half<Out, kD>(a, a.d.pool + off, second, q & 1, i0, row0, h, wide, lane);
      }
      return;
    }
  }
  const int passes = pieces / 4;
#pragma unroll 4
  for (int ps = 0; ps < passes; ++ps) {
    const int task = 32 * ps + lane, r8 = task / pieces, p = task - r8 * pieces, d0 = 8 * p;
    const int i = 8 * second + r8;
    const int kd = __shfl_sync(~0u, kind, i), r = __shfl_sync(~0u, pos, i) & 31;
    const size_t off = __shfl_sync(~0u, static_cast<unsigned long long>(at), i);
    if (kd == 0) continue;
    float k[8], v[8];
    if (kd == 1) {
      const uint8_t *rec = a.d.pool + off;
      const uint32_t kw = *reinterpret_cast<const uint32_t *>(rec + r * (D / 2) + 4 * p);
      float sc[8];
      load_kscales(rec, d0, D, sc);
      const uint32_t *vw = reinterpret_cast<const uint32_t *>(rec + rec_vcode(D)) +
                           vword_at(r >> 4, 0, (r & 7) >> 1, p >> 1, D);
      const int step = D % 64 == 0 ? 16 : 8;  // words from feature to feature
      const float vs = reinterpret_cast<const float *>(rec + rec_vscale(D))[vscale_at(r, d0 >> 5, D)];
      const int sh = 4 * (4 * (r & 1) + 2 * (p & 1) + (r >> 3 & 1));
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = vw[j * step];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] = (static_cast<int>(kw >> (4 * j) & 15) - 8) * sc[j];
        v[j] = (static_cast<int>(w[j] >> sh & 15) - 8) * vs;
      }
    } else {
      const size_t ek = off + ringk_at(r, d0, D), ev = off + 32 * D + ringv_at(r, d0, D);
      if (a.d.win_dt == KVQ_F32) {
        const float *x = static_cast<const float *>(a.d.ring);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          k[j] = x[ek + 2 * (j & 3) + (j >> 2)];
          v[j] = x[ev + 32 * j];
        }
      } else {
        const uint16_t *x = static_cast<const uint16_t *>(a.d.ring);
        const uint4 y = *reinterpret_cast<const uint4 *>(x + ek);
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          k[j] = j < 4 ? bf_lo(w[j & 3]) : bf_hi(w[j & 3]);
          v[j] = bf16_to_f32(x[ev + 32 * j]);
        }
      }
    }
    const size_t o = (static_cast<size_t>(row0 + i) * a.d.Hkv + h) * D + d0;
    store8(a.ctl, static_cast<Out *>(a.k) + o, k);
    store8(a.ctl, static_cast<Out *>(a.v) + o, v);
  }
}

template <typename Out>
void launch_values(const PageValuesArgs &a, cudaStream_t s) {
  const long units = static_cast<long>((a.n + kVlRows - 1) / kVlRows) * a.d.Hkv;
  const dim3 grid(static_cast<unsigned>((units + 1) / 2));
  if (a.d.D == 128)
    launch_dependent(page_values_kernel<Out, 128>, grid, dim3(128), 0, s, a);
  else if (a.d.D == 64)
    launch_dependent(page_values_kernel<Out, 64>, grid, dim3(128), 0, s, a);
  else
    launch_dependent(page_values_kernel<Out, 0>, grid, dim3(128), 0, s, a);
}

template <typename In, typename Win, int kD>
void launch_append_dim(const AppendPagesArgs &a, int num_sms, cudaStream_t s) {
  const int threads = (a.d.D / 2 + 31) / 32 * 32;
  const long items = 2L * a.cap_work * a.d.Hkv;
  const int grid = static_cast<int>(std::min<long>(items, 16L * num_sms));
  launch_dependent(append_pages_kernel<In, Win, kD>, dim3(grid), dim3(threads),
                   20 * a.d.D + threads * 16, s, a);
}

template <typename In, typename Win>
void launch_append_typed(const AppendPagesArgs &a, int num_sms, cudaStream_t s) {
  if (a.d.D == 128)
    launch_append_dim<In, Win, 128>(a, num_sms, s);
  else if (a.d.D == 64)
    launch_append_dim<In, Win, 64>(a, num_sms, s);
  else
    launch_append_dim<In, Win, 0>(a, num_sms, s);
}

}  // namespace

int launch_append_pages(const PagedDims &d, const kvq_page_plan &p, const PageRows &r,
                        const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  AppendPagesArgs a;
  a.d = d;
  a.r = r;
  a.work = p.work;
  a.counts = p.counts;
  // (the entries a step of these rows can fill)
  a.cap_work = page_work_bound(d.window, d.slots, p.rows);
  a.ctl = ctl;
  if (r.dtype == KVQ_F32) {
    if (d.win_dt == KVQ_F32)
      launch_append_typed<float, float>(a, num_sms, s);
    else
      launch_append_typed<float, __nv_bfloat16>(a, num_sms, s);
  } else if (d.win_dt == KVQ_F32) {
    launch_append_typed<__nv_bfloat16, float>(a, num_sms, s);
  } else {
    launch_append_typed<__nv_bfloat16, __nv_bfloat16>(a, num_sms, s);
  }
  return 1;
}

int launch_page_values(const PagedDims &d, const int32_t *slot, const int32_t *pos, int n,
                       void *k, void *v, int out_dt, const KernelCtl &ctl, cudaStream_t s) {
  PageValuesArgs a;
  a.d = d;
  a.slot = slot;
  a.pos = pos;
  a.k = k;
  a.v = v;
  a.n = n;
  a.out_dt = out_dt;
  a.ctl = ctl;
  if (out_dt == KVQ_F32)
    launch_values<float>(a, s);
  else
    launch_values<__nv_bfloat16>(a, s);
  return 1;
}

}  // namespace kvq
