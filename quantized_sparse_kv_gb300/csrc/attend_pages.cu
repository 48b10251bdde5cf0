// kv_attend_pages on the tensor cores: one query row per new token over the pages and the
// window of its request, split over the length and joined (D = 64 or 128, bf16 windows).
//
// Work split. A unit is (query row, KV head, up to eight of its query heads: the columns of an
// MMA; a KV head with more is read once for every eight, and a request with several rows once
// for each). Its items are its int4 groups taken four at a time, then its window tiles of 32
// tokens. The items of all units lie end to end and the persistent grid (three CTAs per SM)
// takes equal contiguous slices, whatever the requests' lengths are; each CTA finds its slice
// from the lengths itself (one sum over the rows), so nothing about them is known to the host. A
// unit that one CTA has from end to end is finished there; the others leave a partial
// (maximum, sum, output before the division) per CTA, which a second kernel joins.
//
// Inside a CTA. Warp 4 loads: lanes 0-3 copy one record each of an item (a group's codes
// and scales of K and V are 40 D consecutive bytes) into a ring of stages, from table
// entries that the whole warp reads eight items ahead. Warps 0-3 take one group each, or
// two of them 16 tokens of a window tile.
//
// Scores: mma.sync m16n8k16 with tokens as rows and the query heads as columns. The K
// scales of a group are multiplied into q; the codes need no conversion: a nibble n + 8
// masked out of a word is the fp16 subnormal (n + 8) 2^-24, or 2^-20 four bits higher,
// which the tensor cores multiply exactly. The factor of 16 between the two is in q (4 and
// 1/4), and the 8s are taken off by one product with a constant -8 for all 32 tokens:
// sum (c - 8) q' = sum c q' - 8 sum q', the same rounded q' in both, so nothing is lost.
// Five logic operations make the operands of eight codes that way, where a conversion to
// centred fp16 takes eleven.
//
// P V: V codes as stored (a record's words hold the four operand registers of one MMA),
// features as rows, tokens as the inner dimension. The V scale of a (token, 32 features) is
// multiplied into P, one copy of P per 32 features: at D = 128 16 packed products a lane and
// group, where scaling the group's 4,096 values would take 64. The 8s come off through a tile of
// row sums of those copies. The upper nibbles' factor 1/16 is in the exponent of the second
// half of P.
//
// Roundings, each to the 11 bits of an fp16 operand: q * scale (also of fp32 q, and for the
// window, which has no copy of q of its own), a K scale, their product; P, a V scale, their
// product. P of the window keeps 15 bits. The sums are fp32.
//
// Softmax in the log2 domain, fp32 state. The reference of a head is raised only when
// score + log2(largest V scale of the group) exceeds it by more than kBias + kLazy, to
// kBias below. Products P * scale stay within fp16 (below 2^12), and P and the products
// keep 11 bits down to 2^-17 of the largest, the scales down to 2^-10 of their group's: scales of
// 2 and more, or below 2^-4, give a power of two to P, so that P has the same range of
// exponents whatever the magnitude of V.
//
// 64 requests of 16 to 32 thousand tokens, 16 heads over 2 (510 MB): 90.7 us, 5.6 TB/s, of which
// 1.5 us until a CTA has its slice, 3.8 until its first item, 6.5 TB/s then until the first
// CTAs end; 10 lie between the mean and the last CTA's end (the first CTA of an SM is
// ahead of its third), 3 are the join. One request of 700 tokens: 8.5 us. D = 64 is bound by the
// MMAs and their operands (336 MB: 84 us; with four CTAs per SM 87, with five 107).
#include <algorithm>

#include "int4_dequant.cuh"
#include "paged.cuh"

namespace kvq {
namespace {

constexpr int kApHeads = 8;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kCtasPerSm = 3;
// Rows whose lengths are held in shared memory: all, up to a row a thread, else the first of the
// slice.
constexpr int kRowsHeld = 192;
static_assert(kRowsHeld >= kThreads);
constexpr float kBias = 7.0f, kLazy = 4.0f;
constexpr float kNone = -1e30f;  // a reference below every score
constexpr float kHeld = 16777216.0f;  // 2^24: O is held times its inverse until it is divided
// -8 as the codes are read: low nibbles 2^-24, high nibbles 2^-20
constexpr uint32_t kLo8 = 0x80088008u, kHi8 = 0x80808080u;

template <int D>
struct Cfg {
  static constexpr int kRecord = 40 * D;
  static constexpr int kStage = 4 * kRecord;  // a window tile takes 128 D
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kPart = D + 4;  // O, m, l of a head, padded to 16 bytes
};

struct AttendPagesArgs {
  PagedDims d;
  const void *q;
  void *out;
  const int32_t *slot, *pos;
  // [unit]: partial of its first item and CTA of its last one; first = -1: finished
  int32_t *first, *last;
  // [CTA][2][8][kPart]: only the first and the last unit of a slice can have others' items
  float *part;
  float scale_log2;
  int q_dt, out_dt, rows, Hq, G, chunks, ctas;
  KernelCtl ctl;
};

__device__ __forceinline__ int units_per_row(const AttendPagesArgs &a) {
  return a.d.Hkv * a.chunks;
}

// Tokens that a row attends (-1: the row is left as it was) and those of them held as int4.
struct RowInfo {
  int slot, n, cut;
};

__device__ __forceinline__ RowInfo row_info(const AttendPagesArgs &a, int row, bool flag) {
  RowInfo r;
  r.slot = row;
  r.n = -1;
  r.cut = 0;
  if (a.slot) r.slot = in_bounds(a.ctl, a.slot + row, 4) ? a.slot[row] : -1;
  int p = 0;
  if (a.pos) p = in_bounds(a.ctl, a.pos + row, 4) ? a.pos[row] : -1;
  if (r.slot == -1) return r;
  int len = -1;
  if (r.slot >= 0 && r.slot < a.d.slots && in_bounds(a.ctl, a.d.lengths + r.slot, 4))
    len = a.d.lengths[r.slot];
  bool ok = a.d.holds(len);
  r.n = len;
  r.cut = paged_cut(len, a.d.window);
  if (a.pos && ok) {
    ok = p >= 0 && p < len;
    r.n = p + 1;
  }
  if (!ok) {
    if (flag) flag_error(a.ctl, KVQ_DEV_INDEX);
    r.n = -1;
  }
  return r;
}

// int4 groups a row attends, its int4 items and all its items.
__device__ __forceinline__ int int4_groups(const RowInfo &r) {
  return r.n > 0 ? (min(r.n, r.cut) + 31) >> 5 : 0;
}
__device__ __forceinline__ int row_items(const RowInfo &r) {
  return ((int4_groups(r) + 3) >> 2) + (r.n > r.cut ? (r.n - r.cut + 31) >> 5 : 0);
}

template <int D>
struct __align__(16) Smem {
  uint8_t stage[Cfg<D>::kStages][Cfg<D>::kStage];
  float red_o[kConsumers][kApHeads / 2][D + 8];
  float red_m[kConsumers][kApHeads], red_l[kConsumers][kApHeads], red_c[kConsumers][kApHeads];
  float red_mx[kApHeads], red_ls[kApHeads];
  uint64_t full[Cfg<D>::kStages], empty[Cfg<D>::kStages];
  int valid[Cfg<D>::kStages][kConsumers];
  RowInfo row[kRowsHeld];
  long long sums[kConsumers + 1];
  int row0, held0;  // first row of the slice, and the first one held
  int abort_flag;
  int quit;  // abort_flag as all consumers see it at the end of a unit
  int at0;  // items of row0 before the slice
};

// A position in the items: unit (row, hc), item j of it.
struct Walk {
  RowInfo r;
  int row, hc, j, int4, items;

  template <int D>
  __device__ __forceinline__ void load(const AttendPagesArgs &a, const Smem<D> &sm) {
    const int i = row - sm.held0;
    if (row >= a.rows)
      r = RowInfo{-1, -1, 0};
    else
      r = i < kRowsHeld ? sm.row[i] : row_info(a, row, false);
    int4 = (int4_groups(r) + 3) >> 2;
    items = row_items(r);
  }
  template <int D>
  __device__ __forceinline__ void start(const AttendPagesArgs &a, const Smem<D> &sm) {
    row = sm.row0;
    load(a, sm);
    hc = items ? sm.at0 / items : 0;
    j = items ? sm.at0 - hc * items : 0;
  }
  template <int D>
  __device__ __forceinline__ void next_unit(const AttendPagesArgs &a, const Smem<D> &sm) {
    j = 0;
    if (++hc < units_per_row(a)) return;
    hc = 0;
    do {
      ++row;
      load(a, sm);
    } while (items == 0 && row < a.rows);
  }
  template <int D>
  __device__ __forceinline__ void next(const AttendPagesArgs &a, const Smem<D> &sm) {
    if (++j >= items) next_unit(a, sm);
  }
};

// ------------------------------------------------------------------ the arithmetic
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B (no accumulator to clear)
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
template <int D>
struct State {
  float o[D / 16][4];  // O^T / kHeld: tile f, features 16f + g and + 8, heads 2t and 2t + 1
  float c[4];          // the 8s of row block g (< D / 32): c[0], c[1] for heads 2t, 2t + 1
  float m[2], l[2];
};

template <int D>
__device__ __forceinline__ void reset(State<D> &st) {
#pragma unroll
  for (int f = 0; f < D / 16; ++f) st.o[f][0] = st.o[f][1] = st.o[f][2] = st.o[f][3] = 0.0f;
  st.c[0] = st.c[1] = st.c[2] = st.c[3] = 0.0f;
  st.m[0] = st.m[1] = kNone;
  st.l[0] = st.l[1] = 0.0f;
}

// Raise the references where mx (+ the scale's exponent) asks for it.
template <int D>
__device__ __forceinline__ void raise(State<D> &st, float mx0, float mx1) {
  if (!__any_sync(~0u, mx0 > st.m[0] + (kBias + kLazy) || mx1 > st.m[1] + (kBias + kLazy))) return;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, o));
  }
  const float n0 = fmaxf(st.m[0], mx0 - kBias), n1 = fmaxf(st.m[1], mx1 - kBias);
  const float c0 = fast_exp2(st.m[0] - n0), c1 = fast_exp2(st.m[1] - n1);
  st.m[0] = n0;
  st.m[1] = n1;
  st.l[0] *= c0;
  st.l[1] *= c1;
  st.c[0] *= c0;
  st.c[1] *= c1;
#pragma unroll
  for (int f = 0; f < D / 16; ++f) {
    st.o[f][0] *= c0;
    st.o[f][1] *= c1;
    st.o[f][2] *= c0;
    st.o[f][3] *= c1;
  }
}

// A pair of fp16 with zeros for NaNs.
__device__ __forceinline__ uint32_t no_nan(uint32_t x) {
  return x & __heq2_mask(as_h2(x), as_h2(x));
}

constexpr uint32_t kLoMask = 0x000F000Fu, kHiMask = 0x00F000F0u;

// Exponents of V scales that are told apart. Their span keeps the sum of a head, which is held
// against a reference that counts the scales, within fp32: the weight of groups at one end against
// groups at the other is lost (2^-126) only where it is below 2^-20 of theirs. Scales above
// 2^kMaxExp have 2^4 of room in the products, those below 2^kMinExp lose no bits until 2^-58.
constexpr int kMinExp = -48, kMaxExp = 52;
__device__ __forceinline__ int held_exponent(int e) { return max(kMinExp, min(kMaxExp, e)); }

constexpr int kTopExp = 55;
constexpr float kNoScale = 72057594037927936.0f;  // 2^(kTopExp + 1): from there on infinite

// Exponent of the largest V scale of a group's first `valid` tokens. Those that are not attended
// set no reference, whatever they hold. kSome: nor do scales from kNoScale on, whose values
// are NaN (else such a scale is answered by its exponent).
template <int D, bool kSome>
__device__ __forceinline__ int scale_exponent(const uint8_t *rec, int valid, int lane) {
  constexpr int V = D / 32;  // a lane's scales are of tokens lane & ~1 and the one behind it, in turn
  float x[V];
  const float *vs = reinterpret_cast<const float *>(rec + rec_vscale(D)) + V * lane;
  if constexpr (D == 128) {
    const float4 z = *reinterpret_cast<const float4 *>(vs);
    x[0] = z.x, x[1] = z.y, x[2] = z.z, x[3] = z.w;
  } else {
    const float2 z = *reinterpret_cast<const float2 *>(vs);
    x[0] = z.x, x[1] = z.y;
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (kSome && ((lane & ~1) + (i & 1) >= valid || !(x[i] < kNoScale))) x[i] = 0.0f;
    m = fmaxf(m, x[i]);
  }
  const int e = static_cast<int>(__reduce_max_sync(~0u, __float_as_uint(m)) >> 23) - 127;
  return kSome ? held_exponent(e) : e;
}
// Scales outside [2^-4, 2) are taken there by 2^-far, which P has instead: P of the reference
// is 2^7 to 2^15 then, and the smallest of its 11-bit values is 17 binades below.
__device__ __forceinline__ int far_of(int ev) { return ev - max(-4, min(0, ev)); }

// One int4 group: 32 tokens, `valid` of them attended, ev the exponent of its V scales.
// kUsual: all are attended and far_of(ev) is 0. kScaled: all are attended and no scale reaches
// kNoScale. (64 requests of 24,576 tokens: 90 us with values of 0.5 to 14 at most in a group, 93
// with larger or smaller ones.)
enum GroupKind { kUsual, kScaled, kAny };
template <int D, GroupKind kKind>
__device__ __forceinline__ void do_group(State<D> &st, const uint8_t *rec,
                                         const uint32_t (&qh)[D / 32][4], int valid, int ev, int g,
                                         int t) {
  constexpr int NB = D / 32;
  const float *ks = reinterpret_cast<const float *>(rec + rec_kscale(D)) + 4 * t;
  const float *vs = reinterpret_cast<const float *>(rec + rec_vscale(D));
  uint32_t bq[2 * NB][2];
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) {
    const float4 s = *reinterpret_cast<const float4 *>(ks + 16 * i);
    bq[i][0] = as_u32(__hmul2(as_h2(qh[i >> 1][2 * (i & 1)]), __floats2half2_rn(s.x, s.y)));
    bq[i][1] = as_u32(__hmul2(as_h2(qh[i >> 1][2 * (i & 1) + 1]), __floats2half2_rn(s.z, s.w)));
  }
  float s[2][4], e[4];
  uint32_t w[2][2][NB];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *p = rec + (16 * mt + 8 * h + g) * (D / 2) + 4 * NB * t;
      if constexpr (NB == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[mt][h][0] = x.x;
        w[mt][h][1] = x.y;
        w[mt][h][2] = x.z;
        w[mt][h][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[mt][h][0] = x.x;
        w[mt][h][1] = x.y;
      }
    }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (i == 0)
      mma_f16_first(e, kLo8, kLo8, kHi8, kHi8, bq[0][0], bq[0][1]);
    else
      mma_f16(e, kLo8, kLo8, kHi8, kHi8, bq[2 * i][0], bq[2 * i][1]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t x = w[mt][0][i], y = w[mt][1][i];
      if (i == 0)
        mma_f16_first(s[mt], x & kLoMask, y & kLoMask, x & kHiMask, y & kHiMask, bq[0][0], bq[0][1]);
      else
        mma_f16(s[mt], x & kLoMask, y & kLoMask, x & kHiMask, y & kHiMask, bq[2 * i][0],
                bq[2 * i][1]);
    }
    mma_f16(e, kLo8, kLo8, kHi8, kHi8, bq[2 * i + 1][0], bq[2 * i + 1][1]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t x = w[mt][0][i] >> 8, y = w[mt][1][i] >> 8;
      mma_f16(s[mt], x & kLoMask, y & kLoMask, x & kHiMask, y & kHiMask, bq[2 * i + 1][0],
              bq[2 * i + 1][1]);
    }
  }
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[mt][k] += e[k & 1];
      if (kKind == kAny && 16 * mt + 8 * (k >> 1) + g >= valid) s[mt][k] = -INFINITY;
    }
    mx0 = fmaxf(mx0, fmaxf(s[mt][0], s[mt][2]));
    mx1 = fmaxf(mx1, fmaxf(s[mt][1], s[mt][3]));
  }
  constexpr float kUnit = 4194304.0f;  // 2^22: low nibbles 2^-24 times 4, high ones 2^-20 / 4
  raise(st, fmaf(mx0, kUnit, static_cast<float>(ev)), fmaf(mx1, kUnit, static_cast<float>(ev)));
  const int far = kKind == kUsual ? 0 : far_of(ev);
  const float shift = kKind == kUsual ? 0.0f : static_cast<float>(far);
  const float back = kKind == kUsual ? 1.0f : __int_as_float((127 - far) << 23);  // 2^-far
  float sum[2] = {0.0f, 0.0f}, sum16[2] = {0.0f, 0.0f};
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      s[mt][k] = fast_exp2(fmaf(s[mt][k], kUnit, shift - st.m[k]));
      s[mt][k + 2] = fast_exp2(fmaf(s[mt][k + 2], kUnit, shift - 4.0f - st.m[k]));
      sum[k] += s[mt][k];
      sum16[k] += s[mt][k + 2];
    }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (kKind == kUsual)
      st.l[k] += fmaf(sum16[k], 16.0f, sum[k]);
    else
      st.l[k] = fmaf(fmaf(sum16[k], 16.0f, sum[k]), back, st.l[k]);
  }

#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const uint32_t p0 = movmatrix_t(pack_h2(s[mt][0], s[mt][1]));
    const uint32_t p1 = movmatrix_t(pack_h2(s[mt][2], s[mt][3]));
    uint32_t b[2][NB];
#pragma unroll
    for (int ps = 0; ps < 2; ++ps)
#pragma unroll
      for (int f = 0; f < NB; f += 2) {
        float4 x = *reinterpret_cast<const float4 *>(vs + ((2 * mt + ps) * 4 + t) * 2 * NB + 2 * f);
        if (kKind == kScaled) {
          x.x *= back;
          x.y *= back;
          x.z *= back;
          x.w *= back;
        } else if (kKind == kAny) {  // (the P of tokens not attended is 0, their scale may be anything)
          const float bad = __int_as_float(0x7fffffff);
          x.x = x.x < kNoScale ? x.x * back : bad;
          x.y = x.y < kNoScale ? x.y * back : bad;
          x.z = x.z < kNoScale ? x.z * back : bad;
          x.w = x.w < kNoScale ? x.w * back : bad;
          const int tok = 16 * mt + 8 * ps + 2 * t;
          if (tok >= valid) x.x = x.z = 0.0f;
          if (tok + 1 >= valid) x.y = x.w = 0.0f;
        }
        const uint32_t p = ps ? p1 : p0;
        b[ps][f] = as_u32(__hmul2(as_h2(p), __floats2half2_rn(x.x, x.y)));
        b[ps][f + 1] = as_u32(__hmul2(as_h2(p), __floats2half2_rn(x.z, x.w)));
      }
#pragma unroll
    for (int f = 0; f < NB; ++f)  // (a NaN is in its block's O; here it would reach every row)
      mma_f16(st.c, g == f ? kLo8 : 0u, 0u, g == f ? kHi8 : 0u, 0u,
              kKind == kAny ? no_nan(b[0][f]) : b[0][f], kKind == kAny ? no_nan(b[1][f]) : b[1][f]);
#pragma unroll
    for (int c = 0; c < NB / 2; ++c) {
      const uint4 x = *reinterpret_cast<const uint4 *>(
          rec + rec_vcode(D) + ((mt * (NB / 2) + c) * 32 + 4 * g + t) * 16);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t y = v[k] >> 8;
        const int f = 4 * c + k;
        mma_f16(st.o[f], v[k] & kLoMask, y & kLoMask, v[k] & kHiMask, y & kHiMask, b[0][f >> 1],
                b[1][f >> 1]);
      }
    }
  }
}

// x and y as two pairs of bf16 whose sum they are, q exactly and P to 15 bits. The parts of a
// number have its sign and are zero only if it is, so that infinite keys and values come
// out as products with the number itself.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
  constexpr float kBelow = 1.0f - 0.0078125f;
  const uint32_t u = __float_as_uint(x * kBelow), v = __float_as_uint(y * kBelow);
  hi = __byte_perm(u, v, 0x7632);
  lo = pack_bf2(x - __uint_as_float(u & 0xffff0000u), y - __uint_as_float(v & 0xffff0000u));
}

// 16 tokens of a bf16 window tile (half 0 or 1), `valid` of them attended. q (the 11 bits that
// the int4 part has of it) and P are split into two bf16 parts each, K and V are exact.
template <int D>
__device__ __forceinline__ void do_window(State<D> &st, const uint16_t *tile, int half,
                                          const uint32_t (&qh)[D / 32][4], int valid, int g, int t) {
  constexpr int NB = D / 32;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t *k0 = tile + (16 * half + g) * D + 8 * t, *k1 = k0 + 8 * D;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int sw = 32 * (i ^ (g & 1));  // (rows g and g + 8 have one parity)
    const uint4 a = *reinterpret_cast<const uint4 *>(k0 + sw);
    const uint4 b = *reinterpret_cast<const uint4 *>(k1 + sw);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 f = __half22float2(as_h2(qh[i][j]));
      f.x *= j & 1 ? 4.0f : 0.25f;
      f.y *= j & 1 ? 4.0f : 0.25f;
      split(f.x, f.y, hi[j], lo[j]);
    }
    mma_bf16(s, a.x, b.x, a.y, b.y, hi[0], hi[1]);
    mma_bf16(s, a.x, b.x, a.y, b.y, lo[0], lo[1]);
    mma_bf16(s, a.z, b.z, a.w, b.w, hi[2], hi[3]);
    mma_bf16(s, a.z, b.z, a.w, b.w, lo[2], lo[3]);
  }
  if (g >= valid) s[0] = s[1] = -INFINITY;
  if (g + 8 >= valid) s[2] = s[3] = -INFINITY;
  raise(st, fmaxf(s[0], s[2]), fmaxf(s[1], s[3]));
#pragma unroll
  for (int k = 0; k < 4; ++k) s[k] = fast_exp2(s[k] - st.m[k & 1] - 24.0f);
  st.l[0] = fmaf(s[0] + s[2], kHeld, st.l[0]);
  st.l[1] = fmaf(s[1] + s[3], kHeld, st.l[1]);
  uint32_t xh0, xl0, xh1, xl1;
  split(s[0], s[1], xh0, xl0);
  split(s[2], s[3], xh1, xl1);
  const uint32_t bh0 = movmatrix_t(xh0), bh1 = movmatrix_t(xh1);
  const uint32_t bl0 = movmatrix_t(xl0), bl1 = movmatrix_t(xl1);
  // tokens that are not attended: their rows may hold anything
  uint32_t mask[2];
#pragma unroll
  for (int ps = 0; ps < 2; ++ps)
    mask[ps] = (8 * ps + 2 * t < valid ? 0xffffu : 0u) |
               (8 * ps + 2 * t + 1 < valid ? 0xffff0000u : 0u);
#pragma unroll
  for (int f = 0; f < NB; ++f) {
    uint4 v[2];
#pragma unroll
    for (int ps = 0; ps < 2; ++ps) {
      v[ps] = *reinterpret_cast<const uint4 *>(
          tile + 32 * D + (((2 * half + ps) * NB + f) * 32 + 4 * g + t) * 8);
      v[ps].x &= mask[ps];
      v[ps].y &= mask[ps];
      v[ps].z &= mask[ps];
      v[ps].w &= mask[ps];
    }
    mma_bf16(st.o[2 * f], v[0].x, v[0].y, v[1].x, v[1].y, bh0, bh1);
    mma_bf16(st.o[2 * f], v[0].x, v[0].y, v[1].x, v[1].y, bl0, bl1);
    mma_bf16(st.o[2 * f + 1], v[0].z, v[0].w, v[1].z, v[1].w, bh0, bh1);
    mma_bf16(st.o[2 * f + 1], v[0].z, v[0].w, v[1].z, v[1].w, bl0, bl1);
  }
}

// First of a unit's query heads and their number; head g's features (D/4) t + ..., scaled,
// as fp16 pairs (8i + j, 8i + 4 + j), times 4 (j even) or 1/4.
template <int D>
__device__ __forceinline__ void load_q(const AttendPagesArgs &a, int row, int hc, int g, int t,
                                       uint32_t (&qh)[D / 32][4]) {
  const int kvh = hc / a.chunks, chunk = hc - kvh * a.chunks;
  const int nh = min(kApHeads, a.G - kApHeads * chunk);
  const size_t e = (static_cast<size_t>(row) * a.Hq + kvh * a.G + kApHeads * chunk + g) * D +
                   (D / 4) * t;
  float x[D / 4];
  if (a.q_dt == KVQ_F32) {
    const float *p = static_cast<const float *>(a.q) + e;
    const bool ok = g < nh && in_bounds(a.ctl, p, D);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float4 v = ok ? reinterpret_cast<const float4 *>(p)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(a.q) + e;
    const bool ok = g < nh && in_bounds(a.ctl, p, D / 2);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = ok ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = bf_lo(w[j]);
        x[8 * i + 2 * j + 1] = bf_hi(w[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = a.scale_log2 * (j & 1 ? 0.25f : 4.0f);
      qh[i][j] = pack_h2(x[8 * i + j] * f, x[8 * i + 4 + j] * f);
    }
}

template <int D>
__device__ __forceinline__ bool aborted(const Smem<D> &sm) {
  return *reinterpret_cast<const volatile int *>(&sm.abort_flag) != 0;
}

// A row that attends nothing: its units are finished; zeros if it is a row at all.
template <int D>
__device__ __noinline__ void no_items(const AttendPagesArgs &a, int row, bool zero) {
  for (int u = row * units_per_row(a); u < (row + 1) * units_per_row(a); ++u)
    if (in_bounds(a.ctl, a.first + u, 4)) a.first[u] = -1;
  const size_t b = a.out_dt == KVQ_F32 ? 4 : 2, bytes = static_cast<size_t>(a.Hq) * D * b;
  uint8_t *o = static_cast<uint8_t *>(a.out) + row * bytes;
  if (!zero || !in_bounds(a.ctl, o, bytes)) return;
  for (size_t i = 0; i < bytes; i += 16) *reinterpret_cast<uint4 *>(o + i) = make_uint4(0u, 0u, 0u, 0u);
}

// This CTA's slice of the items; row0 and at0 say where it starts.
template <int D>
__device__ __forceinline__ void find_slice(const AttendPagesArgs &a, Smem<D> &sm, long long &lo,
                                           long long &hi) {
  const int per = (a.rows + kThreads - 1) / kThreads, lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int r0 = min(a.rows, static_cast<int>(threadIdx.x) * per), r1 = min(a.rows, r0 + per);
  long long mine = 0;
  RowInfo info = {-1, -1, 0};
  for (int r = r0; r < r1; ++r) {
    info = row_info(a, r, blockIdx.x == 0);
    mine += row_items(info);
    if (info.n <= 0 && r % a.ctas == static_cast<int>(blockIdx.x)) no_items<D>(a, r, info.n == 0);
  }
  long long v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sm.sums[warp] = v;
  if (per == 1 && r0 < r1) sm.row[r0] = info;  // (all rows: no more than the threads)
  __syncthreads();
  long long base = v - mine, total = 0;
#pragma unroll
  for (int w = 0; w <= kConsumers; ++w) {
    if (w < warp) base += sm.sums[w];
    total += sm.sums[w];
  }
  const int upr = units_per_row(a);
  total *= upr;
  base *= upr;
  // (with fewer items than CTAs the first ones take one each: none in between has nothing,
  // whose partial would be missing)
  const long long n = min(total, static_cast<long long>(a.ctas));
  const long long c = min(static_cast<long long>(blockIdx.x), n);
  if (total < (1 << 22) && a.ctas < 1024) {  // (products of 32 bits: a shorter division)
    const unsigned t32 = static_cast<unsigned>(total), n32 = max(1u, static_cast<unsigned>(n));
    const unsigned c32 = static_cast<unsigned>(c);
    lo = t32 * c32 / n32;
    hi = t32 * min(c32 + 1, static_cast<unsigned>(n)) / n32;
  } else {
    lo = total * c / n;
    hi = total * min(c + 1, n) / n;
  }
  if (per == 1) {
    if (lo < hi && base <= lo && lo < base + mine * upr) {
      sm.row0 = r0;
      sm.at0 = static_cast<int>(lo - base);
    }
  } else if (lo < hi && base <= lo && lo < base + mine * upr) {
    for (int r = r0; r < r1; ++r) {
      const long long n =
          static_cast<long long>(row_items(row_info(a, r, false))) * upr;
      if (lo < base + n) {
        sm.row0 = r;
        sm.held0 = r;
        sm.at0 = static_cast<int>(lo - base);
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  if (per == 1 || lo >= hi) return;
  for (int i = threadIdx.x; i < kRowsHeld && sm.row0 + i < a.rows; i += kThreads)
    sm.row[i] = row_info(a, sm.row0 + i, false);
  __syncthreads();
}

// The page that holds group 4 j + w of the item (or -1: a window item, none, or no page).
__device__ __forceinline__ int page_of(const AttendPagesArgs &a, const Walk &at, int w) {
  const int g = 4 * at.j + w;
  if (at.j >= at.int4 || g >= int4_groups(at.r)) return -1;
  const int32_t *e = a.d.table + static_cast<size_t>(at.r.slot) * a.d.max_pages + (g >> a.d.gpp_log2());
  return in_bounds(a.ctl, e, 4) ? *e : -1;
}

// bulk_g2s of what is read once: such lines leave the L2 first (1.1 to 1.5 us of a call of 84 MB
// and more; no change where several units read the same bytes and for one short request).
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void bulk_g2s_policy(uint32_t dst, const void *src, uint32_t bytes,
                                                uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], "
      "%2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// Lane w's share of an item into a stage.
template <int D>
__device__ __forceinline__ void load_item(const AttendPagesArgs &a, Smem<D> &sm, const Walk &at,
                                          int page, int w, int st, uint64_t policy) {
  const uint32_t dst = smem_u32(sm.stage[st]), bar = smem_u32(&sm.full[st]);
  const int kvh = at.hc / a.chunks;
  int valid = 0;
  const uint8_t *src = nullptr;
  uint32_t bytes = 0;
  if (at.j < at.int4) {
    const int g = 4 * at.j + w;
    if (g < int4_groups(at.r)) {
      if (page >= 0 && page < a.d.n_pages) {
        src = a.d.record_at(page, g & ((1 << a.d.gpp_log2()) - 1), kvh);
        bytes = Cfg<D>::kRecord;
        valid = min(32, at.r.n - 32 * g);
      } else {
        flag_error(a.ctl, KVQ_DEV_INDEX);
      }
    }
  } else if (w == 0 && at.j < at.items) {
    const int g = (at.r.cut >> 5) + at.j - at.int4;
    src = static_cast<const uint8_t *>(a.d.ring) + 2 * a.d.tile_at(at.r.slot, kvh, g);
    bytes = 128 * D;
    valid = min(32, at.r.n - 32 * g);
  }
  if (bytes && !in_bounds(a.ctl, src, bytes)) bytes = valid = 0;
  sm.valid[st][w] = valid;
  mbar_arrive_expect_tx(bar, bytes);
  if (bytes) bulk_g2s_policy(dst + w * Cfg<D>::kRecord, src, bytes, bar, policy);
}

template <int D>
__device__ __forceinline__ void run_loader(const AttendPagesArgs &a, Smem<D> &sm, long long lo,
                                           int n_items, int lane) {
  constexpr int kStages = Cfg<D>::kStages;
  const int w = lane & 3;
  const uint64_t policy = read_once_policy();
  Walk at = {}, ahead;
  at.start(a, sm);
  ahead = at;  // this lane's item of the next eight
  int pages = page_of(a, ahead, w), later = -1;
  // the first item's copies are issued before the others' pages are looked up (0.5 us of a call)
  if (lane < 4 && lo != a.ctl.drop_item) load_item(a, sm, at, pages, w, 0, policy);
  for (int i = 0; i < (lane >> 2) && i + 1 < n_items; ++i) ahead.next(a, sm);
  if (lane >= 4) pages = (lane >> 2) < n_items ? page_of(a, ahead, w) : -1;
  at.next(a, sm);
  int k = 1;
  for (; k < n_items; ++k) {
    const int st = k % kStages;
    if ((k & 7) == 0) pages = later;
    if ((k & 7) == 3) {  // (not before the first stages are on their way: 1.5 us of a call)
      later = -1;
      if (k + 5 + (lane >> 2) < n_items) {
        for (int i = 0; i < 8; ++i) ahead.next(a, sm);
        later = page_of(a, ahead, w);
      }
    }
    const int page = __shfl_sync(~0u, pages, 4 * (k & 7) + w);
    bool go = true;
    if (k >= kStages) {
      go = mbar_wait(smem_u32(&sm.empty[st]), static_cast<uint32_t>((k / kStages - 1) & 1),
                     a.ctl.wait_limit_ns);
      if (!go) {
        flag_error(a.ctl, KVQ_DEV_TIMEOUT);
        *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
      }
    }
    if (__any_sync(~0u, !go || aborted(sm))) break;
    if (lane < 4 && lo + k != a.ctl.drop_item) load_item(a, sm, at, page, w, st, policy);
    at.next(a, sm);
  }
  // copies still in flight must land before the CTA ends
  for (int i = max(0, k - kStages); i < k; ++i) {
    if (lo + i == a.ctl.drop_item) continue;
    mbar_wait(smem_u32(&sm.full[i % kStages]), static_cast<uint32_t>((i / kStages) & 1),
              2000000000ull);
  }
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32));
}

// The four warps' states of a unit: finished (whole) or left as this CTA's partial (`later`:
// of a unit behind its first).
template <int D>
__device__ __forceinline__ void close_unit(const AttendPagesArgs &a, Smem<D> &sm, State<D> &st,
                                           int row, int hc, bool later, bool starts, bool ends,
                                           int warp, int g, int t) {
  const int unit = row * units_per_row(a) + hc;
  float l0 = st.l[0], l1 = st.l[1];
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(~0u, l0, o);
    l1 += __shfl_xor_sync(~0u, l1, o);
  }
  if (g == 0) {
    sm.red_m[warp][2 * t] = st.m[0];
    sm.red_m[warp][2 * t + 1] = st.m[1];
    sm.red_l[warp][2 * t] = l0;
    sm.red_l[warp][2 * t + 1] = l1;
  }
  // the 8s come off
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    const float c0 = __shfl_sync(~0u, st.c[0], 4 * b + t), c1 = __shfl_sync(~0u, st.c[1], 4 * b + t);
#pragma unroll
    for (int f = 2 * b; f < 2 * b + 2; ++f) {
      st.o[f][0] += c0;
      st.o[f][1] += c1;
      st.o[f][2] += c0;
      st.o[f][3] += c1;
    }
  }
  consumers_sync();
  if (threadIdx.x < kApHeads) {
    const int h = threadIdx.x;
    float mx = kNone, ls = 0.0f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) mx = fmaxf(mx, sm.red_m[w][h]);
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      const float c = exp2f(sm.red_m[w][h] - mx);
      sm.red_c[w][h] = c;
      ls += c * sm.red_l[w][h];
    }
    // (between two barriers: a warp that gave up waiting did so before the first)
    if (h == 0) sm.quit = aborted(sm);
    sm.red_mx[h] = mx;
    sm.red_ls[h] = ls;
  }
  const bool whole = starts && ends;
  const int slot = 2 * blockIdx.x + later;
  float *part = a.part + static_cast<size_t>(slot) * (kApHeads * Cfg<D>::kPart);
  const bool part_ok = whole || in_bounds(a.ctl, part, sizeof(float) * kApHeads * Cfg<D>::kPart);
  const int kvh = hc / a.chunks, chunk = hc - kvh * a.chunks;
  const int nh = min(kApHeads, a.G - kApHeads * chunk);
  const size_t out0 = (static_cast<size_t>(row) * a.Hq + kvh * a.G + kApHeads * chunk) * D;
  if (threadIdx.x == 0 && in_bounds(a.ctl, a.first + unit, 4) && in_bounds(a.ctl, a.last + unit, 4)) {
    if (starts) a.first[unit] = whole ? -1 : slot;
    if (ends) a.last[unit] = blockIdx.x;
  }
  for (int half = 0; half < 2; ++half) {
    if (4 * half >= nh) break;
    if ((t >> 1) == half) {
      const int h = 2 * t - 4 * half;
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        sm.red_o[warp][h][16 * f + g] = st.o[f][0];
        sm.red_o[warp][h + 1][16 * f + g] = st.o[f][1];
        sm.red_o[warp][h][16 * f + 8 + g] = st.o[f][2];
        sm.red_o[warp][h + 1][16 * f + 8 + g] = st.o[f][3];
      }
    }
    consumers_sync();
    for (int i = threadIdx.x; i < 4 * D; i += kConsumers * 32) {
      const int hh = i / D, d = i - hh * D, h = 4 * half + hh;
      if (h >= nh || !part_ok) continue;
      float acc = 0.0f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) acc += sm.red_c[w][h] * sm.red_o[w][hh][d];
      if (whole) {
        const float ls = sm.red_ls[h], y = ls == 0.0f ? 0.0f : acc / ls * kHeld;
        const size_t o = out0 + static_cast<size_t>(h) * D + d, b = a.out_dt == KVQ_F32 ? 4 : 2;
        if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.out) + o * b, b)) continue;
        if (a.out_dt == KVQ_F32)
          static_cast<float *>(a.out)[o] = y;
        else
          static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(y);
      } else {
        part[h * Cfg<D>::kPart + d] = acc;
        if (d == 0) {
          part[h * Cfg<D>::kPart + D] = sm.red_mx[h];
          part[h * Cfg<D>::kPart + D + 1] = sm.red_ls[h];
        }
      }
    }
    consumers_sync();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attend_pages_kernel(const __grid_constant__ AttendPagesArgs a) {
  constexpr int kStages = Cfg<D>::kStages;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  allow_next_grid();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 4);
      mbar_init(smem_u32(&sm.empty[s]), kConsumers);
    }
    sm.abort_flag = 0;
    sm.row0 = sm.held0 = sm.at0 = 0;
    fence_mbar_init();
  }
  wait_prior_grid();
  long long lo, hi;
  find_slice(a, sm, lo, hi);
  const int n_items = static_cast<int>(hi - lo);
  if (n_items == 0) return;
  if (warp == kConsumers) {
    run_loader(a, sm, lo, n_items, lane);
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  State<D> st;
  uint32_t qh[D / 32][4];
  Walk at = {};
  at.start(a, sm);
  int k = 0;
  while (k < n_items && at.row < a.rows) {  // (the rows end first only if lengths changed)
    reset(st);
    load_q<D>(a, at.row, at.hc, g, t, qh);
    const bool starts = at.j == 0;
    const int end = min(n_items, k + at.items - at.j);
    const bool ends = end - k == at.items - at.j;
    for (; k < end; ++k, ++at.j) {
      const int s = k % kStages;
      const uint32_t bar = smem_u32(&sm.full[s]), par = static_cast<uint32_t>((k / kStages) & 1);
      if (!__all_sync(~0u, mbar_try_wait(bar, par))) {
        const bool stop = aborted(sm) || !mbar_wait(bar, par, a.ctl.wait_limit_ns);
        if (__any_sync(~0u, stop)) {
          if (lane == 0 && !aborted(sm)) flag_error(a.ctl, KVQ_DEV_TIMEOUT);
          *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
          break;
        }
      }
      const uint8_t *stage = sm.stage[s];
      if (at.j < at.int4) {
        const int valid = sm.valid[s][warp];
        const uint8_t *rec = stage + warp * Cfg<D>::kRecord;
        const int ev = scale_exponent<D, false>(rec, 32, lane);
        if (valid >= 32 && far_of(ev) == 0)
          do_group<D, kUsual>(st, rec, qh, 32, ev, g, t);
        else if (valid >= 32 && ev <= kTopExp)
          do_group<D, kScaled>(st, rec, qh, 32, held_exponent(ev), g, t);
        else if (valid > 0)
          do_group<D, kAny>(st, rec, qh, valid, scale_exponent<D, true>(rec, valid, lane), g, t);
      } else if ((warp >> 1) == (at.j & 1)) {
        const int valid = sm.valid[s][0] - 16 * (warp & 1);
        if (valid > 0)
          do_window<D>(st, reinterpret_cast<const uint16_t *>(stage), warp & 1, qh, valid, g, t);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[s]));
    }
    // (a unit that starts in the slice, but not with it, is a later one)
    close_unit(a, sm, st, at.row, at.hc, starts && k > at.j, starts, ends, warp, g, t);
    // the four warps leave together, as each unit's end has barriers for all of them
    if (sm.quit) break;
    if (ends) at.next_unit(a, sm);
  }
}

// Joins the partials of a unit that several CTAs had. kWarps warps per
// head take every kWarps-th partial; with one warp a head a CTA has all of a unit's heads.
template <int D, int kWarps>
__global__ void __launch_bounds__(256) attend_pages_join_kernel(const AttendPagesArgs a) {
  constexpr int kPart = Cfg<D>::kPart, V = D / 32;
  __shared__ float sm_m[8], sm_l[8];
  __shared__ float sm_o[8][D];
  wait_prior_grid();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x, upr = units_per_row(a), row = unit / upr, hc = unit - row * upr;
  const int kvh = hc / a.chunks, chunk = hc - kvh * a.chunks;
  const int h = kWarps == 1 ? warp : static_cast<int>(blockIdx.y), w0 = kWarps == 1 ? 0 : warp;
  if (h >= min(kApHeads, a.G - kApHeads * chunk)) return;
  if (!in_bounds(a.ctl, a.first + unit, 4) || !in_bounds(a.ctl, a.last + unit, 4)) return;
  const int slot0 = a.first[unit], c0 = slot0 >> 1, c1 = a.last[unit];
  if (slot0 < 0) return;                // finished by its CTA, or a row that attends nothing
  if (c1 < c0 || c1 >= a.ctas) return;  // (not written: a wait ran out)
  float m = kNone, l = 0.0f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  {
    const int n = c1 - c0 + 1;
    // its partials: slot0, and the first one of every CTA behind
    constexpr size_t kSlot = kApHeads * kPart;
    const float *parts = a.part + h * kPart;
    if (!in_bounds(a.ctl, parts + slot0 * kSlot, sizeof(float) * kPart) ||
        !in_bounds(a.ctl, parts + 2 * c0 * kSlot, sizeof(float) * (2 * (n - 1) * kSlot + kPart)))
      return;
    constexpr int kBatch = 8;
    for (int i0 = w0; i0 < n; i0 += kWarps * kBatch) {
      float pm[kBatch], pl[kBatch], po[kBatch][V];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = i0 + kWarps * i;
        const float *p = parts + (c == 0 ? slot0 : 2 * (c0 + min(c, n - 1))) * kSlot;
        const float2 ml = *reinterpret_cast<const float2 *>(p + D);
        pm[i] = c < n ? ml.x : -INFINITY;
        pl[i] = c < n ? ml.y : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) po[i][v] = c < n ? p[32 * v + lane] : 0.0f;
      }
      float nm = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) nm = fmaxf(nm, pm[i]);
      const float c = exp2f(m - nm);
      l *= c;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= c;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float x = exp2f(pm[i] - nm);
        l = fmaf(x, pl[i], l);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(x, po[i][v], acc[v]);
      }
      m = nm;
    }
    if (kWarps > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) sm_o[warp][32 * v + lane] = acc[v];
      if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
      }
      __syncthreads();
      if (warp) return;
      float nm = kNone;
#pragma unroll
      for (int w = 0; w < 8; ++w) nm = fmaxf(nm, sm_m[w]);
      l = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float x = exp2f(sm_m[w] - nm);
        l = fmaf(x, sm_l[w], l);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(x, sm_o[w][32 * v + lane], acc[v]);
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : kHeld / l;
  const size_t o = (static_cast<size_t>(row) * a.Hq + kvh * a.G + kApHeads * chunk + h) * D;
  const size_t b = a.out_dt == KVQ_F32 ? 4 : 2;
  if (!in_bounds(a.ctl, static_cast<const uint8_t *>(a.out) + o * b, D * b)) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (a.out_dt == KVQ_F32)
      static_cast<float *>(a.out)[o + 32 * v + lane] = acc[v] * inv;
    else
      static_cast<__nv_bfloat16 *>(a.out)[o + 32 * v + lane] = __float2bfloat16_rn(acc[v] * inv);
  }
}

int chunks_of(const PagedDims &d, int Hq) { return (Hq / d.Hkv + kApHeads - 1) / kApHeads; }

// Items of the longest request that the table can hold.
long most_items(const PagedDims &d) {
  return ((static_cast<long>(d.max_pages) << d.page_log2) + 127) / 128 + d.tiles;
}

// CTAs of the grid: no more than there can be items.
int grid_of(const PagedDims &d, int Hq, int rows, int num_sms) {
  const long items = static_cast<long>(rows) * d.Hkv * chunks_of(d, Hq) * most_items(d);
  return static_cast<int>(std::min<long>(items, static_cast<long>(kCtasPerSm) * num_sms));
}

template <int D>
int launch_typed(AttendPagesArgs &a, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>);
  opt_in_smem(attend_pages_kernel<D>, smem);
  launch_dependent(attend_pages_kernel<D>, dim3(a.ctas), dim3(kThreads), smem, s, a);
  const unsigned units = static_cast<unsigned>(a.rows) * a.d.Hkv * a.chunks;
  // few units have many partials each: eight warps a head; many units a few: one warp
  if (static_cast<long>(units) * 16 <= a.ctas)
    launch_dependent(attend_pages_join_kernel<D, 8>, dim3(units, std::min(kApHeads, a.G)), dim3(256),
                     0, s, a);
  else
    launch_dependent(attend_pages_join_kernel<D, 1>, dim3(units), dim3(256), 0, s, a);
  return 2;
}

}  // namespace

bool attend_pages_supported(const PagedDims &d, int Hq, int rows) {
  // (units, and the items of a row and of a CTA, are counted in 32 bits)
  const long upr = static_cast<long>(d.Hkv) * chunks_of(d, Hq);
  return (d.D == 64 || d.D == 128) && d.win_dt == KVQ_BF16 && rows * upr < (1L << 30) &&
         upr * most_items(d) < (1L << 30) && rows * upr * most_items(d) < (1L << 38);
}

size_t attend_pages_workspace(const PagedDims &d, int Hq, int rows, int num_sms) {
  const size_t units = static_cast<size_t>(rows) * d.Hkv * chunks_of(d, Hq);
  return (8 * units + 15) / 16 * 16 +
         sizeof(float) * 2 * grid_of(d, Hq, rows, num_sms) * kApHeads * (d.D + 4);
}

int launch_attend_pages(const PagedDims &d, const void *q, int q_dt, int Hq, int rows,
                        const int32_t *slot, const int32_t *pos, float scale_log2, void *out,
                        int out_dt, void *ws, const KernelCtl &ctl, int num_sms, cudaStream_t s) {
  AttendPagesArgs a;
  a.d = d;
  a.q = q;
  a.out = out;
  a.slot = slot;
  a.pos = pos;
  a.scale_log2 = scale_log2;
  a.q_dt = q_dt;
  a.out_dt = out_dt;
  a.rows = rows;
  a.Hq = Hq;
  a.G = Hq / d.Hkv;
  a.chunks = chunks_of(d, Hq);
  a.ctas = grid_of(d, Hq, rows, num_sms);
  a.ctl = ctl;
  const size_t units = static_cast<size_t>(rows) * d.Hkv * a.chunks;
  a.first = static_cast<int32_t *>(ws);
  a.last = a.first + units;
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + (8 * units + 15) / 16 * 16);
  return d.D == 128 ? launch_typed<128>(a, s) : launch_typed<64>(a, s);
}

}  // namespace kvq
