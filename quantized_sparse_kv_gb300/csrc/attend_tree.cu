// Attention of drafted tokens over a packed cache and their own ancestors
// (kv_attend_tree) on the fifth-generation tensor cores: D = 128, bf16 q.
//
// Mathematics. The T drafted tokens of a sequence times the G query heads of a KV
// head are T * G query rows that attend the same keys: the cache's tokens, all of
// them, and the drafted ones, under a mask. O = softmax(c Q K^T) V is computed
// key tile by key tile with a running reference and sum per row; partial results
// of a row over different key ranges are merged by the log-sum-exp rule.
//
// Work split. A unit is one (sequence, KV head); its rows are cut into row blocks
// of 256 (two MMA tiles of 128), its keys into tiles of 128: the int4 part, then
// the bf16 window and the drafted tokens laid end to end. All (unit, row block,
// tile) items are laid end to end too and one CTA per SM takes an equal contiguous
// slice, so a call with few rows still uses every SM. A CTA writes a partial
// per row block it touches (or the output itself when its slice covers the whole
// row block), tree_combine_kernel merges them.
//
// Inside a CTA (20 warps):
//   warps 0-3, 4-7   softmax groups A and B, a thread per query row;
//   warps 8-15       dequantization, four of K and four of V: packed tile ->
//                    registers (a tile ahead) -> fp16 tile in shared
//                    memory, 128B-swizzled, two stages each;
//   warps 16-19      the MMAs, a warp per group and score buffer (16 also
//                    allocates TMEM).
// Registers move from the other roles to the softmax groups (setmaxnreg).
// With more than 128 rows in the row block group A takes rows 0-127 and group B
// rows 128-255 of every tile (each dequantized tile feeds both); with fewer, both
// work on the same rows, A on the first and B on the second half of every tile,
// and their sums and outputs are merged at the end of the slice. A group's step
// is a half tile (64 keys): S = Q K^T (MMA, both operands in shared memory),
// softmax in registers, P written as fp16 over S in TMEM, O += P V (MMA, A operand
// from TMEM). Its steps alternate between two score buffers, each with an MMA warp
// of its own: S of the step after next is issued once the PV that reads the
// buffer has completed, so the softmax warps find the next scores ready while
// the hand-overs of the last step run.
//
// Precision: fp16 operands (11 bits; K and V are code * scale), fp32 sums and
// softmax state. P is rounded to fp16 against a reference that starts 2^9 below the
// row's maximum and is raised when 64 keys' P sum to more than 61,440 (kRefBias).
//
// Feature order: a nibble word gives features (0,4)(1,5)(2,6)(3,7) of eight in
// pairs without shuffling, so Q, K and V tiles hold every eight features in the
// order 0 4 1 5 2 6 3 7; the output is written back in natural order.
//
// What bounds it. Many rows: the tensor pipe and the hand-overs around it. A tile of
// two groups takes 1.8 us, of which the pipe works 2,560 cycles (a 64-key S step is
// 8 x 48, its operands' shared-memory reads; a PV step 4 x 64). 16 sequences x 64
// tokens x 16 heads over 32,768 keys (275 GFLOP): 212 us on the same inputs back to
// back, 1,300 TFLOP/s, 223 us on changing ones (1,230); without the exponentials it
// would be 3 % faster, without the softmax 14 %, without the tile stores 9 %. Few rows:
// packed bytes and fixed times; 16 sequences x 8 tokens over 8,200 keys (45 MB): 29.9
// us back to back, 34.4 on changing inputs, of which 4.9 us until the first queries are
// in place, 1.1 us a tile (of 128 rows, half of them used), 2 us the output and about
// 5 us the merge.
// Measured and not kept (16 x 64 tokens, the kernel at that time in brackets): S of
// a whole tile in one step (N = 128) 268 us (229); Q as the A operand from TMEM, S
// then 8 x 32 cycles but with one score buffer a group, 264 (213); softmax in
// steps of 32 keys 281 (229); the exponentials' loop not unrolled 238 (229).
#include <math_constants.h>

#include <algorithm>

#include "int4_dequant.cuh"
#include "kvq_internal.h"
#include "tc_common.cuh"

namespace kvq {
namespace {

constexpr int kD = 128;
constexpr int kBM = 128;           // rows of an MMA tile
constexpr int kBN = 128;           // keys of a tile
constexpr int kRowBlock = 2 * kBM;
constexpr int kSoftWarps = 8, kDqWarps = 8;
constexpr int kThreads = (kSoftWarps + kDqWarps + 4) * 32;  // whole warpgroups (setmaxnreg)
// Registers a thread of each role: the launch gives 96 to all 640 (65,536 / 640,
// rounded down to a multiple of 8); the softmax groups take what the others
// leave: 2 * 128 + 2 * 80 + 64 <= 5 * 96.
constexpr int kLaunchRegs = 96, kSoftRegs = 128, kDqRegs = 80, kMmaRegs = 64;
static_assert(2 * kSoftRegs + 2 * kDqRegs + kMmaRegs <= 5 * kLaunchRegs, "register split");
constexpr uint32_t kHalf = 128u * 128u;      // 16 KB: 128 rows x 64 fp16 features
constexpr uint32_t kTileBytes = 2u * kHalf;
constexpr int kStages = 2;                   // K and V tiles in shared memory, each
constexpr int kMaskWords = KVQ_TREE_MAX / 32;
// Tiles' worth of time that starting a row block takes (queries, masks, first
// scores) and that ending one does (the tail's slower tiles, the output), with two
// groups of rows and with shared ones (a tile takes 1.8 us, or 1.1 us).
constexpr int kLeadTwo = 5, kLeadShared = 4, kTrail = 2;
// P is fp16, and l its fp32 sum before that rounding: the reference is set 2^kRefBias
// below the row's maximum, so that keys 15.9 nats below it keep 11 bits of P and keys 23
// nats below it still count (from a reference at the maximum: 9.7 and 17), and raised when
// 64 P sum to more than kSumBound, which every P of the 64 then is below (fp16: 65,504).
// 64 equal scores sum to 2^15. (Raises cost a pass over 64 scores and one over O. The
// reference at the maximum and a bound of 2^12 in brackets, 16 x 64 tokens over 32,768
// keys: scores of standard deviation 1 223 us (222), 2 229 (222), 4 248 (232).)
constexpr float kRefBias = 9.0f, kSumBound = 61440.0f;
// A partial: O of 256 rows as [32 pieces][256 rows] float4 (a warp's store is
// consecutive rows of one piece), then (m, l) of the rows.
constexpr long kPartFloats = kRowBlock * (kD + 2);

struct __align__(1024) TreeSmem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  int par[KVQ_TREE_MAX];                     // parents of the sequence
  uint32_t seen[KVQ_TREE_MAX][kMaskWords];   // ancestor bits of every drafted token
  uint32_t live[kMaskWords];                 // drafted tokens that exist
  uint32_t odd_v[kMaskWords];                // drafted tokens with a V element beyond fp16
  float mm[2][kBM], ml[2][kBM];              // row states of the two groups (alternate tiles)
  uint64_t k_full[kStages][2], k_empty[kStages][2], v_full[kStages][2], v_empty[kStages][2];  // [half]
  uint64_t q_full, s_full[2][2], p_full[2][2], o_done[2][2], mma_done;  // [group][buffer]
  uint32_t tmem_base;
  int abort_flag;
};

struct TreeArgs {
  const uint8_t *k_codes;
  const float *k_scales;
  const uint8_t *v_codes;
  const float *v_scales;
  const uint16_t *k_window, *v_window;  // bf16
  const uint16_t *k_tree, *v_tree;      // bf16 [unit][T][128]
  const uint16_t *q;                    // bf16 [batch][Hq][T][128]
  const int32_t *parents;
  int Hkv, G, T, R, cut, Gk, Gs, Vs, Ws;
  int rows, row_blocks;                 // T * G, and per unit
  int int4_tiles, tiles;                // key tiles per unit
  // Items are laid out as if every row block had `lead` more tiles before its
  // first and some behind its last (the time its queries, masks, tail and
  // output take), so that slices that begin or end a row block get fewer tiles.
  int lead, span;                       // span = lead + tiles + those behind
  long items;                           // units * row_blocks * span
  int ctas, slots;                      // slots: partials reserved per row block
  float scale_log2;
  void *out;
  int out_dtype;
  float *partials;                      // [unit * row_blocks][slots][kPartFloats]
  KernelCtl ctl;
};

// ------------------------------------------------------------------ PTX wrappers
// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// O += P V with P (A operand, fp16 pairs, one lane per row) in TMEM.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one lane of a fully active warp, always the same one. MMAs are issued
// under it from code the whole warp runs, with operands the compiler can see to
// be warp-uniform: a batch of eight (N = 128) then issues in the 512 cycles
// it executes in, against 1,026 under `lane == 0`.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A bounded wait by testing the barrier in a loop: the MMA warps do nothing else,
// and waking from a suspended wait takes longer.
__device__ __forceinline__ bool spin_wait(int *abort_flag, uint32_t bar, uint32_t parity,
                                          const KernelCtl &ctl) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_test(bar, parity)); ++i) {
    if ((i & 1023u) != 0) continue;
    const uint64_t now = global_ns();
    if (i == 1024u) t0 = now;
    if (__any_sync(0xffffffffu, cta_aborted(abort_flag) || now - t0 > ctl.wait_limit_ns)) {
      flag_error(ctl, KVQ_DEV_TIMEOUT);
      *reinterpret_cast<volatile int *>(abort_flag) = 1;
      return false;
    }
  }
  return true;
}

// The value of lane 0, which the compiler then knows to be warp-uniform.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// A shared-memory descriptor (smem_desc) from its low word, which holds the
// address / 16 and the leading offset, and its constant high word.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1,024, version 1, 128B swizzle
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// 32 words to 32 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}

// Instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator, M = 128,
// N = n, A K-major, B K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t b_mn_major, uint32_t n) {
  return (1u << 4) | (b_mn_major << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// Whether a bf16 (its bits) is beyond fp16: 2^16 and more, infinite, NaN. (bf16's next
// lower value, 65,280, is an fp16 number.)
__device__ __forceinline__ bool odd_bf16(uint32_t bits) { return (bits & 0x7fffu) >= 0x4780u; }

// Eight bf16 (four words, natural order) as fp16 in the tiles' feature order. Elements
// beyond fp16 become infinite, or (kNan: queries and keys) NaN, whose scores are NaN
// whatever they meet: h + 0 h is h, and NaN where h is infinite.
template <bool kNan>
__device__ __forceinline__ uint4 bf8_to_h8(const uint4 &w) {
  auto cvt = [](float lo, float hi) {
    const __half2 h = as_h2(pack_h2(lo, hi));
    return as_u32(kNan ? __hfma2(h, __half2half2(__ushort_as_half(0)), h) : h);
  };
  return make_uint4(cvt(bf_lo(w.x), bf_lo(w.z)), cvt(bf_hi(w.x), bf_hi(w.z)),
                    cvt(bf_lo(w.y), bf_lo(w.w)), cvt(bf_hi(w.y), bf_hi(w.w)));
}

// Place of 16-byte chunk c (0..15, eight features each) of row r in a tile.
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
  return (c >> 3) * kHalf + swz(r, c & 7u);
}

// Slice of CTA c: items [items * c / ctas, items * (c + 1) / ctas), of which the
// ones before a row block's first tile and behind its last are no work.
__device__ __forceinline__ uint32_t slice_lo(const TreeArgs &a, int c) {
  return static_cast<uint32_t>(a.items * c / a.ctas);
}
// A CTA's work: segments of consecutive tiles of one row block each.
struct Segment {
  uint32_t rb;       // unit * row_blocks + row block
  int t_lo, n;       // first tile, tiles (> 0)
};
// The segment that begins at or after item x (moved behind it); false when
// the slice ending at hi holds no further tile.
__device__ __forceinline__ bool next_segment(const TreeArgs &a, uint32_t &x, uint32_t hi,
                                             Segment &s) {
  while (x < hi) {
    s.rb = x / static_cast<uint32_t>(a.span);
    const uint32_t start = s.rb * a.span, end = min(start + a.span, hi);
    const int lo = max(0, static_cast<int>(x - start) - a.lead);
    s.t_lo = lo;
    s.n = min(static_cast<int>(end - start) - a.lead, a.tiles) - lo;
    x = end;
    if (s.n > 0) return true;
  }
  return false;
}
// CTA whose slice holds item x.
__device__ __forceinline__ int cta_of(const TreeArgs &a, long x) {
  return static_cast<int>(((x + 1) * a.ctas - 1) / a.items);
}

// ------------------------------------------------------------------ dequantization
// Four warps make the K tiles and four the V tiles. Warp grp of either takes
// the tile's rows 32 grp .. 32 grp + 31 (one K group), lane (r, cb) the 32
// features of block cb of rows r, r + 8, r + 16, r + 24 (16 bytes of codes
// each): a quarter-warp stores eight consecutive rows of one feature block, so
// its swizzled 16-byte stores meet all banks.
struct Raw {
  uint4 c[4];
  float4 s;  // K: scales 4r .. 4r + 3 of the block (eight lanes share theirs); V: one per row
};

// Where a warp's next tile lies (its lane's first 16 bytes and scale).
struct RawPtr {
  const uint8_t *c;
  const float *s;
};

template <bool kV>
__device__ __forceinline__ RawPtr raw_ptr(const TreeArgs &a, long u, int tile, int grp, int r,
                                          int cb) {
  RawPtr p;
  if (kV) {
    const long row = u * a.Vs + kBN * tile + 32 * grp + r;
    p.c = a.v_codes + row * 64 + 16 * cb;
    p.s = a.v_scales + row * 4 + cb;
  } else {
    const long gi = u * a.Gs + 4 * tile + grp;
    p.c = a.k_codes + (gi * 32 + r) * 64 + 16 * cb;
    p.s = a.k_scales + gi * 128 + 32 * cb + 4 * r;
  }
  return p;
}

template <bool kV>
__device__ __forceinline__ void load_raw(const TreeArgs &a, const RawPtr &p, int tile, int grp,
                                         int r, Raw &x) {
  const uint4 zero = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);  // code 0
  if (kV) {
    float *s = reinterpret_cast<float *>(&x.s);
    const int left = a.cut - (kBN * tile + 32 * grp + r);  // rows from this lane's first on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = 8 * i < left && in_bounds(a.ctl, p.c + 512 * i, 16) &&
                      in_bounds(a.ctl, p.s + 32 * i, 4);
      x.c[i] = ok ? *reinterpret_cast<const uint4 *>(p.c + 512 * i) : zero;
      s[i] = ok ? p.s[32 * i] : 0.0f;
    }
  } else {
    const bool have = 4 * tile + grp < a.Gk;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x.c[i] = have && in_bounds(a.ctl, p.c + 512 * i, 16)
                   ? *reinterpret_cast<const uint4 *>(p.c + 512 * i)
                   : zero;
    x.s = have && in_bounds(a.ctl, p.s, 16) ? *reinterpret_cast<const float4 *>(p.s)
                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
}

// Eight codes of a word times their scales (pairs in the tiles' feature order).
__device__ __forceinline__ uint4 dq8(uint32_t w, __half2 s04, __half2 s15, __half2 s26,
                                     __half2 s37) {
  const uint32_t h = w >> 8;
  return make_uint4(as_u32(__hmul2(as_h2(dq_lo(w)), s04)), as_u32(__hmul2(as_h2(dq_hi(w)), s15)),
                    as_u32(__hmul2(as_h2(dq_lo(h)), s26)), as_u32(__hmul2(as_h2(dq_hi(h)), s37)));
}

// The lane's part of a tile to shared memory; `row` is the lane's first row's
// place and sw its swizzle (the rows differ by multiples of eight).
template <bool kV>
__device__ __forceinline__ void store_raw(const Raw &x, int r, int cb, uint8_t *row) {
  const uint32_t h01 = pack_h2(x.s.x, x.s.y), h23 = pack_h2(x.s.z, x.s.w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint8_t *dst = row + (cb >> 1) * kHalf + ((((4 * cb + j) & 7) ^ r) << 4);
    __half2 s0, s1, s2, s3;
    if (!kV) {
      // word j's scales: 0-3 from lane 2j of the eight, 4-7 from lane 2j + 1
      const int from = 8 * cb + 2 * j;
      const uint32_t p01 = __shfl_sync(0xffffffffu, h01, from);
      const uint32_t p23 = __shfl_sync(0xffffffffu, h23, from);
      const uint32_t p45 = __shfl_sync(0xffffffffu, h01, from + 1);
      const uint32_t p67 = __shfl_sync(0xffffffffu, h23, from + 1);
      s0 = as_h2(prmt(p01, p45, 0x5410u)), s1 = as_h2(prmt(p01, p45, 0x7632u));
      s2 = as_h2(prmt(p23, p67, 0x5410u)), s3 = as_h2(prmt(p23, p67, 0x7632u));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = j == 0 ? x.c[i].x : j == 1 ? x.c[i].y : j == 2 ? x.c[i].z : x.c[i].w;
      if (kV) s0 = s1 = s2 = s3 = as_h2(prmt(i < 2 ? h01 : h23, 0u, i & 1 ? 0x3232u : 0x1010u));
      *reinterpret_cast<uint4 *>(dst + 1024 * i) = dq8(w, s0, s1, s2, s3);
    }
  }
}

// Rows of the tail (window, then drafted tokens) from key k0 on, zeros past
// its end; V elements of drafted tokens beyond fp16 become zero (they are added, as
// infinities or NaN, for the rows that see them when the output is written).
template <bool kV>
__device__ __noinline__ void copy_tail(const TreeArgs &a, long u, int k0, int grp, int r, int cb,
                                          uint8_t *tile) {
  const uint16_t *win = kV ? a.v_window : a.k_window, *tree = kV ? a.v_tree : a.k_tree;
#pragma unroll 2
  for (int i = 0; i < 4; ++i) {
    const int row = 32 * grp + r + 8 * i, key = k0 + row;
    const uint16_t *p = key < a.R ? win + (u * a.Ws + key) * kD
                                  : tree + (u * a.T + (key - a.R)) * kD;
    const bool ok = key < a.R + a.T && in_bounds(a.ctl, p, 2 * kD);
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = ok ? reinterpret_cast<const uint4 *>(p + 32 * cb)[j] : make_uint4(0u, 0u, 0u, 0u);
    if (kV && key >= a.R) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t *e = reinterpret_cast<uint32_t *>(&w[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (odd_bf16(e[k])) e[k] &= 0xffff0000u;
          if (odd_bf16(e[k] >> 16)) e[k] &= 0x0000ffffu;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4 *>(tile + chunk_at(row, 4 * cb + j)) = bf8_to_h8<!kV>(w[j]);
  }
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------------ the kernel
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The same barrier, returning in every thread whether any thread passed true:
// the one place where the softmax threads agree to stop.
__device__ __forceinline__ bool soft_sync_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}

// A bounded wait of a whole warp: true only when every lane's wait ended in time.
__device__ __forceinline__ bool warp_wait(int *abort_flag, uint32_t bar, uint32_t parity,
                                          const KernelCtl &ctl) {
  return __all_sync(0xffffffffu, wait_or_abort(abort_flag, bar, parity, ctl));
}

// Features d0 .. d0 + 31 of a row just written to dst whose seen drafted tokens
// hold V elements beyond fp16 there (zeroed in the tiles): the sum of those, as
// infinities or NaN, is the result. k_lo, k_hi: the tail keys the row's sum covers; step: elements from
// one piece of four features to the next.
__device__ __noinline__ void put_odd_values(const TreeArgs &a, const TreeSmem &sm, long u, int tok,
                                            int k_lo, int k_hi, int d0, void *dst, int step, bool bf16) {
  for (int e = d0; e < d0 + 32; ++e) {
    float s = 0.0f;
    for (int j = max(0, k_lo - a.R); j < min(a.T, k_hi - a.R); ++j) {
      if (!((sm.odd_v[j >> 5] & sm.seen[tok][j >> 5]) >> (j & 31) & 1u)) continue;
      const uint16_t *p = a.v_tree + (u * a.T + j) * kD + e;
      const float x = in_bounds(a.ctl, p, 2) ? bf16_to_f32(*p) : 0.0f;
      if (!(fabsf(x) < 65536.0f)) s += x * CUDART_INF_F;
    }
    if (s == 0.0f) continue;
    const long at = static_cast<long>(e >> 2) * step + (e & 3);
    if (bf16)
      static_cast<__nv_bfloat16 *>(dst)[at] = __float2bfloat16_rn(s);
    else
      static_cast<float *>(dst)[at] = s;
  }
}

// One dequantization warp: its rows of every K (or V) tile of the CTA's items, each
// with codes and scales loaded a tile earlier. (Loading two tiles ahead needs the
// loop twice; the code of all roles then no longer fits the instruction caches
// and the call takes half as long again. Bulk copies to a raw stage per warp,
// the next one issued when a fence has shown that every lane has read the stage, take
// 219 us where this takes 208: 16 sequences of 64 drafted tokens, 32K keys.)
template <bool kV>
__device__ __forceinline__ void dequant_warp(const TreeArgs &a, TreeSmem &sm, uint32_t lo,
                                             uint32_t hi, int grp, int lane) {
  const int r = lane & 7, cb = lane >> 3;
  auto unit_of = [&](uint32_t rb) {
    return static_cast<long>(rb / static_cast<uint32_t>(a.row_blocks));
  };
  // the tile at hand and the one loaded ahead: segment, tile, tiles left
  Segment cur, ahead;
  uint32_t cur_x = lo, ahead_x = lo;
  bool more = next_segment(a, ahead_x, hi, ahead);
  if (!more) return;
  next_segment(a, cur_x, hi, cur);
  RawPtr ptr = raw_ptr<kV>(a, unit_of(ahead.rb), ahead.t_lo, grp, r, cb);
  Raw x;
  auto load = [&]() {
    if (!more) return;
    if (ahead.t_lo < a.int4_tiles) load_raw<kV>(a, ptr, ahead.t_lo, grp, r, x);
    ptr.c += 8192;
    ptr.s += 512;
    ++ahead.t_lo;
    if (--ahead.n == 0) {
      more = next_segment(a, ahead_x, hi, ahead);
      if (more) ptr = raw_ptr<kV>(a, unit_of(ahead.rb), ahead.t_lo, grp, r, cb);
    }
  };
  load();
#pragma unroll 1
  for (int j = 0;; ++j) {
    const int st = j % kStages;
    uint64_t *empty = kV ? &sm.v_empty[st][grp >> 1] : &sm.k_empty[st][grp >> 1];
    uint64_t *full = kV ? &sm.v_full[st][grp >> 1] : &sm.k_full[st][grp >> 1];
    uint8_t *tile = kV ? sm.v[st] : sm.k[st];
    if (j >= kStages && !warp_wait(&sm.abort_flag, smem_u32(empty),
                                   static_cast<uint32_t>((j / kStages - 1) & 1), a.ctl))
      break;
    if (cur.t_lo < a.int4_tiles)
      store_raw<kV>(x, r, cb, tile + (32 * grp + r) * 128);
    else
      copy_tail<kV>(a, unit_of(cur.rb), kBN * (cur.t_lo - a.int4_tiles), grp, r, cb, tile);
    fence_async_smem();
    __syncwarp();
    // (test hook: the keys of a dropped tile never arrive)
    if (lane == 0 && (kV || static_cast<int>(cur.rb) * a.tiles + cur.t_lo != a.ctl.drop_item))
      mbar_arrive(smem_u32(full));
    load();
    ++cur.t_lo;
    if (--cur.n == 0 && !next_segment(a, cur_x, hi, cur)) break;
  }
}

__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  TreeSmem &sm = *reinterpret_cast<TreeSmem *>(smem_raw + (((base + 1023u) & ~1023u) - base));
  int *const abort_flag = &sm.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t lo = slice_lo(a, blockIdx.x), hi = slice_lo(a, blockIdx.x + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kStages; ++i) {
      mbar_init(smem_u32(&sm.k_full[i >> 1][i & 1]), kDqWarps / 4);
      mbar_init(smem_u32(&sm.v_full[i >> 1][i & 1]), kDqWarps / 4);
      mbar_init(smem_u32(&sm.k_empty[i >> 1][i & 1]), 2);
      mbar_init(smem_u32(&sm.v_empty[i >> 1][i & 1]), 2);
    }
    mbar_init(smem_u32(&sm.q_full), 2 * kBM + 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sm.s_full[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&sm.p_full[i >> 1][i & 1]), kBM / 32);
      mbar_init(smem_u32(&sm.o_done[i >> 1][i & 1]), 1);
    }
    mbar_init(smem_u32(&sm.mma_done), 4);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSoftWarps + kDqWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&sm.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_prior_grid();
  allow_next_grid();
  const uint32_t tmem = sm.tmem_base;
  auto t_s = [&](int g) { return tmem + 256u * g; };
  auto t_o = [&](int g) { return tmem + 256u * g + 128u; };

  if (warp >= kSoftWarps && warp < kSoftWarps + kDqWarps) {
    // ------------------------------------------------ dequantization
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDqRegs));
    // K on the schedulers (warp % 4) 0 and 1, V on 2 and 3: each holds one's code
    const int grp = (warp & 1) + ((warp & 4) >> 1);
    if (warp & 2)
      dequant_warp<true>(a, sm, lo, hi, grp, lane);
    else
      dequant_warp<false>(a, sm, lo, hi, grp, lane);
  } else if (warp >= kSoftWarps + kDqWarps) {
    // ------------------------------------------------ MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    // Warp 16 + 2g + b: buffer b of group g, that is the group's steps b, b + 2, ...
    constexpr uint32_t id_qk = idesc_f16(0, 64), id_pv = idesc_f16(1, 128);
    const uint32_t g = uniform((warp - (kSoftWarps + kDqWarps)) >> 1), buf = uniform(warp & 1);
    const uint32_t to = uniform(tmem) + 256u * g + 128u, ts = uniform(tmem) + 256u * g + 64u * buf;
    const uint32_t q_lo = uniform((smem_u32(sm.q[0]) >> 4) | (1u << 16));   // leading offset 16
    const uint32_t k_lo = uniform((smem_u32(sm.k[0]) >> 4) | (1u << 16));
    const uint32_t v_lo = uniform((smem_u32(sm.v[0]) >> 4) | (kHalf >> 4) << 16);
    const uint32_t s_bar = smem_u32(&sm.s_full[g][buf]), p_bar = smem_u32(&sm.p_full[g][buf]);
    const uint32_t o_bar = smem_u32(&sm.o_done[g][buf]), o_other = smem_u32(&sm.o_done[g][buf ^ 1]);
    uint32_t base_j = 0;  // tiles of the CTA before this segment
    uint32_t seg = 0;
    uint32_t done = 0;    // PV MMAs issued so far
    uint32_t other = 0;   // the other buffer's in earlier segments
    bool ok = true;
    uint32_t x = lo;
    // A segment's queries are announced by the softmax threads and by the four MMA
    // warps, each of which has seen the announcement before: a warp without a step in a
    // segment (shared rows, one tile) cannot fall two phases of q_full behind.
    if (elect_one()) mbar_arrive(smem_u32(&sm.q_full));
    __syncwarp();
    for (Segment sg; ok && next_segment(a, x, hi, sg); ++seg) {
      const int n = uniform(sg.n);
      const int row0 = kRowBlock * static_cast<int>(sg.rb % static_cast<uint32_t>(a.row_blocks));
      const bool two = uniform(a.rows - row0 > kBM ? 1u : 0u) != 0u;
      const uint32_t qd = q_lo + (two ? g : 0u) * (kTileBytes >> 4);
      if (!spin_wait(abort_flag, smem_u32(&sm.q_full), seg & 1, a.ctl)) break;
      if (elect_one()) mbar_arrive(smem_u32(&sm.q_full));
      __syncwarp();
      // Two groups of rows: step s is half s & 1 of tile s / 2, and each half of a
      // stage is freed by both groups. Shared rows: step s is half g of tile s,
      // freed by that group alone, in both arrivals.
      const int steps = two ? 2 * n : n;
      bool first = true;
      for (int at = static_cast<int>(buf); at < steps; at += 2) {
        const uint32_t h = two ? buf : g;
        const uint32_t jj = base_j + (two ? at >> 1 : at), st = uniform(jj % kStages);
        const uint32_t par = (jj / kStages) & 1;
        // S: K is there and this buffer's last PV has read P
        if (!spin_wait(abort_flag, smem_u32(&sm.k_full[st][h]), par, a.ctl) ||
            (!first && !spin_wait(abort_flag, o_bar, (done - 1) & 1, a.ctl))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t kd = k_lo + st * (kTileBytes >> 4) + h * (8192u >> 4);
        const uint32_t k_bar = smem_u32(&sm.k_empty[st][h]), v_bar = smem_u32(&sm.v_empty[st][h]);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // (descriptor addresses count 16 bytes)
            const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4;
            tc_mma_f16(ts, desc_of(qd + off), desc_of(kd + off), id_qk, kk > 0 ? 1u : 0u);
          }
          tc_commit(s_bar);
          tc_commit(k_bar);
          if (!two) tc_commit(k_bar);
        }
        __syncwarp();
        // O += P V, step after step (the last one's PV is the other buffer's): the sums'
        // order, and so the result, does not depend on which warp comes first
        if (!spin_wait(abort_flag, smem_u32(&sm.v_full[st][h]), par, a.ctl) ||
            !spin_wait(abort_flag, p_bar, done & 1, a.ctl) ||
            (at > 0 && !spin_wait(abort_flag, o_other, (other + ((at + 1) >> 1) - 1) & 1, a.ctl))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t vd = v_lo + st * (kTileBytes >> 4) + h * (8192u >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_ta(to, ts + 8u * kk, desc_of(vd + (kk * 2048u >> 4)), id_pv,
                          at > 0 || kk > 0 ? 1u : 0u);
          tc_commit(o_bar);
          tc_commit(v_bar);
          if (!two) tc_commit(v_bar);
        }
        __syncwarp();
        ++done;
        first = false;
      }
      base_j += n;
      other += (steps + buf) >> 1;
    }
    // all MMAs of this CTA complete before TMEM is released
    if (elect_one()) tc_commit(smem_u32(&sm.mma_done));
    __syncwarp();
    mbar_wait(smem_u32(&sm.mma_done), 0, 2000000000ull);
  } else {
    // ------------------------------------------------ softmax groups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int g = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_row = t_s(g) + lane_off, o_row = t_o(g) + lane_off;
    uint32_t used0 = 0, used1 = 0;  // steps of this group so far, by buffer
    bool ok = true;
    uint32_t x = lo;
    for (Segment sg; next_segment(a, x, hi, sg);) {
      const long rb = sg.rb;
      const int t_lo = sg.t_lo, n = sg.n;
      const uint32_t u32 = sg.rb / static_cast<uint32_t>(a.row_blocks);
      const long u = u32;
      const int row0 = kRowBlock * static_cast<int>(sg.rb - u32 * a.row_blocks);
      const bool two = a.rows - row0 > kBM;
      const long b = u32 / static_cast<uint32_t>(a.Hkv);
      const int kvh = static_cast<int>(u32 - static_cast<uint32_t>(b) * a.Hkv);
      const int r = row0 + (two ? kBM * g : 0) + row;  // row of the unit: token r / G, head r % G
      const int tok = r < a.rows ? r / a.G : 0, head = r - tok * a.G;
      // ---- the tree's masks and this segment's queries. Half a warp loads a
      // query row; the first four pairs of rows are in flight while the masks
      // are made. Two groups of rows: a group loads its own 128, else
      // both load 64 of the shared ones.
      const int tid = threadIdx.x;  // 0..255
      const int q_first = two ? 32 * (warp & 3) : 16 * warp;  // within the MMA tile
      const int q_r = row0 + (two ? kBM * g : 0) + q_first + (lane >> 4);
      int q_tok = q_r / a.G, q_head = q_r - q_tok * a.G, q_left = a.rows - q_r;
      uint8_t *const q_tile = sm.q[two ? g : 0];
      const uint16_t *const q_unit = a.q + u * a.G * a.T * kD + 8 * (lane & 15);
      // four rows of the lane, two apart, into w; their tokens into tk (-1: none)
      auto load_q = [&](uint4 (&w)[4], int (&tk)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t *p = q_unit + (q_head * a.T + q_tok) * kD;
          const bool on = q_left > 0 && in_bounds(a.ctl, p, 16);
          w[i] = on ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
          tk[i] = on ? q_tok : -1;
          q_left -= 2;
          q_head += 2;
          while (q_head >= a.G) q_head -= a.G, ++q_tok;
        }
      };
      uint4 qw[4];
      int qt[4];
      {
        const int32_t *p = a.parents + b * a.T;
        const bool pok = in_bounds(a.ctl, p, sizeof(int32_t) * a.T);
        if (tid < a.T) sm.par[tid] = pok ? p[tid] : -2;
        if (tid < kMaskWords) sm.live[tid] = sm.odd_v[tid] = 0u;
      }
      load_q(qw, qt);
      soft_sync();
      if (tid < a.T) {
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) sm.seen[tid][w] = 0u;
        // up the parents (each below its child) to the cache; anything else
        // met on the way: no token
        int j = tid;
        for (;;) {
          const int p = sm.par[j];
          if (p < -1 || p >= j) {
            if ((p != -2 || j != tid) && t_lo == 0 && row0 == 0 && kvh == 0)
              flag_error(a.ctl, KVQ_DEV_INDEX);
            break;
          }
          sm.seen[tid][j >> 5] |= 1u << (j & 31);
          if (p == -1) {
            atomicOr(&sm.live[tid >> 5], 1u << (tid & 31));
            break;
          }
          j = p;
        }
      }
      const bool has_tail = t_lo + n > a.int4_tiles;
      const int tail_lo = kBN * max(0, t_lo - a.int4_tiles);        // tail keys of this segment
      const int tail_hi = kBN * (t_lo + n - a.int4_tiles);
      if (has_tail) {
        // drafted tokens with a V element beyond fp16: a warp per token, four at a time
        const int j1 = min(a.T, tail_hi - a.R);
        for (int j0 = max(0, tail_lo - a.R) + warp; j0 < j1; j0 += 4 * kSoftWarps) {
          uint2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kSoftWarps;
            const uint16_t *p = a.v_tree + (u * a.T + j) * kD + 4 * lane;
            w[i] = j < j1 && in_bounds(a.ctl, p, 8) ? *reinterpret_cast<const uint2 *>(p)
                                                    : make_uint2(0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kSoftWarps;
            const bool odd = odd_bf16(w[i].x) || odd_bf16(w[i].x >> 16) || odd_bf16(w[i].y) ||
                             odd_bf16(w[i].y >> 16);
            if (__any_sync(0xffffffffu, odd) && lane == 0) atomicOr(&sm.odd_v[j >> 5], 1u << (j & 31));
          }
        }
      }
      soft_sync();
      const bool mine = r < a.rows && (sm.live[tok >> 5] >> (tok & 31) & 1u);
      const long qrow = (u * a.G + head) * a.T + tok;
#pragma unroll 1
      for (int i0 = q_first + (lane >> 4);;) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // zeros for a row without a token
          const bool on = qt[i] >= 0 && (sm.live[qt[i] >> 5] >> (qt[i] & 31) & 1u);
          *reinterpret_cast<uint4 *>(q_tile + chunk_at(i0 + 2 * i, lane & 15)) =
              on ? bf8_to_h8<true>(qw[i]) : make_uint4(0u, 0u, 0u, 0u);
        }
        i0 += 8;
        if (i0 >= q_first + (two ? 32 : 16)) break;
        load_q(qw, qt);
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(smem_u32(&sm.q_full));

      float m = -CUDART_INF_F, l = 0.0f;
#pragma unroll 1
      for (int step = 0; step < (two ? 2 * n : n); ++step) {
        const int buf = step & 1, h = two ? buf : g;
        const int tile = t_lo + (two ? step >> 1 : step);
        const uint32_t used = buf ? used1 : used0, used_other = buf ? used0 : used1;
        if (!warp_wait(abort_flag, smem_u32(&sm.s_full[g][buf]), used & 1, a.ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // Keys of the tile this row sees: all of them, else by bits (word c:
        // keys 32c .. 32c + 31): the first ones of the int4 part's last tile;
        // in the tail the window and the row's drafted tokens.
        const bool int4 = tile < a.int4_tiles;
        const int k0 = kBN * (int4 ? tile : tile - a.int4_tiles);
        const int plain = (int4 ? a.cut : a.R) - k0;  // keys from the tile's first seen by every row
        const bool all = plain >= kBN;
        auto see_word = [&](int c) -> uint32_t {
          const int s = 32 * c - plain;  // word c's first key counted from the end of those
          if (s <= -32) return ~0u;
          uint32_t bits = s < 0 ? (1u << -s) - 1u : 0u;
          if (!int4) {
            // keys past the window: drafted tokens s, s + 1, ...
            const int w = s >> 5, sh = s & 31;
            const uint32_t w0 = w >= 0 && w < kMaskWords ? sm.seen[tok][w] : 0u;
            const uint32_t w1 = w + 1 < kMaskWords ? sm.seen[tok][w + 1] : 0u;
            bits |= sh == 0 ? w0 : __funnelshift_r(w0, w1, sh);
          }
          return bits;
        };
        // ---- P over S (32 words over 64 scores). No maximum is taken as long as
        // the 64 keys' sum of P stays below kSumBound, which bounds every P of
        // it; above that (and for a row's first keys) the step is redone with a
        // reference from its maximum, and O and l follow.
        bool with_max = __any_sync(0xffffffffu, m == -CUDART_INF_F);
        uint32_t p[32];
        float s;
        for (;;) {
          float v[32], w[32];
          tmem_ld32(s_row + 64u * buf, v);
          tmem_ld32(s_row + 64u * buf + 32u, w);
          tmem_wait_ld();
          reg_fence(v);
          reg_fence(w);
          if (!all) {
            const uint32_t see0 = see_word(2 * h), see1 = see_word(2 * h + 1);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              v[e] = see0 >> e & 1u ? v[e] : -CUDART_INF_F;
              w[e] = see1 >> e & 1u ? w[e] : -CUDART_INF_F;
            }
          }
          if (with_max) {
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(fmaxf(mx, v[e]), w[e]);
            mx = mx * a.scale_log2 - kRefBias;
            const float f = mx > m ? fast_exp2(m - mx) : 1.0f;
            m = fmaxf(m, mx);
            l *= f;
            if (step > 0) {  // (before the first step there is no O)
              // O holds still once the other buffer's last PV is done (this
              // one's was before its S was issued)
              if (used_other > 0)
                ok = warp_wait(abort_flag, smem_u32(&sm.o_done[g][buf ^ 1]), (used_other - 1) & 1,
                               a.ctl);
              if (!ok) break;
              tc_fence_after();
              scale_tmem_row(o_row, f);
            }
          }
          const float neg_m = m == -CUDART_INF_F ? 0.0f : -m;
          float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float y0, y1, z0, z1;
            fma2(y0, y1, v[2 * e], v[2 * e + 1], a.scale_log2, neg_m);
            fma2(z0, z1, w[2 * e], w[2 * e + 1], a.scale_log2, neg_m);
            y0 = fast_exp2(y0);
            y1 = fast_exp2(y1);
            z0 = fast_exp2(z0);
            z1 = fast_exp2(z1);
            add2(s0, s1, y0, y1);
            add2(s2, s3, z0, z1);
            p[e] = pack_h2(y0, y1);
            p[16 + e] = pack_h2(z0, z1);
          }
          s = (s0 + s1) + (s2 + s3);
          if (with_max || !__any_sync(0xffffffffu, !(s <= kSumBound))) break;
          with_max = true;
        }
        if (!ok) break;
        l += s;
        tmem_st32u(s_row + 64u * buf, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[g][buf]));
        if (buf)
          ++used1;
        else
          ++used0;
      }
      // (after a wait that ran out: on to the barrier below, where all stop)
      if (ok && used0 > 0)
        ok = warp_wait(abort_flag, smem_u32(&sm.o_done[g][0]), (used0 - 1) & 1, a.ctl);
      if (ok && used1 > 0)
        ok = warp_wait(abort_flag, smem_u32(&sm.o_done[g][1]), (used1 - 1) & 1, a.ctl);
      // ---- write the segment's rows: the output when the slice covers all
      // of the row block's tiles, else a partial
      if (!two) {
        sm.mm[g][row] = m;
        sm.ml[g][row] = l;
      }
      tc_fence_before();
      // both groups' last PV is done and their states are there
      if (soft_sync_any(!ok || cta_aborted(abort_flag))) break;
      tc_fence_after();
      float fa = 1.0f, fb = 0.0f;
      if (!two) {
        const float ma = sm.mm[0][row], mb = sm.mm[1][row];
        m = fmaxf(ma, mb);
        fa = ma == -CUDART_INF_F ? 0.0f : fast_exp2(ma - m);
        fb = mb == -CUDART_INF_F ? 0.0f : fast_exp2(mb - m);
        l = fa * sm.ml[0][row] + fb * sm.ml[1][row];
      }
      const bool whole = n == a.tiles;
      const float inv = whole ? 1.0f / l : 1.0f;
      float *part = nullptr;  // this row's first float4, pieces kRowBlock apart
      float2 *part_ml = nullptr;
      if (!whole) {
        const int slot = static_cast<int>(blockIdx.x) - cta_of(a, rb * a.span + a.lead);
        float *p = a.partials + (rb * a.slots + slot) * kPartFloats;
        part = p + 4 * (r - row0);
        part_ml = reinterpret_cast<float2 *>(p + kRowBlock * kD) + (r - row0);
        if (!in_bounds(a.ctl, p, sizeof(float) * kPartFloats)) part = nullptr;
      }
      bool odd = false;  // a seen drafted token with a V element beyond fp16
      if (has_tail) {
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) odd |= (sm.odd_v[w] & sm.seen[tok][w]) != 0u;
      }
      // (two: all four chunks of this group's rows; shared rows: half of them each)
      for (int c = two ? 0 : 2 * g; c < (two ? 4 : 2 * g + 2); ++c) {
        float v[32];
        if (two) {
          tmem_ld32(o_row + 32u * c, v);
          tmem_wait_ld();
          reg_fence(v);
        } else {
          tmem_ld32(t_o(0) + lane_off + 32u * c, v);
          tmem_wait_ld();
          reg_fence(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= fa;
          float w[32];
          tmem_ld32(t_o(1) + lane_off + 32u * c, w);
          tmem_wait_ld();
          reg_fence(w);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = fmaf(fb, w[e], v[e]);
        }
        if (!mine) continue;
        // back to natural feature order: column 8k + i holds feature 8k + nat[i]
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int i = e & 7, nat = (i >> 1) + 4 * (i & 1);
          y[(e & ~7) + nat] = v[e] * inv;
        }
        if (!whole) {
          if (!part) continue;
          float4 *o = reinterpret_cast<float4 *>(part) + static_cast<long>(8 * c) * kRowBlock;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[e * kRowBlock] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          if (odd) put_odd_values(a, sm, u, tok, tail_lo, tail_hi, 32 * c, part, 4 * kRowBlock, false);
        } else if (a.out_dtype == KVQ_F32) {
          float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + qrow * kD + 32 * c);
          if (!in_bounds(a.ctl, o, 128)) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          if (odd)
            put_odd_values(a, sm, u, tok, tail_lo, tail_hi, 32 * c,
                           static_cast<float *>(a.out) + qrow * kD, 4, false);
        } else {
          uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + qrow * kD + 32 * c);
          if (!in_bounds(a.ctl, o, 64)) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = make_uint4(pack_bf2(y[8 * e], y[8 * e + 1]), pack_bf2(y[8 * e + 2], y[8 * e + 3]),
                              pack_bf2(y[8 * e + 4], y[8 * e + 5]),
                              pack_bf2(y[8 * e + 6], y[8 * e + 7]));
          if (odd)
            put_odd_values(a, sm, u, tok, tail_lo, tail_hi, 32 * c,
                           static_cast<uint16_t *>(a.out) + qrow * kD, 4, true);
        }
      }
      // (a row without a token leaves a partial that says so)
      if (part && r < a.rows && (two || g == 0))
        *part_ml = mine ? make_float2(m, l) : make_float2(-CUDART_INF_F, 0.0f);
      tc_fence_before();
      soft_sync();  // O, masks and states are read before the next segment rewrites them
      tc_fence_after();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kDqWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Merge of the partials of the CTAs whose slices overlap a row block (log-sum-exp),
// for 32 rows (lane = row) and, per warp, 16 features: a warp's loads are
// consecutive rows of one piece, and each thread stores whole 32-byte sectors.
// Row blocks inside one slice were written by the kernel itself. kWide (few row
// blocks, each over many CTAs): one block per 16 features, its warps take every
// eighth slot and meet in shared memory.
constexpr int kCombineWarps = 8;
// The narrow form takes a row block's slots one after the other, which the wide one
// does eight at a time with eight times the CTAs: it pays while those are few. Whole
// calls in us, wide and narrow, sequences x tokens, keys: 1 x 1, 1,024 11.2, 12.0; 4 x
// 16, 8,192 19.7, 26.0; 1 x 64, 32,768 29.4, 42.3; 8 x 8, 8,192 21.0, 23.4; 2 x 64,
// 32,768 42.5, 46.2; but 16 x 8, 8,200 32.5, 31.2; 4 x 64, 8,192 36.0, 32.4; 3 x 100,
// 16,384 63.1, 58.1.
__host__ bool wide_combine(int slots, long ctas) { return slots > 3 && 8L * slots > ctas; }

struct RowState {
  float m, l, o[16];
};
__device__ __forceinline__ void merge_slot(RowState &s, const float2 &ml, const float4 (&o)[4]) {
  if (ml.y == 0.0f) return;  // no key (a NaN sum stays in)
  const float mn = fmaxf(s.m, ml.x);
  const float ws = s.m == -CUDART_INF_F ? 0.0f : exp2f(s.m - mn);
  const float w = ml.x == -CUDART_INF_F ? 1.0f : exp2f(ml.x - mn);
  s.l = s.l * ws + ml.y * w;
  s.m = mn;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.o[4 * i] = s.o[4 * i] * ws + o[i].x * w;
    s.o[4 * i + 1] = s.o[4 * i + 1] * ws + o[i].y * w;
    s.o[4 * i + 2] = s.o[4 * i + 2] * ws + o[i].z * w;
    s.o[4 * i + 3] = s.o[4 * i + 3] * ws + o[i].w * w;
  }
}

template <bool kWide>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const TreeArgs a) {
  wait_prior_grid();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rb = blockIdx.x;
  const uint32_t u = rb / static_cast<uint32_t>(a.row_blocks);
  const int row0 = kRowBlock * static_cast<int>(rb - u * a.row_blocks);
  const int in_rb = 32 * blockIdx.y + lane, r = row0 + in_rb;
  if (row0 + 32 * static_cast<int>(blockIdx.y) >= a.rows) return;
  const int c0 = cta_of(a, static_cast<long>(rb) * a.span + a.lead);
  const int c1 = cta_of(a, static_cast<long>(rb) * a.span + a.lead + a.tiles - 1);
  const int n = c1 - c0 + 1;
  if (n == 1) return;
  const int grp = kWide ? blockIdx.z : warp;  // features 16 grp .. + 15
  const float *p = a.partials + static_cast<long>(rb) * a.slots * kPartFloats;
  if (!in_bounds(a.ctl, p, sizeof(float) * kPartFloats * n)) return;
  const float4 *po = reinterpret_cast<const float4 *>(p) + 4 * grp * kRowBlock + in_rb;
  const float2 *pml = reinterpret_cast<const float2 *>(p + kRowBlock * kD) + in_rb;
  RowState s;
  s.m = -CUDART_INF_F;
  s.l = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) s.o[e] = 0.0f;
  constexpr int kBatch = 3;  // slots in flight
  const int first = kWide ? warp : 0, step = kWide ? kCombineWarps : 1;
  for (int i0 = first; i0 < n; i0 += kBatch * step) {
    float2 ml[kBatch];
    float4 o[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * step;
      ml[k] = make_float2(-CUDART_INF_F, 0.0f);
      if (i < n) {
        ml[k] = pml[i * (kPartFloats / 2)];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] = po[i * (kPartFloats / 4) + e * kRowBlock];
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) merge_slot(s, ml[k], o[k]);
  }
  if (kWide) {
    __shared__ float2 sml[kCombineWarps][32];
    __shared__ float4 so[kCombineWarps][4][32];
    sml[warp][lane] = make_float2(s.m, s.l);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      so[warp][e][lane] = make_float4(s.o[4 * e], s.o[4 * e + 1], s.o[4 * e + 2], s.o[4 * e + 3]);
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kCombineWarps; ++w) {
      const float4 o[4] = {so[w][0][lane], so[w][1][lane], so[w][2][lane], so[w][3][lane]};
      merge_slot(s, sml[w][lane], o);
    }
  }
  if (r >= a.rows || s.l == 0.0f) return;  // (l == 0: the row holds no token)
  const float inv = 1.0f / s.l;
  const int tok = r / a.G, head = r - tok * a.G;
  const long at = ((static_cast<long>(u) * a.G + head) * a.T + tok) * kD + 16 * grp;
#pragma unroll
  for (int e = 0; e < 16; ++e) s.o[e] *= inv;
  if (a.out_dtype == KVQ_F32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
    if (!in_bounds(a.ctl, o, 64)) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = make_float4(s.o[4 * e], s.o[4 * e + 1], s.o[4 * e + 2], s.o[4 * e + 3]);
  } else {
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at);
    if (!in_bounds(a.ctl, o, 32)) return;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      o[e] = make_uint4(pack_bf2(s.o[8 * e], s.o[8 * e + 1]), pack_bf2(s.o[8 * e + 2], s.o[8 * e + 3]),
                        pack_bf2(s.o[8 * e + 4], s.o[8 * e + 5]),
                        pack_bf2(s.o[8 * e + 6], s.o[8 * e + 7]));
  }
}

struct TreePlan {
  int rows, row_blocks, int4_tiles, tiles, lead, span, ctas, slots;
  long units, items;
};

TreePlan tree_plan(const kvq_cache &c, int Hq, int T, int num_sms) {
  const CacheDims d = dims_of(c);
  TreePlan p;
  p.rows = T * (Hq / d.Hkv);
  p.row_blocks = (p.rows + kRowBlock - 1) / kRowBlock;
  p.int4_tiles = (d.cut + kBN - 1) / kBN;
  p.tiles = p.int4_tiles + (d.R + T + kBN - 1) / kBN;
  p.units = static_cast<long>(d.B) * d.Hkv;
  const long work = p.units * p.row_blocks * p.tiles;
  p.ctas = static_cast<int>(std::min<long>(work, num_sms));
  // They only balance calls whose slices hold several tiles: with a tile or
  // two a CTA every row block is split over many anyway.
  // Without them: 16 sequences of 8 tokens over 8K keys 33.5 -> 39.2 us, 16 of 64
  // over 32K 210 -> 217 us, 64 of 21 over 8K 127 -> 129 us.
  const bool several = work >= 4L * num_sms;
  p.lead = !several ? 0 : p.rows > kBM ? kLeadTwo : kLeadShared;
  p.span = p.lead + p.tiles + (several ? kTrail : 0);
  p.items = p.units * p.row_blocks * p.span;
  // a row block's tiles meet at most (tiles - 2) / min_per + 2 slices
  const long min_per = p.items / p.ctas;
  p.slots = p.tiles >= 2 ? static_cast<int>((p.tiles - 2) / min_per + 2) : 1;
  return p;
}

}  // namespace

bool tree_tensor_supported(const kvq_cache &c, int q_dtype, int tree_dtype, int Hq, int T) {
  const bool win = c.recent == 0 || (c.kwin_dtype == KVQ_BF16 && c.vwin_dtype == KVQ_BF16);
  // an MXFP8 window type rounds Q even when the window is empty
  return c.head_dim == kD && win && c.kwin_dtype != KVQ_MXFP8 && q_dtype == KVQ_BF16 &&
         tree_dtype == KVQ_BF16 &&
         static_cast<long>(T) * (Hq / c.kv_heads) <= (1L << 24) &&
         static_cast<long>(c.n_tokens) + T < (1L << 30) &&
         // items (32-bit in the kernel): row blocks of 256, tiles of 128 keys and two partial ones
         static_cast<long>(c.batch) * c.kv_heads * (static_cast<long>(T) * (Hq / c.kv_heads) / 256 + 1) *
                 (c.n_tokens / 128 + 4 + kLeadTwo + kTrail) < (1L << 30);
}

size_t tree_workspace_bytes(const kvq_cache &c, int Hq, int T, int num_sms) {
  const TreePlan p = tree_plan(c, Hq, T, num_sms);
  return sizeof(float) * static_cast<size_t>(p.units) * p.row_blocks * p.slots * kPartFloats;
}

int launch_attend_tree(const kvq_cache &c, const void *q, int Hq, int T, const void *k_tree,
                       const void *v_tree, const int32_t *parents, float scale_log2, void *out,
                       int out_dtype, void *ws, const KernelCtl &ctl, int num_sms,
                       cudaStream_t s) {
  const CacheDims d = dims_of(c);
  const TreePlan p = tree_plan(c, Hq, T, num_sms);
  TreeArgs a;
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.v_codes = c.v_codes;
  a.v_scales = c.v_scales;
  a.k_window = static_cast<const uint16_t *>(c.k_window);
  a.v_window = static_cast<const uint16_t *>(c.v_window);
  a.k_tree = static_cast<const uint16_t *>(k_tree);
  a.v_tree = static_cast<const uint16_t *>(v_tree);
  a.q = static_cast<const uint16_t *>(q);
  a.parents = parents;
  a.Hkv = d.Hkv;
  a.G = Hq / d.Hkv;
  a.T = T;
  a.R = d.R;
  a.cut = d.cut;
  a.Gk = d.Gk;
  a.Gs = d.Gs;
  a.Vs = d.Vs;
  a.Ws = d.Ws;
  a.rows = p.rows;
  a.row_blocks = p.row_blocks;
  a.int4_tiles = p.int4_tiles;
  a.tiles = p.tiles;
  a.lead = p.lead;
  a.span = p.span;
  a.items = p.items;
  a.ctas = p.ctas;
  a.slots = p.slots;
  a.scale_log2 = scale_log2;
  a.out = out;
  a.out_dtype = out_dtype;
  a.partials = static_cast<float *>(ws);
  a.ctl = ctl;
  const size_t smem = sizeof(TreeSmem) + 1024;
  if (opt_in_smem(tree_kernel, smem) != cudaSuccess) return -1;
  launch_dependent(tree_kernel, dim3(p.ctas), dim3(kThreads), smem, s, a);
  const unsigned blocks = static_cast<unsigned>(p.units * p.row_blocks);
  const unsigned groups = static_cast<unsigned>(std::min(p.rows, kRowBlock) + 31) / 32;
  if (wide_combine(p.slots, static_cast<long>(blocks) * groups))
    launch_dependent(tree_combine_kernel<true>, dim3(blocks, groups, kD / 16),
                     dim3(kCombineWarps * 32), 0, s, a);
  else
    launch_dependent(tree_combine_kernel<false>, dim3(blocks, groups), dim3(kCombineWarps * 32), 0,
                     s, a);
  return 2;
}

}  // namespace kvq
